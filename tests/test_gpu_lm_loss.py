"""Losses of packed sequences and their gradients on the GPU against 64-bit forms.

A tile's sum has at most 8 terms of a lane and 5 halvings, the tiles are joined in 64 bits: off by 13
U32 of the terms' magnitudes, and the result by one rounding (16 U32 are allowed for
both).  expf and expm1f are taken to be off by 4 U32 of their values, and an argument of
magnitude |c| that was rounded moves exp(c) by U32 |c| of it."""
import math

import pytest
import torch

import zero_optimizer_step_rs_gb300 as z
from tests import lm_ref as R

pytestmark = pytest.mark.gpu
U = R.U32
NAN = float("nan")


def offsets_of(lengths, before=0, dtype=torch.int64):
    off = [before]
    for n in lengths:
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=dtype, device="cuda")


# tokens before the first sequence, lengths, tokens behind the last one
CASES = {
    "one token": (0, [1, 0], 0),
    "one pair": (0, [5, 9], 0),
    "empty": (3, [0, 0, 0, 0], 4),
    "gaps": (7, [30, 0, 1, 0, 0, 77], 13),
    "tiles": (0, [256, 256, 512, 255, 1, 257], 0),
    "past a tile": (255, [1, 1, 300, 2], 1),
    "many short": (1, [k % 4 for k in range(1000)], 2),
    "ones": (0, [1] * 700, 0),
    "one long": (10, [50_000, 3], 5),
    "two long": (0, [3, 40_001, 0, 70_000], 0),
    "ragged": (0, [(k * 7919) % 1500 for k in range(64)], 31),
    "what one block takes": (0, [2000, 47, 0, 1], 0),
    "more than one block takes": (0, [2000, 47, 1, 1], 0),
    "sequences for more than one block": (3, [7] * 130, 0),
    "tiles of 64": (0, [64, 63, 1, 65, 128, 127], 2000),
    "around where tiles grow": (0, [60_000, 5535], 0),
    "where tiles grow": (0, [60_000, 5536], 0),
    "past where tiles grow": (1, [60_000, 100, 5437, 0], 0),
    "many short in large tiles": (5, [1, 0, 3, 200, 7] * 400, 3),
}


class Case:
    def __init__(self, name, wide=True, seed=0, holes=0.2):
        before, lengths, after = CASES[name]
        g = R.gen(seed + len(name))
        T = self.T = before + sum(lengths) + after
        self.S = len(lengths)
        self.offsets = offsets_of(lengths, before, torch.int64 if wide else torch.int32)
        ids = torch.randint(0, 1000, (T,), generator=g, device="cuda")
        ids[torch.rand(T, generator=g, device="cuda") < holes] = -1
        self.targets = ids if wide else ids.int()
        dead = ids < 0
        dead[:before] = True
        dead[T - after:] = True
        self.seq = [(int(a), int(b)) for a, b in zip(self.offsets, self.offsets[1:])]

        def values(base, sigma):
            """One element past a 16-byte boundary; NaN and Inf where nothing counts."""
            x = torch.empty(T + 1, device="cuda")[1:]
            x.copy_(base + torch.randn(T, generator=g, device="cuda") * sigma)
            x[dead] = NAN
            x[dead & (torch.arange(T, device="cuda") % 2 == 0)] = math.inf
            return x
        base = torch.rand(T, generator=g, device="cuda") * 8
        self.nll, self.ref, self.old = values(base, 0.0), values(base, 0.5), values(base, 0.3)
        self.per_token = values(torch.zeros(T, device="cuda"), 1.0)
        self.advantages = torch.randn(self.S, generator=g, device="cuda")
        self.advantages[::5] = 0
        self.live = ids >= 0
        self.inside = torch.zeros(T, dtype=torch.bool, device="cuda")
        self.inside[before:T - after] = True
        self.g = g

    def sums(self, x):
        """Over each sequence's tokens that count, and how many they are."""
        out = torch.zeros(self.S, dtype=R.F, device="cuda")
        n = torch.zeros(self.S, dtype=R.F, device="cuda")
        for s, (a, b) in enumerate(self.seq):
            at = self.live[a:b]
            out[s], n[s] = x[a:b][at].to(R.F).sum(), at.sum()
        return out, n

    def spread(self, x):
        """A number per sequence as one per token (0 outside)."""
        out = torch.zeros(self.T, dtype=R.F, device="cuda")
        for s, (a, b) in enumerate(self.seq):
            out[a:b] = x[s]
        return out


def check_tokens(c, got, want, off, what):
    """dnll: within bounds where a token counts, 0 where it does not, untouched outside."""
    counts = c.inside & c.live
    R.within(got[counts], want[counts], off[counts], what)
    assert not got[c.inside & ~c.live].any()
    assert bool((got[~c.inside] == 9).all())


def fresh(n, dtype=torch.float32):
    return torch.full((n + 1,), 9, dtype=dtype, device="cuda")[1:]


def scratch_of(size, *args):
    return torch.full((size(*args),), 255, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------ preference --

KINDS = [(z.ZERO_PREF_SIGMOID, 0.0, 0.0), (z.ZERO_PREF_SIGMOID, 0.2, 0.7),
         (z.ZERO_PREF_HINGE, 0.0, -0.3), (z.ZERO_PREF_IPO, 0.0, 0.25)]


def preference(c, kind=0, smoothing=0.0, margin=0.0, beta=0.1, average=False, ref=True,
               dloss=None, status=None, stream=None):
    P = c.S // 2
    loss, slope, ratios, counts = fresh(P), fresh(P), fresh(c.S), fresh(c.S, torch.int32)
    z.zero_preference(c.nll, c.ref if ref else None, c.targets, c.offsets, loss, slope, ratios,
                      counts, scratch_of(z.zero_preference_scratch_bytes, c.T, P), kind=kind,
                      beta=beta, smoothing=smoothing, margin=margin, average=average,
                      dev_status=status, stream=stream)
    dnll = fresh(c.T)
    if dloss is not None:
        z.zero_preference_grad(c.targets, c.offsets, slope, counts, dloss, dnll, average=average,
                               stream=stream)
    return loss, slope, ratios, counts, dnll


def preference_loss(d, kind, smoothing, margin, beta):
    """The loss, and its derivative by d."""
    zz = beta * d - margin
    if kind == z.ZERO_PREF_IPO:
        e = d - margin - 0.5 / beta
        return e * e, 2 * e
    if kind == z.ZERO_PREF_HINGE:
        return (1 - zz).clamp(min=0), -beta * (zz < 1).to(R.F)
    sp = torch.nn.functional.softplus
    return ((1 - smoothing) * sp(-zz, threshold=100) + smoothing * sp(zz, threshold=100),
            beta * (smoothing * torch.sigmoid(zz) - (1 - smoothing) * torch.sigmoid(-zz)))


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("kind,smoothing,margin", KINDS)
@pytest.mark.parametrize("average,ref,wide", [(False, True, True), (True, True, False),
                                              (True, False, True)])
def test_preference(name, kind, smoothing, margin, average, ref, wide):
    c = Case(name, wide)
    P, beta = c.S // 2, 0.1
    dloss = torch.randn(P, generator=c.g, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, slope, ratios, counts, dnll = preference(c, kind, smoothing, margin, beta, average, ref,
                                                   dloss, status)
    assert status.item() == 0
    terms = (c.ref.to(R.F) if ref else 0) - c.nll.to(R.F)
    q, n = c.sums(terms)
    size, _ = c.sums(terms.abs())
    assert torch.equal(counts.to(R.F), n)
    share = 1 / n.clamp(min=1) if average else torch.ones_like(n)
    q, off = q * share, 16 * U * size * share
    R.within(ratios, q, off, "ratios")
    d, d_off = q[0::2] - q[1::2], off[0::2] + off[1::2]
    want, by_d = preference_loss(d, kind, smoothing, margin, beta)
    if kind == z.ZERO_PREF_SIGMOID:
        zz = beta * d - margin
        rel = beta * d_off + U * zz.abs() + 16 * U
        R.within(loss, want, want * rel, "loss")
        s_off = rel * beta * (smoothing * torch.sigmoid(zz) + (1 - smoothing) * torch.sigmoid(-zz))
    elif kind == z.ZERO_PREF_IPO:
        e = (d - margin - 0.5 / beta).abs()
        R.within(loss, want, 2 * e * d_off + d_off ** 2 + 2 * U * want, "loss")
        s_off = 2 * d_off + 2 * U * by_d.abs()
    else:
        R.within(loss, want, beta * d_off + 2 * U * want, "loss")
        s_off = 2 * U * by_d.abs()
    R.within(slope, by_d, s_off, "slope")
    sign = torch.tensor([-1.0, 1.0], dtype=R.F, device="cuda").repeat(P)
    back = dloss.to(R.F).repeat_interleave(2) * sign * share
    g = c.spread(by_d.repeat_interleave(2) * back)
    g_off = c.spread(s_off.repeat_interleave(2) * back.abs()) + 4 * U * g.abs()
    check_tokens(c, dnll, g, g_off, "dnll")
    again = preference(c, kind, smoothing, margin, beta, average, ref, dloss)
    assert all(torch.equal(a, b) for a, b in zip(again, (loss, slope, ratios, counts, dnll)))


def test_preference_of_far_pairs():
    """Differences of hundreds: neither side overflows, and the loss does not vanish early."""
    c = Case("one pair", holes=0.0)
    for shift in (-3000.0, -900.0, -300.0, 300.0, 900.0, 3000.0):
        c.nll[:5] = 1.0 + shift / 5
        c.ref[:5], c.nll[5:], c.ref[5:] = 1.0, 1.0, 1.0
        loss, slope, ratios, _, _ = preference(c)
        want, by_d = preference_loss(torch.tensor(-shift, dtype=R.F), 0, 0.0, 0.0, 0.1)
        R.within(loss, want.cuda()[None], want.item() * 400 * U + 2.0 ** -140)
        R.within(slope, by_d.cuda()[None], abs(by_d.item()) * 400 * U + 2.0 ** -140)


def test_preference_values_that_are_not_finite_stay_in_their_pair():
    c = Case("ragged")
    clean = preference(c, dloss=torch.ones(c.S // 2, device="cuda"))
    a, b = c.seq[9]
    at = a + int(c.live[a:b].nonzero()[0])
    for bad in (NAN, math.inf, -math.inf):
        c.nll[at] = bad
        got = preference(c, dloss=torch.ones(c.S // 2, device="cuda"))
        other = torch.arange(c.S // 2, device="cuda") != 4
        assert all(torch.equal(x[other], y[other]) for x, y in zip(got[:2], clean[:2]))
        assert math.isnan(got[0][4].item()) == math.isnan(bad)
        if bad == math.inf:                                 # the rejected one is impossible
            assert got[0][4].item() == 0 and got[1][4].item() == 0
        if bad == -math.inf:
            assert got[0][4].item() == math.inf and got[1][4].item() == pytest.approx(-0.1)


def test_preference_by_differences():
    c = Case("gaps")
    dloss = torch.randn(c.S // 2, generator=c.g, device="cuda")
    step = torch.randn(c.T, generator=c.g, device="cuda").to(R.F) * (c.live & c.inside)
    for kind, smoothing, margin in KINDS:
        for average in (False, True):
            dnll = preference(c, kind, smoothing, margin, 0.1, average, True, dloss)[4]

            def f(e):
                q, n = c.sums(c.ref.to(R.F) - (c.nll.to(R.F) + e * step))
                if average:
                    q = q / n.clamp(min=1)
                return (preference_loss(q[0::2] - q[1::2], kind, smoothing, margin, 0.1)[0] *
                        dloss.to(R.F)).sum().item()
            slope = (f(1e-5) - f(-1e-5)) / 2e-5
            at = c.live & c.inside
            got = (dnll[at].to(R.F) * step[at]).sum().item()
            size = (dnll[at].to(R.F) * step[at]).abs().sum().item()
            assert abs(got - slope) <= 1e-6 * size + 1e-8


# ---------------------------------------------------------------- policy --

def policy(c, old=True, ref=True, per_token=False, low=0.2, high=0.28, kl_coef=0.05, average=True,
           dloss=None, status=None, stream=None):
    adv = c.per_token if per_token else c.advantages
    how = dict(per_token=per_token, clip_low=low, clip_high=high, kl_coef=kl_coef, average=average,
               stream=stream)
    args = (c.nll, c.old if old else None, c.ref if ref else None, adv, c.targets, c.offsets)
    loss, kl = fresh(c.S), fresh(c.S)
    clipped, counts = fresh(c.S, torch.int32), fresh(c.S, torch.int32)
    z.zero_policy(*args, loss, kl, clipped, counts,
                  scratch_of(z.zero_policy_scratch_bytes, c.T, c.S), dev_status=status, **how)
    dnll = fresh(c.T)
    if dloss is not None:
        z.zero_policy_grad(*args, counts, dloss, dnll, **how)
    return loss, kl, clipped, counts, dnll


def policy_terms(c, nll, old, ref, per_token, low, high, kl_coef):
    """Each token's term, estimate and derivative in 64 bits, whether it is clipped, and bounds."""
    x = nll.to(R.F)
    change = c.old.to(R.F) - x if old else torch.zeros_like(x)
    r = change.exp()
    A = (c.per_token.to(R.F) if per_token else c.spread(c.advantages))
    over = torch.where(A > 0, change > math.log1p(high),
                       (A < 0) & (change < (math.log1p(-low) if low < 1 else -math.inf)))
    bound = torch.where(A > 0, 1 + high, 1 - low)
    surrogate = -torch.where(over, bound, r) * A
    d = x - c.ref.to(R.F) if ref else torch.zeros_like(x)
    k = torch.expm1(d) - d
    term = surrogate + kl_coef * k
    slope = torch.where(over, torch.zeros_like(r), r * A) + kl_coef * torch.expm1(d)
    s_off = surrogate.abs() * (U * change.abs() + 6 * U)
    e1 = torch.expm1(d).abs()
    k_off = U * d.abs() * e1 + 16 * U * k + torch.where(d.abs() > 1, 4 * U * (e1 + d.abs()), 0.0)
    t_off = s_off + kl_coef * (k_off + 2 * U * k) + U * term.abs()
    g_off = ((r * A).abs() * (U * change.abs() + 6 * U) +
             kl_coef * (U * d.abs() * d.exp() + 6 * U * e1))
    return term, k, over, slope, t_off, k_off, g_off


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("old,ref,per_token,average,wide,kl_coef", [
    (True, True, False, True, True, 0.05), (True, True, True, False, False, 0.05),
    (False, True, True, True, True, 1.5), (True, False, False, False, True, 0.0),
    (True, True, False, False, False, 0.0), (False, False, True, True, True, 0.0)])
def test_policy(name, old, ref, per_token, average, wide, kl_coef):
    c = Case(name, wide, seed=3)
    low, high = 0.2, 0.28
    dloss = torch.randn(c.S, generator=c.g, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, kl, clipped, counts, dnll = policy(c, old, ref, per_token, low, high, kl_coef, average,
                                             dloss, status)
    assert status.item() == 0
    term, k, over, slope, t_off, k_off, g_off = policy_terms(c, c.nll, old, ref, per_token, low,
                                                             high, kl_coef)
    want, n = c.sums(term)
    share = 1 / n.clamp(min=1) if average else torch.ones_like(n)
    off = c.sums(t_off + 16 * U * term.abs())[0]
    assert torch.equal(counts.to(R.F), n)
    assert torch.equal(clipped.to(R.F), c.sums(over.to(R.F))[0])
    R.within(loss, want * share, off * share + 2 * U * (want * share).abs(), "loss")
    want, off = c.sums(k)[0], c.sums(k_off + 16 * U * k)[0]
    R.within(kl, want * share, off * share + 2 * U * want * share, "kl")
    back = c.spread(dloss.to(R.F) * share)
    g = slope * back
    check_tokens(c, dnll, g, g_off * back.abs() * 1.01 + 8 * U * g.abs(), "dnll")
    again = policy(c, old, ref, per_token, low, high, kl_coef, average, dloss)
    assert all(torch.equal(a, b) for a, b in zip(again, (loss, kl, clipped, counts, dnll)))


def test_policy_at_its_bounds():
    """Ratios at, just above and just below either bound: decided on the exact difference."""
    low, high = 0.2, 0.28
    edges = [math.log1p(high), math.log1p(-low)]
    change = torch.tensor(edges, dtype=R.F).repeat_interleave(600)
    near = change.float()
    old = torch.rand(1200, generator=torch.Generator().manual_seed(1)) * 0.7
    nll = old - near                        # rounded: differences spread around the bound
    c = Case("one pair")
    c.T, c.S = 1200, 1
    c.nll, c.old, c.ref = nll.cuda(), old.cuda(), old.cuda()
    c.targets = torch.zeros(1200, dtype=torch.int64, device="cuda")
    c.offsets = torch.tensor([0, 1200], device="cuda")
    exact = old.to(R.F) - nll.to(R.F)
    for sign in (1.0, -1.0):
        c.advantages = torch.tensor([sign], device="cuda")
        clipped = policy(c, low=low, high=high, dloss=torch.ones(1, device="cuda"))
        over = exact > edges[0] if sign > 0 else exact < edges[1]
        assert clipped[2].item() == int(over.sum()) and 100 < int(over.sum()) < 1100
        got = policy(c, low=low, high=high, kl_coef=0.0, dloss=torch.ones(1, device="cuda"),
                     average=False)[4]
        assert torch.equal(got.cpu() == 0, over)


@pytest.mark.parametrize("low,high", [(0.0, 0.0), (1.0, 0.0), (0.0, 1e6), (1.0, 1e6)])
def test_policy_with_other_bounds(low, high):
    c = Case("ragged")
    _, _, clipped, _, dnll = policy(c, low=low, high=high, dloss=torch.ones(c.S, device="cuda"),
                                    average=False)
    _, _, over, slope, _, _, g_off = policy_terms(c, c.nll, True, True, False, low, high, 0.05)
    assert torch.equal(clipped.to(R.F), c.sums(over.to(R.F))[0])
    check_tokens(c, dnll, slope, 1.01 * g_off + 8 * U * slope.abs(), "dnll")


def test_policy_of_far_tokens():
    """Losses far apart: a bounded ratio stays bounded, an advantage of 0 gives 0."""
    c = Case("one pair", holes=0.0)
    c.advantages = torch.tensor([2.0, 0.0], device="cuda")
    c.nll[:], c.old[:], c.ref[:] = 1.0, 1.0, 1.0
    c.old[0] = c.old[6] = 500.0                            # r = Inf
    loss, kl, clipped, _, dnll = policy(c, kl_coef=0.0, dloss=torch.ones(2, device="cuda"),
                                        average=False)
    assert loss[0].item() == pytest.approx(-2 * (4 + 1.28), rel=1e-6) and loss[1].item() == 0
    assert clipped.tolist() == [1, 0] and not dnll[5:].any() and dnll[0].item() == 0
    assert bool((dnll[1:5] == 2).all())


def test_kl_estimates_of_all_sizes():
    """exp(d) - d - 1 keeps its relative accuracy down to the smallest differences."""
    d = torch.cat([s * torch.logspace(-12, 1.2, 400) for s in (1, -1)]).float().cuda()
    c = Case("one pair")
    c.T = c.S = d.numel()
    c.ref = torch.zeros(c.T, device="cuda")
    c.nll, c.old = d.clone(), d.clone()
    c.targets = torch.zeros(c.T, dtype=torch.int64, device="cuda")
    c.offsets = torch.arange(c.T + 1, device="cuda")
    c.advantages = torch.zeros(c.T, device="cuda")
    _, kl, _, _, dnll = policy(c, kl_coef=1.0, dloss=torch.ones(c.S, device="cuda"))
    x = d.to(R.F)
    # exp(x) - x - 1 as a sum of its series' terms, without cancellation, where x is small
    small = sum(x ** n / float(math.factorial(n)) for n in range(2, 22))
    want = torch.where(x.abs() < 1, small, torch.expm1(x) - x)
    e1 = torch.expm1(x).abs()
    off = 16 * U * want + torch.where(x.abs() > 1, 4 * U * (e1 + x.abs()), 0.0)
    R.within(kl, want, off)
    R.within(dnll, torch.expm1(x), 8 * U * e1)


def test_policy_by_differences():
    c = Case("gaps")
    dloss = torch.randn(c.S, generator=c.g, device="cuda")
    at = c.live & c.inside
    step = torch.randn(c.T, generator=c.g, device="cuda").to(R.F) * at
    for per_token in (False, True):
        dnll = policy(c, per_token=per_token, dloss=dloss, average=False)[4]

        def f(e):
            term = policy_terms(c, c.nll.to(R.F) + e * step, True, True, per_token, 0.2, 0.28,
                                0.05)[0]
            return (c.sums(term)[0] * dloss.to(R.F)).sum().item()
        slope = (f(1e-6) - f(-1e-6)) / 2e-6                # no bound is that near
        got = (dnll[at].to(R.F) * step[at]).sum().item()
        size = (dnll[at].to(R.F) * step[at]).abs().sum().item()
        assert abs(got - slope) <= 1e-6 * size + 1e-8


# ------------------------------------------------------------------ both --

@pytest.mark.parametrize("bad", [[5, 3, 9, 20, 21], [-4, 3, 9, 20, 21], [0, 3, 9, 20, 1 << 40],
                                 [1 << 40, 0, 3, 4, 5], [40, 30, 20, 10, 0], [0, 3, 9, 20, 41]])
@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
def test_bad_offsets_are_reported(bad, dtype):
    """What the offsets say is bounded by T wherever an address is made from it."""
    c = Case("one pair")
    c.T, c.S = 40, 4
    c.nll, c.ref, c.old = (torch.ones(40, device="cuda") for _ in range(3))
    c.targets = torch.zeros(40, dtype=torch.int64, device="cuda")
    c.advantages = torch.ones(4, device="cuda")
    c.offsets = torch.tensor([min(b, 2 ** 31 - 1) for b in bad] if dtype == torch.int32 else bad,
                             dtype=dtype, device="cuda")
    dloss = {preference: torch.ones(2, device="cuda"), policy: torch.ones(4, device="cuda")}
    for call in (preference, policy):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(c, status=status, dloss=dloss[call])
        assert status.item() == z.ZERO_DEV_BAD_OFFSETS
        call(c)                                             # nobody asks


def test_no_sequences_and_no_tokens():
    e, i = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    n, room = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(256, dtype=torch.uint8,
                                                                           device="cuda")
    none, five = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(7, dtype=torch.int64, device="cuda")
    z.zero_preference(e, e, i, none, e, e, e, n, room)
    z.zero_policy(e, e, e, e, i, none, e, e, n, n, room)
    loss, slope, ratios, counts = fresh(3), fresh(3), fresh(6), fresh(6, torch.int32)
    z.zero_preference(e, e, i, five, loss, slope, ratios, counts, room)
    assert torch.allclose(loss, torch.full_like(loss, math.log(2))) and not counts.any()
    assert not ratios.any()
    z.zero_preference_grad(i, five, slope, counts, loss, e)
    clipped, n6 = fresh(6, torch.int32), fresh(6, torch.int32)
    kl, l6 = fresh(6), fresh(6)
    z.zero_policy(e, None, None, torch.ones(6, device="cuda"), i, five, l6, kl, clipped, n6, room)
    assert not (l6.any() or kl.any() or clipped.any() or n6.any())


def test_tokens_up_to_the_last_that_32_bits_count():
    """2^31 - 1024 tokens: addresses past 32 bits, counts that fp32 does not hold."""
    T = (1 << 31) - 1024
    cut = [1, 1 << 30, T - 301, T - 300]
    off = torch.tensor([0, *cut[:3], T], dtype=torch.int32, device="cuda")
    targets = torch.zeros(T, dtype=torch.int32, device="cuda")
    nll = torch.zeros(T, device="cuda")
    nll[-200:] = 2.0
    targets[-100:] = -1
    nll[-50:] = NAN
    nll[(1 << 30) + 5] = 1e6
    dnll = torch.full((T,), 9.0, device="cuda")
    f = lambda n: torch.zeros(n, device="cuda")  # noqa: E731
    loss, slope, ratios, counts = f(2), f(2), f(4), torch.zeros(4, dtype=torch.int32, device="cuda")
    lengths = [1, (1 << 30) - 1, T - 301 - (1 << 30), 301 - 100]
    for average in (False, True):
        room = scratch_of(z.zero_preference_scratch_bytes, T, 2)
        z.zero_preference(nll, None, targets, off, loss, slope, ratios, counts, room, average=average)
        assert counts.tolist() == lengths
        n = [lengths[2], lengths[3]] if average else [1, 1]
        assert ratios.tolist() == pytest.approx([0.0, 0.0, -1e6 / n[0], -200.0 / n[1]], rel=1e-6)
        z.zero_preference_grad(targets, off, slope, counts, torch.ones(2, device="cuda"), dnll, average=average)
        n = lengths[1] if average else 1
        assert dnll[1].item() == dnll[(1 << 30) - 1].item() == pytest.approx(-0.05 / n, rel=1e-6)
        assert not dnll[-100:].any() and dnll[-101].item() < 0
    loss, kl, cut_n, n4 = f(4), f(4), *(torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(2))
    room = scratch_of(z.zero_policy_scratch_bytes, T, 4)
    adv = torch.tensor([1.0, 2.0, 3.0, -4.0], device="cuda")
    z.zero_policy(nll, None, None, adv, targets, off, loss, kl, cut_n, n4, room)
    assert n4.tolist() == lengths and loss.tolist() == [-1.0, -2.0, -3.0, 4.0]
    z.zero_policy_grad(nll, None, None, adv, targets, off, n4, torch.ones(4, device="cuda"), dnll)
    assert dnll[-101].item() == pytest.approx(-4 / lengths[3], rel=1e-6) and not dnll[-100:].any()
    assert dnll[0].item() == 1.0 and dnll[5].item() == pytest.approx(2 / lengths[1], rel=1e-6)


def test_two_calls_at_once():
    """On two streams, each with its own scratch and outputs."""
    cases = [Case("ragged", seed=k) for k in range(2)]
    dloss = [torch.ones(c.S, device="cuda") for c in cases]
    want = [policy(c, dloss=d) for c, d in zip(cases, dloss)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for c, d, s in zip(cases, dloss, streams):
            with torch.cuda.stream(s):
                got.append(policy(c, dloss=d))
    torch.cuda.synchronize()
    for k, result in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(result, want[k % 2]))


@pytest.mark.parametrize("name", ["gaps", "two long"])
def test_another_stream_and_a_graph(name):
    c = Case(name)
    P = c.S // 2
    d_pair, d_seq = torch.ones(P, device="cuda"), torch.ones(c.S, device="cuda")
    out = [torch.zeros(n, device="cuda") for n in (P, P, c.S, c.T, c.S, c.S, c.T)]
    n = [torch.zeros(c.S, dtype=torch.int32, device="cuda") for _ in range(3)]
    a = scratch_of(z.zero_preference_scratch_bytes, c.T, P)
    b = scratch_of(z.zero_policy_scratch_bytes, c.T, c.S)
    args = (c.nll, c.old, c.ref, c.advantages, c.targets, c.offsets)

    def calls(stream=None):
        z.zero_preference(c.nll, c.ref, c.targets, c.offsets, *out[:3], n[0], a, stream=stream)
        z.zero_preference_grad(c.targets, c.offsets, out[1], n[0], d_pair, out[3], stream=stream)
        z.zero_policy(*args, *out[4:6], n[1], n[2], b, kl_coef=0.1, stream=stream)
        z.zero_policy_grad(*args, n[2], d_seq, out[6], kl_coef=0.1, stream=stream)
    calls()
    want = [x.clone() for x in (*out, *n)]

    def same():
        torch.cuda.synchronize()
        assert all(torch.equal(x, w) for x, w in zip((*out, *n), want))
        for x in (*out, *n):
            x.zero_()
    same()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    calls(s)
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(2):
        graph.replay()
        same()
