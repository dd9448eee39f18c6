"""The losses of packed sequences where their numbers are far apart: sequences by the million, most
of them empty, as a program with buffers of a fixed size has them."""
import math
import time

import pytest
import torch

import zero_optimizer_step_rs_gb300 as z
from tests import test_gpu_lm_loss as losses
from tests.test_gpu_lm_loss import fresh, scratch_of

pytestmark = pytest.mark.gpu


def seconds(call):
    """Of the second call, from a GPU that has nothing to do until it has nothing to do again."""
    call()
    torch.cuda.synchronize()
    start = time.perf_counter()
    call()
    torch.cuda.synchronize()
    return time.perf_counter() - start


def test_many_sequences_without_tokens():
    """Their results in parallel: 2^22 of them in turn, 32 at a time, would wait for 2^17 loads of 0.3
    us each (40 ms); side by side they are 2^22 warps with two loads, under 1 ms."""
    S = 1 << 22
    e, ids = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    offsets = torch.zeros(S + 1, dtype=torch.int64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, kl, adv = fresh(S), fresh(S), torch.ones(S, device="cuda")
    clipped, counts = fresh(S, torch.int32), fresh(S, torch.int32)
    room = scratch_of(z.zero_policy_scratch_bytes, 0, S)
    assert seconds(lambda: z.zero_policy(e, e, e, adv, ids, offsets, loss, kl, clipped, counts, room,
                                         kl_coef=0.1, dev_status=status)) < 0.01
    assert status.item() == 0
    assert not (loss.any() or kl.any() or clipped.any() or counts.any())
    P = S // 2
    loss, slope, ratios, counts = fresh(P), fresh(P), fresh(S), fresh(S, torch.int32)
    room = scratch_of(z.zero_preference_scratch_bytes, 0, P)
    assert seconds(lambda: z.zero_preference(e, e, ids, offsets, loss, slope, ratios, counts, room,
                                             beta=0.5, dev_status=status)) < 0.01
    assert status.item() == 0 and not (ratios.any() or counts.any())
    assert bool((loss == loss[0]).all()) and abs(loss[0].item() - math.log(2)) < 1e-6
    assert bool((slope == -0.25).all())
    # one sequence that the tokens do not reach to
    offsets[-1] = 1
    z.zero_preference(e, e, ids, offsets, loss, slope, ratios, counts, room, dev_status=status)
    assert status.item() == z.ZERO_DEV_BAD_OFFSETS


def places(T, cuts, empty):
    """The offsets of sequences between `cuts`, with `empty` empty ones at each cut, and where the
    sequences that are not empty stand."""
    parts, at = [], []
    for k, c in enumerate(cuts):
        parts.append(torch.full((empty + 1,), c, dtype=torch.int32))
        at.append((k + 1) * (empty + 1) - 1)
    return torch.cat(parts).cuda(), torch.tensor(at[:-1], device="cuda")


@pytest.mark.parametrize("T,cuts", [
    (1000, [0, 1, 100, 900]),                     # inside of tiles of 32 tokens, tokens behind
    (1000, [96, 128, 1000]),                      # at their ends
    (90_000, [5, 700, 701, 60_000, 89_999]),      # and of larger tiles
])
@pytest.mark.parametrize("empty", [1, 30, 31, 32, 33, 62, 63, 64, 65, 1000, 1 << 20])
def test_empty_sequences_between_others(T, cuts, empty):
    """They cost next to nothing wherever they stand: in turn, 31 at a time, 2^20 at each of four cuts
    would wait for 135000 loads of 0.3 us (40 ms)."""
    g = torch.Generator(device="cuda").manual_seed(empty)
    nll, ref, old = (torch.rand(T, generator=g, device="cuda") for _ in range(3))
    targets = torch.randint(-1, 5, (T,), generator=g, device="cuda")
    few = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    offsets, at = places(T, cuts, empty)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    adv = torch.randn(offsets.numel() - 1, generator=g, device="cuda")
    dloss = torch.randn(offsets.numel() - 1, generator=g, device="cuda")

    def policy(offsets, adv, dloss):
        S = offsets.numel() - 1
        loss, kl, clipped, counts = fresh(S), fresh(S), fresh(S, torch.int32), fresh(S, torch.int32)
        room, dnll = scratch_of(z.zero_policy_scratch_bytes, T, S), fresh(T)
        args = (nll, old, ref, adv, targets, offsets)
        forward = seconds(lambda: z.zero_policy(*args, loss, kl, clipped, counts, room, kl_coef=0.1,
                                                dev_status=status))
        backward = seconds(lambda: z.zero_policy_grad(*args, counts, dloss, dnll, kl_coef=0.1))
        assert forward < 0.01 and backward < 0.01
        return loss, kl, clipped, counts, dnll
    want = policy(few, adv[at].contiguous(), dloss[at].contiguous())
    got = policy(offsets, adv, dloss)
    for a, b in zip(got[:2], want):                       # (parts may be joined in another order)
        assert torch.allclose(a[at], b, rtol=1e-6, atol=0)
        a[at] = 0
        assert not a.any()
    for a, b in zip(got[2:4], want[2:]):
        assert torch.equal(a[at], b)
        a[at] = 0
        assert not a.any()
    assert torch.equal(got[4], want[4])

    # the same places for pairs, each one's gradient what its slope and sign say
    if (offsets.numel() - 1) % 2:
        offsets = torch.cat([offsets, offsets[-1:]])
    S = offsets.numel() - 1
    P = S // 2
    loss, slope, ratios, counts = fresh(P), fresh(P), fresh(S), fresh(S, torch.int32)
    room, dnll = scratch_of(z.zero_preference_scratch_bytes, T, P), fresh(T)
    up = torch.randn(P, generator=g, device="cuda")
    assert seconds(lambda: z.zero_preference(nll, ref, targets, offsets, loss, slope, ratios, counts,
                                             room, dev_status=status)) < 0.01
    assert seconds(lambda: z.zero_preference_grad(targets, offsets, slope, counts, up, dnll)) < 0.01
    assert status.item() == 0
    want = torch.full((T,), 9.0, device="cuda")
    for s, lo, hi in zip(at.tolist(), cuts, cuts[1:]):
        live = targets[lo:hi] >= 0
        assert counts[s].item() == int(live.sum())
        q = (ref[lo:hi].double() - nll[lo:hi].double())[live]
        assert abs(ratios[s].item() - q.sum().item()) <= 16 * 2.0 ** -24 * q.abs().sum().item()
        back = up[s // 2] * slope[s // 2] * (1 if s % 2 else -1)
        want[lo:hi] = torch.where(live, back, torch.zeros_like(back))
    counts[at], ratios[at] = 0, 0
    assert torch.equal(dnll, want) and not counts.any() and not ratios.any()


@pytest.mark.parametrize("pattern", [[0, 5], [7, 0], [5, 5, 5, 0], [900, 3, 3, 1000], [3, 4, 5, 2000]])
@pytest.mark.parametrize("T", [1000, 70_000])
def test_many_offsets_that_fall(pattern, T):
    S = 1 << 20
    offsets = torch.tensor(pattern, device="cuda").repeat(S // len(pattern) + 1)[:S + 1].contiguous()
    ones = torch.ones(max(S, T), device="cuda")
    targets = torch.zeros(T, dtype=torch.int64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, kl, clipped, counts = fresh(S), fresh(S), fresh(S, torch.int32), fresh(S, torch.int32)
    room, dnll = scratch_of(z.zero_policy_scratch_bytes, T, S), fresh(T)
    args = (ones[:T], ones[:T], ones[:T], ones[:S], targets, offsets)
    assert seconds(lambda: z.zero_policy(*args, loss, kl, clipped, counts, room, dev_status=status)) < 0.05
    assert seconds(lambda: z.zero_policy_grad(*args, counts, ones[:S], dnll)) < 0.05
    assert status.item() == z.ZERO_DEV_BAD_OFFSETS


# Around where one block takes a call alone: 48 tiles of 32 tokens, 16 sequences.  With a token a lane
# a tile's sum is 5 halvings deep; the parts are joined as two fp32 numbers each, whose rest is
# off by U32 of itself: both far inside what the checks allow.
ALONE = {
    "32 tiles": (0, [64] * 16, 0),
    "a second tile for one warp": (0, [64] * 15 + [65], 0),
    "48 tiles of one sequence": (0, [1536, 0], 0),
    "48 tiles of 16 sequences": (0, [96] * 16, 0),
    "48 tiles cut anywhere": (5, [1, 0, 333, 31, 64, 33, 127, 0, 700, 2, 95, 1, 40, 77, 0, 20], 7),
    "49 tiles": (0, [96] * 15 + [97], 0),
    "18 sequences": (3, [80] * 17 + [60], 4),
    "two halves": (0, [768, 768], 0),
    "49 tiles of two sequences": (1, [1500, 31], 5),
}


@pytest.mark.parametrize("name", ALONE)
@pytest.mark.parametrize("average", [False, True])
def test_around_what_one_block_takes(name, average, monkeypatch):
    monkeypatch.setitem(losses.CASES, name, ALONE[name])
    for kind, smoothing, margin in losses.KINDS:
        losses.test_preference(name, kind, smoothing, margin, average, True, average)
    for per_token in (False, True):
        losses.test_policy(name, True, True, per_token, average, average, 0.05)
    losses.test_policy(name, False, False, False, average, True, 0.0)
