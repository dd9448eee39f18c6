"""Plain 64-bit forms of the language-model operators, and the bounds their
kernels are held to.  Every bound follows from the types: U16 is the relative
error of one rounding to bf16, U32 of one fp32 operation; a sum of n fp32
terms is off by at most n * U32 times the sum of the magnitudes (2 * U32 a
term on the tensor cores, which may truncate)."""
import torch

U16 = 2.0 ** -8
U32 = 2.0 ** -24
BLOCK = 128
F = torch.float64


def bf16(g, shape, sigma=1.0, device="cuda"):
    return (torch.randn(shape, generator=g, device=device) * sigma).to(torch.bfloat16)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def strided(x, extra, filler=float("nan")):
    """The same rows with `extra` columns of filler behind each."""
    T, D = x.shape
    big = torch.full((T, D + extra), filler, dtype=x.dtype, device=x.device)
    big[:, :D] = x
    return big[:, :D]


def within(got, want, bound, what=""):
    """Every element within its bound; NaN exactly where wanted."""
    got, want = got.to(F), want.to(F)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    ok = ((got - want).abs() <= bound) | torch.isnan(want) | (got == want)
    if not bool(ok.all()):
        i = int((~ok).flatten().nonzero()[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} off, first at {i}: "
                             f"{got.flatten()[i].item()} for {want.flatten()[i].item()}")


def norm_close(got, want, bound, what=""):
    """The 2-norm of the difference over the 2-norm of the result."""
    got, want = got.to(F), want.to(F)
    n = want.norm().item()
    off = (got - want).norm().item()
    assert off <= bound * n, f"{what}: {off / n if n else off} over {bound}"


# ------------------------------------------------------------- embedding --

def embed_grad(dy, tokens, V, scale, base=None):
    """(the sums, the magnitudes that went into them, how many terms)"""
    D = dy.shape[1]
    out = torch.zeros((V, D), dtype=F, device=dy.device)
    mag = torch.zeros_like(out)
    n = torch.zeros(V, dtype=F, device=dy.device)
    at = ((tokens >= 0) & (tokens < V)).nonzero()[:, 0]
    t = tokens[at].long()
    part = dy[at].to(F) * float(torch.tensor(scale, dtype=torch.float32))
    out.index_add_(0, t, part)
    mag.index_add_(0, t, part.abs())
    n.index_add_(0, t, torch.ones_like(t, dtype=F))
    if base is not None:
        out += base.to(F)
        mag += base.to(F).abs()
    return out, mag, n


# ------------------------------------------------------------------ norm --

def checkpoint(total):
    """codes and scales of a 32-bit matrix, bit for bit (IEEE operations)."""
    T, D = total.shape
    nb = -(-D // BLOCK)
    codes = torch.zeros((T, D), dtype=torch.int8, device=total.device)
    scales = torch.zeros((T, nb), dtype=torch.float32, device=total.device)
    for b in range(nb):
        part = total[:, b * BLOCK:(b + 1) * BLOCK]
        amax = part.abs().amax(1)                       # NaN stays NaN
        full = torch.full_like(amax, 127.0)
        bad = ~torch.isfinite(amax)
        used = (amax >= torch.tensor(1e-30)) & ~bad
        one = torch.ones_like(amax)
        scale = torch.where(used, torch.where(used, amax, one) / full, torch.zeros_like(amax))
        inv = torch.where(used, full / torch.where(used, amax, one), torch.zeros_like(amax))
        scales[:, b] = torch.where(bad, torch.full_like(amax, float("nan")), scale)
        q = torch.round(part * inv[:, None])
        codes[:, b * BLOCK:(b + 1) * BLOCK] = torch.where(torch.isnan(q), torch.zeros_like(q),
                                                          q).to(torch.int8)
    return codes, scales


def xhat(codes, scales, rstd):
    spread = scales.to(F).repeat_interleave(BLOCK, 1)[:, : codes.shape[1]]
    return codes.to(F) * spread * rstd.to(F)[:, None]


# --------------------------------------------------------- cross entropy --

def logits(h, table):
    """The logits and the largest error an fp32 sum of their terms may have, per row."""
    l = h.to(F) @ table.to(F).T
    mag = (h.to(F).abs() @ table.to(F).abs().T).amax(1)
    return l, h.shape[1] * 2 * U32 * mag


def live(targets, V):
    return (targets >= 0) & (targets < V)


def xent(h, table, targets):
    """loss, lse and their bound: the logits' error, and the exponentials' (an
    argument of magnitude |l| rounded in fp32, an approximate exp2 and sums of
    up to V terms joined tile by tile: under 2^-18 together)."""
    l, off = logits(h, table)
    lse = torch.logsumexp(l, 1)
    ok = live(targets, table.shape[0])
    at = l.gather(1, torch.where(ok, targets, torch.zeros_like(targets)).long()[:, None])[:, 0]
    loss = torch.where(ok, lse - at, torch.zeros_like(lse))
    return loss, lse, 2 * off + 2.0 ** -18 + 2.0 ** -21 * (lse.abs() + l.abs().amax(1))


def xent_grad(h, table, targets, lse, dloss):
    """dh, dtable, and elementwise bounds: P is off by U16 (its rounding) and
    the exponential's relative error, the sums by their fp32 terms, the result
    by its own rounding."""
    V = table.shape[0]
    l, off = logits(h, table)
    ok = live(targets, V)
    p = torch.exp(l - lse.to(F)[:, None])
    rel = off + 2.0 ** -18 + 2.0 ** -21 * (lse.to(F).abs() + l.abs().amax(1))
    p_off = p * rel[:, None]
    p[ok, targets[ok].long()] -= 1
    g = torch.where(ok, dloss.to(F), torch.zeros_like(dloss, dtype=F))
    p = torch.where(ok[:, None], p * g[:, None], torch.zeros_like(p))
    p_off = torch.where(ok[:, None], p_off * g[:, None].abs(), torch.zeros_like(p)) + p.abs() * U16
    hc = torch.where(ok[:, None], h.to(F), torch.zeros_like(h, dtype=F))
    e = table.to(F)
    dh, dt = p @ e, p.T @ hc
    bh = (p_off + p.abs() * V * 2 * U32) @ e.abs() + 2 * U16 * dh.abs()
    bt = (p_off + p.abs() * h.shape[0] * 2 * U32).T @ hc.abs() + 2 * U16 * dt.abs()
    return dh, dt, bh, bt
