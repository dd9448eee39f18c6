"""Layer norm of activation + residual and its gradients on the GPU against 64-bit forms.

A sum of D fp32 terms is taken as 16 of a thread's, 5 halvings in a warp and up to 32
warps: under 64 roundings deep, so off by at most 64 U32 times the sum of the
magnitudes whatever D is.  With delta that error of the mean, the sum of squared
distances is off by 64 U32 of itself and by the cross terms 2 D |distance| delta that the
warps' own means leave, that is rstd by 32 U32 + delta * rstd of itself (twice that is
allowed)."""
import pytest
import torch

import zero_optimizer_step_rs_gb300 as z
from tests import lm_ref as R

pytestmark = pytest.mark.gpu

SIZES = [(1, 8), (2, 120), (3, 128), (5, 136), (333, 256), (7, 264), (65, 512), (9, 520),
         (333, 768), (130, 1024), (11, 1032), (700, 2048), (6, 2056), (40, 4096), (3, 4104),
         (2100, 8192), (3, 8200), (5, 16384)]
EPS = 1e-5
DEEP = 64 * R.U32


def like(x, extra=0):
    y = torch.zeros_like(x, memory_format=torch.contiguous_format)
    return R.strided(y, extra) if extra else y


def forward(x, w, b, res=None, want_sum=True, extra=0, eps=EPS):
    T, D = x.shape
    y = like(x, extra)
    total = like(x, extra) if want_sum else None
    mean, rstd = (torch.full((T + 1,), 9.0, device="cuda")[1:] for _ in range(2))
    z.zero_layer_norm(x, w, b, y, mean, rstd, residual=res, sum_out=total, eps=eps)
    return y, total, mean, rstd


@pytest.mark.parametrize("T,D", SIZES)
@pytest.mark.parametrize("with_res", [False, True])
def test_forward(T, D, with_res):
    g = R.gen(T + D)
    x = R.strided(R.bf16(g, (T, D)) + 3, 24)             # a mean that is not zero
    res = R.strided(R.bf16(g, (T, D), 3.0), 8) if with_res else None
    w, b = R.bf16(g, (D,)), R.bf16(g, (D,))
    if T > 2:
        x[1] = -1.25
        if with_res:
            res[1] = 0                                   # a row of one value
    y, total, mean, rstd = forward(x, w, b, res, extra=8)
    s32 = x.float() + res.float() if with_res else x.float()
    assert torch.equal(total, s32.to(torch.bfloat16))
    s = s32.to(R.F)
    m = s.mean(1)
    d = s - m[:, None]
    r = 1 / (d.square().mean(1) + EPS).sqrt()
    delta = DEEP * s.abs().mean(1)
    R.within(mean, m, delta, "mean")
    rel = DEEP + 2 * delta * r
    R.within(rstd, r, r * rel, "rstd")
    want = d * r[:, None] * w.to(R.F) + b.to(R.F)
    size = (d * r[:, None] * w.to(R.F)).abs()
    off = size * (rel + 4 * R.U32)[:, None] + (delta * r)[:, None] * w.to(R.F).abs()
    R.within(y, want, off + (R.U16 + 2 * R.U32) * (want.abs() + off), "y")
    again = forward(x, w, b, res, want_sum=False)
    for p, q in zip((again[0], *again[2:]), (y, mean, rstd)):
        assert torch.equal(p, q)
    # without a weight, a bias or both: ones and zeros
    one, zero = torch.ones_like(w), torch.zeros_like(b)
    assert torch.equal(forward(x, None, b, res)[0], forward(x, one, b, res)[0])
    assert torch.equal(forward(x, w, None, res)[0], forward(x, w, zero, res)[0])
    assert torch.equal(forward(x, None, None, res)[0], forward(x, one, zero, res)[0])


def backward(dy, x, mean, rstd, w, dsum=None, extra=0, sides=(True, True)):
    T, D = dy.shape
    dx = like(dy, extra)
    dw, db = (torch.empty(D, dtype=torch.bfloat16, device="cuda") if s else None for s in sides)
    scratch = torch.full((z.zero_layer_norm_grad_scratch_bytes(T, D),), 255, dtype=torch.uint8,
                         device="cuda") if any(sides) else None
    z.zero_layer_norm_grad(dy, x, mean, rstd, w, dx, dw, db, scratch, dsum=dsum)
    return dx, dw, db


def check_gradient(T, D):
    g = R.gen(T * 7 + D)
    x, w, b = R.strided(R.bf16(g, (T, D), 2.0) + 1, 8), R.bf16(g, (D,)), R.bf16(g, (D,))
    _, _, mean, rstd = forward(x, w, b)
    dy = R.strided(R.bf16(g, (T, D)), 8)
    r = rstd.to(R.F)[:, None]
    h = (x.to(R.F) - mean.to(R.F)[:, None]) * r
    e = dy.to(R.F)
    for weight in (w, None):
        u = e * weight.to(R.F) if weight is not None else e
        for dsum in (None, R.strided(R.bf16(g, (T, D)), 32)):
            dx, dw, db = backward(dy, x, mean, rstd, weight, dsum, extra=8)
            inner, outer = (u * h).mean(1, keepdim=True), u.mean(1, keepdim=True)
            want = r * (u - outer - h * inner)
            size = r * (u.abs() + u.abs().mean(1, keepdim=True) +
                        h.abs() * (u * h).abs().mean(1, keepdim=True))
            if dsum is not None:
                want, size = want + dsum.to(R.F), size + dsum.to(R.F).abs()
            off = (DEEP + 16 * R.U32) * size
            R.within(dx, want, off + R.U16 * (want.abs() + off), "dx")
            for got, terms in ((dw, e * h), (db, e)):
                total = terms.sum(0)
                off = (T + 16) * R.U32 * terms.abs().sum(0)
                R.within(got, total, off + R.U16 * (total.abs() + off), "weights")
            again = backward(dy, x, mean, rstd, weight, dsum)
            assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))
            for sides in ((True, False), (False, True), (False, False)):
                some = backward(dy, x, mean, rstd, weight, dsum, sides=sides)
                assert torch.equal(some[0], dx)
                assert all(p is None or torch.equal(p, q) for p, q in zip(some[1:], (dw, db)))


@pytest.mark.parametrize("T,D", SIZES)
def test_gradient(T, D):
    check_gradient(T, D)


@pytest.mark.parametrize("T,D", [(12001, 256), (12001, 264), (12001, 512), (4001, 768),
                                 (4001, 1024), (4001, 2048), (2001, 4096), (1001, 8192),
                                 (601, 16384), (20001, 64), (9001, 120), (6001, 192), (3001, 328),
                                 (7001, 1304), (4001, 2056), (3001, 2800), (3003, 4104), (1501, 5608),
                                 (153, 1032), (305, 2048), (461, 1304)])
def test_gradient_with_more_rows_than_fit_at_once(T, D):
    check_gradient(T, D)


def test_gradient_by_differences():
    g = R.gen(4)
    T, D = 20, 384
    x, w, b, dy = R.bf16(g, (T, D)), R.bf16(g, (D,)), R.bf16(g, (D,)), R.bf16(g, (T, D))
    _, _, mean, rstd = forward(x, w, b)
    dx, dw, db = backward(dy, x, mean, rstd, w)

    def f(a, v, c):
        m = a.mean(1, keepdim=True)
        n = (a - m) / ((a - m).square().mean(1, keepdim=True) + EPS).sqrt()
        return (dy.to(R.F) * (n * v + c)).sum()
    at = [t.to(R.F) for t in (x, w, b)]
    e = 1e-4
    for i, grad in enumerate((dx, dw, db)):
        step = R.bf16(g, tuple(at[i].shape)).to(R.F)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + e * step, at[i] - e * step
        slope = (f(*up) - f(*down)) / (2 * e)            # off by the order of e^2
        assert abs((grad.to(R.F) * step).sum() - slope) <= R.U16 * grad.to(R.F).norm() * step.norm()


def test_the_sum_is_what_the_gradient_takes():
    """With a residual: the gradient from sum_out against the formula at x + residual,
    which the rounded sum is off from by U16 of each element."""
    g = R.gen(6)
    T, D = 64, 768
    x, res, w, dy = R.bf16(g, (T, D)), R.bf16(g, (T, D)), R.bf16(g, (D,)), R.bf16(g, (T, D))
    _, total, mean, rstd = forward(x, w, None, res)
    dx, dw, db = backward(dy, total, mean, rstd, w)
    s = (x.to(R.F) + res.to(R.F)).requires_grad_()
    v = w.to(R.F).requires_grad_()
    m = s.mean(1, keepdim=True)
    n = (s - m) / ((s - m).square().mean(1, keepdim=True) + EPS).sqrt()
    (dy.to(R.F) * (n * v)).sum().backward()
    # one rounding of the sum, one of the result
    R.norm_close(dx, s.grad, 2 * R.U16)
    R.norm_close(dw, v.grad, 2 * R.U16)
    R.norm_close(db, dy.to(R.F).sum(0), R.U16)


def test_values_that_are_not_finite_stay_in_their_row():
    g = R.gen(9)
    T, D = 6, 2048
    x, w, b = R.bf16(g, (T, D)), R.bf16(g, (D,)), R.bf16(g, (D,))
    clean = forward(x, w, b)
    dy = R.bf16(g, (T, D))
    clean_dx = backward(dy, x, *clean[2:], w)[0]
    x[1, 130], x[3, 5] = float("nan"), float("inf")
    got = forward(x, w, b)
    dx = backward(dy, x, *got[2:], w)[0]
    for k in (0, 2, 4, 5):
        assert all(torch.equal(p[k], q[k]) for p, q in zip(got, clean))
        assert torch.equal(dx[k], clean_dx[k])
    for k in (1, 3):
        assert bool(torch.isnan(got[0][k]).all()) and bool(torch.isnan(dx[k]).all())


@pytest.mark.parametrize("value", [0.0, 1.0, -257.0, 3e38])
@pytest.mark.parametrize("D", [8, 768, 1032, 2056, 8200])
def test_rows_of_one_value(value, D):
    """Where the variance is 0, y is the bias but for what rounding leaves of the mean."""
    x = torch.full((3, D), value, dtype=torch.bfloat16, device="cuda")
    b = R.bf16(R.gen(D), (D,))
    if value > 1e30:
        # the sum of the row passes fp32's range: Inf, and no other row is touched
        x[0], x[2] = 1.0, 2.0
    y, _, mean, rstd = forward(x, None, b)
    rows = [0, 2] if value > 1e30 else [0, 1, 2]
    v = x.to(R.F)[rows]
    delta = DEEP * v.abs().mean(1)
    R.within(mean[rows], v.mean(1), delta)
    off = (delta / EPS ** 0.5)[:, None]
    want = b.to(R.F)[None].expand(len(rows), D)
    R.within(y[rows], want, off + R.U16 * (want.abs() + off) * 1.01)


@pytest.mark.parametrize("D", [8, 72, 200, 264, 776, 1032, 2056, 4104, 8200])
def test_gradient_where_the_mean_over_the_deviation_overflows(D):
    """A row of one large value: xhat is 0, mean * rstd is past fp32's range, and the threads
    past the row's end must not make anything of that."""
    g = R.gen(D)
    T = 3
    x = torch.zeros((T, D), dtype=torch.bfloat16, device="cuda")
    x[1] = 2.0 ** 125
    dy, w = R.bf16(g, (T, D)), R.bf16(g, (D,))
    mean, rstd = x[:, 0].float().contiguous(), torch.full((T,), 300.0, device="cuda")
    dx, dw, db = backward(dy, x, mean, rstd, w)
    u = dy.to(R.F) * w.to(R.F)
    want = 300 * (u - u.mean(1, keepdim=True))
    off = (DEEP + 16 * R.U32) * 300 * (u.abs() + u.abs().mean(1, keepdim=True))
    R.within(dx, want, off + R.U16 * (want.abs() + off))
    assert not dw.any()
    R.within(db, dy.to(R.F).sum(0), (R.U16 + 8 * R.U32) * dy.to(R.F).abs().sum(0))


def test_no_tokens():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    y, _, mean, rstd = forward(e, w, w)
    dw, db = w.clone(), w.clone()
    z.zero_layer_norm_grad(e, e, mean, rstd, w, y, dw, db, None)
    assert not dw.any() and not db.any()


def test_rows_past_32_bits():
    T, D = 140_000, 16384
    x = torch.zeros((T, D), dtype=torch.bfloat16, device="cuda")
    x[-1, ::2] = 4.0
    y, _, mean, rstd = forward(x, None, None, want_sum=False)
    assert y[-1, 0].item() == 1.0 and y[-1, -1].item() == -1.0 and mean[-1].item() == 2.0
    assert not y[-2].any()
    dx, dw, db = backward(y, x, mean, rstd, None)
    assert dw[0].item() == 1.0 and db[-1].item() == -1.0
