"""The residual norm with its 8-bit checkpoint on the GPU against 64-bit forms."""
import pytest
import torch

import zero_optimizer_step_rs_gb300 as z
from tests import lm_ref as R

pytestmark = pytest.mark.gpu

SIZES = [(1, 8), (2, 120), (3, 128), (5, 136), (333, 256), (7, 264), (65, 512), (9, 520),
         (333, 768), (130, 1024), (11, 1032), (700, 2048), (6, 2056), (40, 4096), (3, 4104),
         (2100, 8192), (3, 8200), (5, 16384)]
EPS = 1e-5


def forward(x, w, res=None, want_sum=True, keep=True, extra=0):
    T, D = x.shape
    y = R.strided(torch.zeros_like(x).contiguous(), extra) if extra else torch.empty_like(
        x, memory_format=torch.contiguous_format)
    total = torch.empty((T, D), dtype=torch.bfloat16, device="cuda") if want_sum else None
    codes = torch.full((T, D), 99, dtype=torch.int8, device="cuda") if keep else None
    scales = torch.full((T, -(-D // R.BLOCK)), 9.0, device="cuda") if keep else None
    rstd = torch.empty(T, device="cuda")
    z.zero_norm(x, w, y, codes, scales, rstd, residual=res, sum_out=total, eps=EPS)
    return y, total, codes, scales, rstd


@pytest.mark.parametrize("T,D", SIZES)
@pytest.mark.parametrize("with_res", [False, True])
def test_forward(T, D, with_res):
    g = R.gen(T + D)
    x = R.strided(R.bf16(g, (T, D)), 24)
    res = R.strided(R.bf16(g, (T, D), 3.0), 8) if with_res else None
    w = R.bf16(g, (D,))
    if T > 2:
        x[1] = 0
        if with_res:
            res[1] = 0                                   # a row of zeros
    y, total, codes, scales, rstd = forward(x, w, res, extra=8)
    s32 = x.float() + res.float() if with_res else x.float()
    # the sum is one fp32 addition, the checkpoint IEEE operations: the same bits
    assert torch.equal(total, s32.to(torch.bfloat16))
    want_codes, want_scales = R.checkpoint(s32)
    assert torch.equal(codes, want_codes) and torch.equal(scales, want_scales)
    s = s32.to(R.F)
    r = 1 / (s.square().mean(1) + EPS).sqrt()
    off = (D + 8) * R.U32                                # of the sum of squares, before the root
    R.within(rstd, r, r * off, "rstd")
    want = s * r[:, None] * w.to(R.F)
    R.within(y, want, want.abs() * (R.U16 + 2 * off), "y")
    # without a checkpoint or a sum: the same y
    again = forward(x, w, res, want_sum=False, keep=False)
    assert torch.equal(again[0], y) and torch.equal(again[4], rstd)


@pytest.mark.parametrize("T,D", SIZES)
def test_replay_and_gradient(T, D):
    g = R.gen(T * 7 + D)
    x, w = R.bf16(g, (T, D), 2.0), R.bf16(g, (D,))
    _, _, codes, scales, rstd = forward(x, w)
    h = R.xhat(codes, scales, rstd)
    y = R.strided(torch.zeros((T, D), dtype=torch.bfloat16, device="cuda"), 16)
    z.zero_norm_replay(codes, scales, rstd, w, y)
    want = h * w.to(R.F)
    R.within(y, want, want.abs() * (R.U16 + 8 * R.U32), "replay")
    # half a code off at most: what the checkpoint stands for, against the input
    s = x.to(R.F)
    half = scales.to(R.F).repeat_interleave(R.BLOCK, 1)[:, :D] * 0.5
    assert bool(((h / rstd.to(R.F)[:, None] - s).abs() <= half * (1 + 1e-4)).all())

    dy = R.strided(R.bf16(g, (T, D)), 8)
    scratch = torch.full((z.zero_norm_grad_scratch_bytes(T, D),), 255, dtype=torch.uint8,
                         device="cuda")
    for dsum in (None, R.strided(R.bf16(g, (T, D)), 32)):
        dx = R.strided(torch.zeros((T, D), dtype=torch.bfloat16, device="cuda"), 8)
        dw = torch.empty(D, dtype=torch.bfloat16, device="cuda")
        z.zero_norm_grad(dy, codes, scales, rstd, w, dx, dw, scratch, dsum=dsum)
        u, r = dy.to(R.F) * w.to(R.F), rstd.to(R.F)[:, None]
        inner = (u * h).mean(1, keepdim=True)
        want = r * (u - h * inner)
        size = r * (u.abs() + h.abs() * (u * h).abs().mean(1, keepdim=True))
        if dsum is not None:
            want, size = want + dsum.to(R.F), size + dsum.to(R.F).abs()
        R.within(dx, want, R.U16 * (1 + R.U16) * want.abs() + (D + 16) * R.U32 * size, "dx")
        want_w = (dy.to(R.F) * h).sum(0)
        size_w = (dy.to(R.F) * h).abs().sum(0)
        R.within(dw, want_w, R.U16 * (1 + R.U16) * want_w.abs() + (T + 16) * R.U32 * size_w, "dw")
        dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
        z.zero_norm_grad(dy, codes, scales, rstd, w, dx2, dw2, scratch, dsum=dsum)
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_gradient_by_differences():
    """Along a direction of s, with the checkpoint's own values as the input."""
    g = R.gen(4)
    T, D = 20, 384
    x, w, dy = R.bf16(g, (T, D)), R.bf16(g, (D,)), R.bf16(g, (T, D))
    _, _, codes, scales, _ = forward(x, w)
    s = codes.to(R.F) * scales.to(R.F).repeat_interleave(R.BLOCK, 1)[:, :D]
    rstd = (1 / (s.square().mean(1) + EPS).sqrt()).float()
    dx = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
    dw = torch.empty(D, dtype=torch.bfloat16, device="cuda")
    scratch = torch.empty(z.zero_norm_grad_scratch_bytes(T, D), dtype=torch.uint8, device="cuda")
    z.zero_norm_grad(dy, codes, scales, rstd, w, dx, dw, scratch)

    def f(a, b):
        return (dy.to(R.F) * a / (a.square().mean(1, keepdim=True) + EPS).sqrt() * b).sum()
    ds, db = R.bf16(g, (T, D)).to(R.F), R.bf16(g, (D,)).to(R.F)
    e = 1e-4
    slope = (f(s + e * ds, w.to(R.F)) - f(s - e * ds, w.to(R.F))) / (2 * e)
    # the differences' own error is of order e^2
    assert abs((dx.to(R.F) * ds).sum() - slope) <= R.U16 * dx.to(R.F).norm() * ds.norm()
    slope = (f(s, w.to(R.F) + e * db) - f(s, w.to(R.F) - e * db)) / (2 * e)
    assert abs((dw.to(R.F) * db).sum() - slope) <= R.U16 * dw.to(R.F).norm() * db.norm()


def test_values_that_are_not_finite_stay_in_their_row():
    g = R.gen(9)
    T, D = 6, 512
    x, w = R.bf16(g, (T, D)), R.bf16(g, (D,))
    clean = forward(x, w)
    x[1, 130] = float("nan")
    x[3, 5] = float("inf")
    x[4] = 0
    x[4, 7] = 1e-35                                     # below what a block keeps
    y, total, codes, scales, rstd = forward(x, w)
    for k in (0, 2, 5):
        assert all(torch.equal(a[k], b[k]) for a, b in zip((y, total, codes, scales, rstd), clean))
    assert bool(torch.isnan(y[1]).all())
    assert torch.isnan(scales[1]).tolist() == [False, True, False, False]
    assert torch.isnan(scales[3]).tolist() == [True, False, False, False]
    assert not codes[1, 128:256].any() and not codes[3, :128].any()
    assert not codes[4].any() and not scales[4].any()
    want_codes, want_scales = R.checkpoint(x.float())
    assert torch.equal(codes, want_codes)
    assert torch.equal(scales.nan_to_num(-1), want_scales.nan_to_num(-1))


def test_no_tokens():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    y, _, codes, scales, rstd = forward(e, w)
    z.zero_norm_replay(codes, scales, rstd, w, y)
    dw = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    scratch = torch.empty(16, dtype=torch.uint8, device="cuda")
    z.zero_norm_grad(e, codes, scales, rstd, w, y, dw, scratch)
    assert not dw.any()


def test_rows_past_32_bits():
    T, D = 140_000, 16384
    x = torch.zeros((T, D), dtype=torch.bfloat16, device="cuda")
    x[-1] = 4.0
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    y, _, codes, scales, rstd = forward(x, w, want_sum=False)
    assert y[-1, -1].item() == 1.0 and codes[-1, -1].item() == 127 and not y[-2].any()
    dw = torch.empty(D, dtype=torch.bfloat16, device="cuda")
    scratch = torch.empty(z.zero_norm_grad_scratch_bytes(T, D), dtype=torch.uint8, device="cuda")
    z.zero_norm_grad(y, codes, scales, rstd, w, x, dw, scratch)
    assert dw[0].item() == 1.0 and dw[-1].item() == 1.0
