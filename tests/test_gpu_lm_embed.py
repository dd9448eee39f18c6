"""The embedding lookup and its gradient on the GPU against 64-bit forms."""
import math

import pytest
import torch

import zero_optimizer_step_rs_gb300 as z
from tests import lm_ref as R
from zero_optimizer_step_rs_gb300 import binding as B

pytestmark = pytest.mark.gpu


def ids(g, T, V, kind, dtype=torch.int64):
    if kind == "same":
        t = torch.full((T,), V - 1, device="cuda")
    elif kind == "distinct":
        t = torch.randperm(max(T, V), generator=g, device="cuda")[:T] % V
    elif kind == "none":
        t = torch.full((T,), -1, device="cuda")
    else:                                     # frequency falls as one over the rank
        u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
        t = (torch.exp(u * math.log(V + 1)).floor().long() - 1).clamp(0, V - 1)
        t[torch.rand(T, generator=g, device="cuda") < 0.1] = -7
    return t.to(dtype)


@pytest.mark.parametrize("T,V,D", [(1, 1, 8), (3, 5, 16), (77, 1000, 72), (129, 333, 256),
                                   (1000, 50257, 768), (513, 129, 2048), (65, 40, 4104)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_lookup(T, V, D, dtype):
    g = R.gen(T + V + D)
    table = R.bf16(g, (V, D), 0.02)
    t = ids(g, T, V, "text", dtype)
    scale = math.sqrt(D)
    out = R.strided(torch.zeros((T, D), dtype=torch.bfloat16, device="cuda"), 8, 5.0)
    z.zero_embed(table, t, out, scale=scale)
    # one fp32 product and one rounding: the same bits
    want = table[t.clamp(min=0).long()].float() * torch.tensor(scale, device="cuda")
    want = torch.where((t >= 0)[:, None], want, torch.zeros_like(want)).to(torch.bfloat16)
    assert torch.equal(out, want)
    if T > 1:
        behind = out.as_strided((T - 1, 8), (out.stride(0), 1), out.storage_offset() + D)
        assert bool((behind == 5.0).all())              # the gaps between rows are not written


def test_lookup_ids_past_the_table_set_the_status_word():
    table = torch.ones((10, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full((4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    z.zero_embed(table, torch.tensor([9, -1, 3, -5], device="cuda"), out, dev_status=status)
    assert z.zero_get_device_status(status) == (B.ZERO_OK, 0)
    z.zero_embed(table, torch.tensor([9, 10, 1 << 40, -1], device="cuda"), out, dev_status=status)
    assert z.zero_get_device_status(status) == (B.ZERO_OK, z.ZERO_DEV_BAD_TOKEN)
    assert out.float().sum(1).tolist() == [64.0, 0.0, 0.0, 0.0]


def run_grad(dy, t, grad, scale=1.0, accumulate=False, status=None):
    V, D = grad.shape
    n = z.zero_embed_grad_scratch_bytes(t.numel(), V, D)
    scratch = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    z.zero_embed_grad(dy, t, grad, scratch, scale=scale, accumulate=accumulate, dev_status=status)
    return grad


@pytest.mark.parametrize("kind", ["text", "same", "distinct", "none"])
@pytest.mark.parametrize("T,V,D", [
    (1, 1, 8), (2, 7, 16), (31, 3, 264), (32, 100, 64), (33, 1, 256), (64, 2, 512),
    (65, 50257, 72), (1000, 515, 768), (4096, 50257, 136), (4097, 128256, 256),
    (9000, 11, 40), (40000, 128256, 64), (70001, 300, 16)])
def test_gradient(T, V, D, kind):
    g = R.gen(T * 3 + V + D)
    t = ids(g, T, V, kind, torch.int32 if T % 2 else torch.int64)
    dy = R.strided(R.bf16(g, (T, D)), 16)
    scale = 1.7
    for accumulate in (False, True):
        base = R.bf16(g, (V, D)) if accumulate else None
        got = base.clone() if accumulate else torch.full((V, D), float("nan"),
                                                         dtype=torch.bfloat16, device="cuda")
        run_grad(dy, t, got, scale, accumulate)
        want, mag, n = R.embed_grad(dy, t, V, scale, base)
        R.within(got, want, R.U16 * want.abs() * (1 + R.U16) + (n + 4)[:, None] * R.U32 * mag,
                 f"{kind} accumulate={accumulate}")
        if accumulate:
            untouched = n == 0
            assert torch.equal(got[untouched], base[untouched])
        again = base.clone() if accumulate else torch.empty_like(got)
        assert torch.equal(run_grad(dy, t, again, scale, accumulate), got)      # the same bits


@pytest.mark.parametrize("run", [1, 31, 32, 33, 34, 63, 64, 65, 96, 97, 200])
def test_gradient_of_runs_around_the_chunk(run):
    """Runs of equal ids of one length, at every place in the 32-wide chunks."""
    V, D = 70, 24
    t = torch.arange(V, device="cuda").repeat_interleave(run)
    g = R.gen(run)
    t = t[torch.randperm(t.numel(), generator=g, device="cuda")]
    dy = R.bf16(g, (t.numel(), D))
    got = run_grad(dy, t, torch.empty((V, D), dtype=torch.bfloat16, device="cuda"))
    want, mag, n = R.embed_grad(dy, t, V, 1.0)
    R.within(got, want, R.U16 * want.abs() * (1 + R.U16) + (n + 4)[:, None] * R.U32 * mag)


def test_gradient_counts_exactly():
    """Ones: the sums are the counts, which bf16 holds exactly up to 256."""
    g = R.gen(5)
    t = torch.randint(-2, 300, (20000,), generator=g, device="cuda")
    dy = torch.ones((20000, 8), dtype=torch.bfloat16, device="cuda")
    got = run_grad(dy, t, torch.empty((300, 8), dtype=torch.bfloat16, device="cuda"))
    want = torch.bincount(t[t >= 0], minlength=300)
    assert int(want.max()) <= 256
    assert torch.equal(got[:, 0].long(), want) and torch.equal(got[:, 7].long(), want)


def test_gradient_ignores_what_masked_rows_hold():
    t = torch.tensor([2, -1, 2, 9], device="cuda")
    dy = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    dy[1] = float("nan")
    dy[3] = float("inf")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_grad(dy, t, torch.empty((4, 64), dtype=torch.bfloat16, device="cuda"), status=status)
    assert got.float().sum(1).tolist() == [0, 0, 128, 0]
    assert z.zero_get_device_status(status) == (B.ZERO_OK, z.ZERO_DEV_BAD_TOKEN)


def test_no_tokens():
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    none = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    z.zero_embed(torch.ones((3, 64), dtype=torch.bfloat16, device="cuda"), t, none)
    grad = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    run_grad(none, t, grad, accumulate=True)
    assert bool((grad == 1).all())
    run_grad(none, t, grad)
    assert bool((grad == 0).all())


def test_differences():
    """The gradient of <c, embed(E)> along a direction, by differences in 64 bits."""
    g = R.gen(11)
    T, V, D, scale = 500, 200, 64, 3.0
    t, c = ids(g, T, V, "text"), R.bf16(g, (T, D))
    table, d = R.bf16(g, (V, D)).to(R.F), R.bf16(g, (V, D)).to(R.F)

    def f(e):
        return (c.to(R.F) * (e[t.clamp(min=0)] * (t >= 0)[:, None]) * scale).sum()
    slope = (f(table + 1e-3 * d) - f(table - 1e-3 * d)) / 2e-3
    got = run_grad(c, t, torch.empty((V, D), dtype=torch.bfloat16, device="cuda"), scale).to(R.F)
    assert abs((got * d).sum() - slope) <= R.U16 * got.norm() * d.norm()


def test_rows_past_32_bits():
    """A table of more than 2^31 elements: its last rows, read and written."""
    V, D = 300_000, 8192
    table = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    table[-1], table[-2] = 3.0, 5.0
    t = torch.tensor([V - 1, 0, V - 2, V - 1], device="cuda")
    out = torch.empty((4, D), dtype=torch.bfloat16, device="cuda")
    z.zero_embed(table, t, out)
    assert out[:, 0].tolist() == [3.0, 0.0, 5.0, 3.0] and out[:, -1].tolist() == [3.0, 0.0, 5.0, 3.0]
    table.fill_(7.0)
    run_grad(out, t, table)
    assert table[-1, -1].item() == 6.0 and table[-2, 0].item() == 5.0
    assert float(table[:-2].abs().max()) == 0.0


def test_other_stream_and_graph():
    """Calls on a side stream, and captured once and replayed."""
    g = R.gen(3)
    T, V, D = 5000, 3000, 128
    t, dy = ids(g, T, V, "text"), R.bf16(g, (T, D))
    want = run_grad(dy, t, torch.empty((V, D), dtype=torch.bfloat16, device="cuda"))
    scratch = torch.empty(z.zero_embed_grad_scratch_bytes(T, V, D), dtype=torch.uint8,
                          device="cuda")
    got = torch.empty((V, D), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z.zero_embed_grad(dy, t, got, scratch, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    got.fill_(1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z.zero_embed_grad(dy, t, got, scratch)
    got.fill_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
