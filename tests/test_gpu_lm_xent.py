"""The vocabulary cross entropy and its gradients on the GPU against 64-bit forms."""
import pytest
import torch

import zero_optimizer_step_rs_gb300 as z
from tests import lm_ref as R
from zero_optimizer_step_rs_gb300 import binding as B

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 8), (1, 257, 64), (2, 2, 16), (17, 5003, 72), (31, 255, 136), (33, 256, 264),
         (127, 1000, 64), (128, 511, 512), (129, 513, 200), (255, 2000, 128), (256, 256, 256),
         (257, 769, 320), (300, 1001, 776), (600, 20001, 48)]


def problem(T, V, D, seed=0, dtype=torch.int64, sigma=1.0):
    g = R.gen(seed + T + V + D)
    h, table = R.strided(R.bf16(g, (T, D), sigma), 16), R.bf16(g, (V, D), 0.3)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    t[torch.rand(T, generator=g, device="cuda") < 0.15] = -100
    return h, table, t.to(dtype)


def forward(h, table, t, flags=0, status=None):
    T, (V, D) = t.numel(), table.shape
    loss, lse = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    scratch = torch.full((z.zero_xent_scratch_bytes(T, V, D),), 255, dtype=torch.uint8,
                         device="cuda")
    z.zero_xent(h, table, t, loss, lse, scratch, flags=flags, dev_status=status)
    return loss, lse


def backward(h, table, t, lse, dloss, piece=0, flags=0, status=None, extra=8):
    T, (V, D) = t.numel(), table.shape
    n = z.zero_xent_grad_scratch_bytes(T, V, D, piece)
    scratch = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    dh = R.strided(torch.zeros((T, D), dtype=torch.bfloat16, device="cuda"), extra)
    dt = torch.full((V, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    z.zero_xent_grad(h, table, t, lse, dloss, dh, dt, scratch, piece=piece, flags=flags,
                     dev_status=status)
    return dh, dt


@pytest.mark.parametrize("T,V,D", SIZES)
def test_loss(T, V, D):
    h, table, t = problem(T, V, D, dtype=torch.int32 if T % 2 else torch.int64)
    loss, lse = forward(h, table, t)
    want, want_lse, bound = R.xent(h, table, t)
    R.within(lse, want_lse, bound, "lse")
    R.within(loss, want, bound, "loss")
    assert not loss[t < 0].any()
    again = forward(h, table, t)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)


@pytest.mark.parametrize("T,V,D", SIZES)
@pytest.mark.parametrize("piece", [0, 256, 768])
def test_gradients(T, V, D, piece):
    h, table, t = problem(T, V, D, seed=1)
    lse = torch.logsumexp(h.to(R.F) @ table.to(R.F).T, 1).float()
    dloss = torch.randn(T, generator=R.gen(2), device="cuda")
    dh, dt = backward(h, table, t, lse, dloss, piece)
    want_h, want_t, bound_h, bound_t = R.xent_grad(h, table, t, lse, dloss)
    R.within(dh, want_h, bound_h, "dh")
    R.within(dt, want_t, bound_t, "dtable")
    if V > 8:              # two independent roundings to bf16, each under U16 / sqrt(3) in norm
        R.norm_close(dh, want_h, R.U16, "dh")
        R.norm_close(dt, want_t, R.U16, "dtable")
    again = backward(h, table, t, lse, dloss, piece)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dt)


def test_gradients_by_differences():
    """The summed loss along directions of h and of the table, by differences in 64 bits."""
    T, V, D = 90, 700, 96
    h, table, t = problem(T, V, D, seed=3)
    g = R.gen(4)
    dloss = torch.rand(T, generator=g, device="cuda")
    _, lse = forward(h, table, t)
    dh, dt = backward(h, table, t, lse, dloss)
    h64, e64 = h.to(R.F), table.to(R.F)

    def f(a, b):
        l = a @ b.T
        per = torch.logsumexp(l, 1) - l.gather(1, t.clamp(min=0)[:, None])[:, 0]
        return (per * dloss.to(R.F) * (t >= 0)).sum()
    e = 1e-4
    d = R.bf16(g, (T, D)).to(R.F)
    slope = (f(h64 + e * d, e64) - f(h64 - e * d, e64)) / (2 * e)
    assert abs((dh.to(R.F) * d).sum() - slope) <= R.U16 * dh.to(R.F).norm() * d.norm()
    d = R.bf16(g, (V, D)).to(R.F)
    slope = (f(h64, e64 + e * d) - f(h64, e64 - e * d)) / (2 * e)
    assert abs((dt.to(R.F) * d).sum() - slope) <= R.U16 * dt.to(R.F).norm() * d.norm()


def test_large_logits():
    """Logits in the hundreds: nothing overflows, and the bound grows with them."""
    h, table, t = problem(70, 900, 64, seed=5, sigma=60.0)
    loss, lse = forward(h, table, t)
    want, want_lse, bound = R.xent(h, table, t)
    assert float(want_lse.max()) > 200
    R.within(lse, want_lse, bound, "lse")
    R.within(loss, want, bound, "loss")


def test_ignored_rows_leave_no_trace():
    """NaN and Inf in the rows (and in dloss) of ignored tokens reach nothing else."""
    T, V, D = 300, 1500, 128
    h, table, t = problem(T, V, D, seed=6)
    dloss = torch.rand(T, generator=R.gen(1), device="cuda")
    clean = h.clone()
    clean[t < 0] = 0
    loss, lse = forward(clean, table, t)
    dh, dt = backward(clean, table, t, lse, dloss)
    gone = (t < 0).nonzero()[:, 0]
    h[gone[0]] = float("nan")
    h[gone[1]] = float("inf")
    h[gone[2], 5] = float("-inf")
    loss2, lse2 = forward(h, table, t)
    dloss[gone] = float("nan")
    dh2, dt2 = backward(h, table, t, lse2, dloss)
    assert torch.equal(loss2, loss)
    assert torch.equal(lse2[t >= 0], lse[t >= 0])
    assert torch.equal(dt2, dt) and torch.equal(dh2, dh)
    assert not dh2[t < 0].any()


@pytest.mark.parametrize("T", [1, 300])
def test_nothing_but_ignored_tokens(T):
    h, table, t = problem(T, 400, 64)
    t.fill_(-1)
    loss, lse = forward(h, table, t)
    assert not loss.any()
    dh, dt = backward(h, table, t, lse, torch.ones(T, device="cuda"))
    assert not dh.any() and not dt.any()


def test_targets_past_the_table():
    h, table, t = problem(40, 300, 64)
    t[3], t[9] = 300, 1 << 35
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, lse = forward(h, table, t, status=status)
    assert z.zero_get_device_status(status) == (B.ZERO_OK, z.ZERO_DEV_BAD_TOKEN)
    status.zero_()
    dh, _ = backward(h, table, t, lse, torch.ones(40, device="cuda"), status=status)
    assert z.zero_get_device_status(status) == (B.ZERO_OK, z.ZERO_DEV_BAD_TOKEN)
    assert loss[3].item() == 0 and loss[9].item() == 0 and not dh[[3, 9]].any()


def test_a_nan_row_stays_in_its_row_of_the_loss():
    h, table, t = problem(64, 600, 64)
    t.clamp_(min=0)
    loss, lse = forward(h, table, t)
    h[7, 3] = float("nan")
    loss2, lse2 = forward(h, table, t)
    assert torch.isnan(loss2).nonzero()[:, 0].tolist() == [7]
    keep = torch.arange(64, device="cuda") != 7
    assert torch.equal(loss2[keep], loss[keep]) and torch.equal(lse2[keep], lse[keep])


def test_no_tokens():
    table = torch.ones((300, 64), dtype=torch.bfloat16, device="cuda")
    h = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = forward(h, table, t)
    dh, dt = backward(h, table, t, lse, loss)
    assert not dt.any()


def test_rows_past_32_bits():
    """A table of more than 2^31 elements."""
    T, V, D = 4, 270_000, 8192
    g = R.gen(8)
    h = R.bf16(g, (T, D), 0.1)
    table = torch.empty((V, D), dtype=torch.bfloat16, device="cuda")
    for part in table.split(20_000):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * 0.1)
    t = torch.tensor([V - 1, 0, V - 2, -1], device="cuda")
    loss, lse = forward(h, table, t)
    l = torch.cat([h.to(R.F) @ part.to(R.F).T for part in table.split(20_000)], 1)
    want_lse = torch.logsumexp(l, 1)
    off = D * 2 * R.U32 * float((h.abs().float() @ table[-100:].abs().float().T).amax()) * 2 + 1e-5
    R.within(lse, want_lse, off * torch.ones(T, device="cuda"), "lse")
    R.within(loss[:3], (want_lse - l[torch.arange(T), t.clamp(min=0)])[:3],
             2 * off * torch.ones(3, device="cuda"), "loss")
    dh, dt = backward(h, table, t, lse, torch.ones(T, device="cuda"))
    p = torch.exp(l - lse.to(R.F)[:, None])
    p[torch.arange(3), t[:3]] -= 1
    p[3] = 0
    R.norm_close(dt[-1000:], p[:, -1000:].T @ h.to(R.F), R.U16, "dtable")
    R.norm_close(dh, sum(p[:, i:i + 20_000] @ table[i:i + 20_000].to(R.F)
                         for i in range(0, V, 20_000)), R.U16, "dh")


def test_expired_waits_are_reported():
    """Every bounded wait gives up at once: the calls end, the status word says so."""
    h, table, t = problem(300, 1000, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, lse = forward(h, table, t, flags=z.ZERO_FLAG_DEBUG_EXPIRE_WAITS, status=status)
    code, word = z.zero_get_device_status(status)
    assert code == B.ZERO_ERR_DEVICE_TIMEOUT and word == z.ZERO_DEV_TIMEOUT
    status.zero_()
    _, lse = forward(h, table, t, status=status)
    backward(h, table, t, lse, torch.ones(300, device="cuda"),
             flags=z.ZERO_FLAG_DEBUG_EXPIRE_WAITS, status=status)
    code, word = z.zero_get_device_status(status)
    assert code == B.ZERO_ERR_DEVICE_TIMEOUT and word == z.ZERO_DEV_TIMEOUT
    # the next calls are as ever
    status.zero_()
    loss, lse = forward(h, table, t, status=status)
    want, want_lse, bound = R.xent(h, table, t)
    R.within(loss, want, bound)
    assert z.zero_get_device_status(status) == (B.ZERO_OK, 0)


def test_other_stream_and_graph():
    h, table, t = problem(200, 3000, 128)
    dloss = torch.ones(200, device="cuda")
    loss, lse = forward(h, table, t)
    dh, dt = backward(h, table, t, lse, dloss)
    s1 = torch.empty(z.zero_xent_scratch_bytes(200, 3000, 128), dtype=torch.uint8, device="cuda")
    s2 = torch.empty(z.zero_xent_grad_scratch_bytes(200, 3000, 128), dtype=torch.uint8,
                     device="cuda")
    l2, e2 = torch.zeros_like(loss), torch.zeros_like(lse)
    h2, t2 = torch.zeros((200, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros_like(dt)

    def both(stream=None):
        z.zero_xent(h, table, t, l2, e2, s1, stream=stream)
        z.zero_xent_grad(h, table, t, e2, dloss, h2, t2, s2, stream=stream)

    def same():
        torch.cuda.synchronize()
        assert torch.equal(l2, loss) and torch.equal(e2, lse)
        assert torch.equal(h2, dh) and torch.equal(t2, dt)
        for x in (l2, e2, h2, t2):
            x.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    both(s)
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    graph.replay()
    same()
