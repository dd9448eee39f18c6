"""The forms of the language-model operators' kernels that large sizes use,
against 64-bit forms: several units of work for each pair of thread blocks,
chunks of 32 places and of 8 in the embedding gradient, rows enough for the norm
gradient's ring to go round; and all operators on a side stream and in a graph."""
import pytest
import torch

import zero_optimizer_step_rs_gb300 as z
from tests import lm_ref as R
from tests import test_gpu_lm_embed as E
from tests import test_gpu_lm_norm as N
from tests.test_gpu_lm_xent import backward, problem

pytestmark = pytest.mark.gpu


# --------------------------------------------------------- cross entropy --

@pytest.mark.parametrize("T,V,D,piece", [
    # on 76 pairs (152 SMs), units of dh: 120, so that 32 pairs have one less and take
    # units of the table's gradient first; the same with three pieces, added; 76; 160,
    # two or three a pair; a width that no tile divides
    (5000, 3000, 1024, 0), (5000, 3000, 1024, 1024), (4800, 2000, 1024, 0),
    (10000, 1500, 1024, 512), (6000, 2500, 776, 768),
])
def test_gradients_with_several_units_a_pair(T, V, D, piece):
    h, table, t = problem(T, V, D, seed=9)
    lse = torch.logsumexp(h.to(R.F) @ table.to(R.F).T, 1).float()
    dloss = torch.randn(T, generator=R.gen(T), device="cuda")
    dh, dt = backward(h, table, t, lse, dloss, piece)
    want_h, want_t, bound_h, bound_t = R.xent_grad(h, table, t, lse, dloss)
    R.within(dh, want_h, bound_h, "dh")
    R.within(dt, want_t, bound_t, "dtable")
    R.norm_close(dh, want_h, R.U16, "dh")
    R.norm_close(dt, want_t, R.U16, "dtable")
    again = backward(h, table, t, lse, dloss, piece)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dt)


# ----------------------------------------------------- embedding gradient --

def places(T, D):
    """The chunks' width: 32 where that leaves 2432 warps of 256 columns, else 8."""
    return 32 if -(-T // 32) * -(-D // 256) >= 2432 else 8


def check(t, V, D, seed):
    T = t.numel()
    g = R.gen(seed)
    dy = R.strided(R.bf16(g, (T, D)), 8)
    for accumulate in (False, True):
        base = R.bf16(g, (V, D)) if accumulate else None
        got = base.clone() if accumulate else torch.full((V, D), float("nan"),
                                                         dtype=torch.bfloat16, device="cuda")
        E.run_grad(dy, t, got, 1.5, accumulate)
        want, mag, n = R.embed_grad(dy, t, V, 1.5, base)
        R.within(got, want, R.U16 * want.abs() * (1 + R.U16) + (n + 4)[:, None] * R.U32 * mag,
                 f"accumulate={accumulate}")
        again = base.clone() if accumulate else torch.empty_like(got)
        assert torch.equal(E.run_grad(dy, t, again, 1.5, accumulate), got)


@pytest.mark.parametrize("kind", ["text", "same", "distinct", "none"])
@pytest.mark.parametrize("T,V,D", [(10001, 5003, 2056), (2600, 50000, 8192), (33000, 700, 768)])
def test_embedding_gradient_in_chunks_of_32(T, V, D, kind):
    assert places(T, D) == 32
    check(E.ids(R.gen(T), T, V, kind), V, D, T)


def runs(lengths, seed):
    """Ids of runs of these lengths (in the order of the ids, which the sort restores)."""
    t = torch.arange(len(lengths), device="cuda").repeat_interleave(
        torch.tensor(lengths, device="cuda"))
    return t[torch.randperm(t.numel(), generator=R.gen(seed), device="cuda")]


@pytest.mark.parametrize("width,D,least", [(32, 8192, 2500), (8, 24, 1100)])
@pytest.mark.parametrize("run", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 34, 63, 64, 65, 97, 200])
def test_embedding_gradient_of_runs_of_one_length(run, width, D, least):
    V = max(70, -(-least // run))
    t = runs([run] * V, run)
    assert t.numel() > 1024 and places(t.numel(), D) == width
    check(t, V, D, run)


@pytest.mark.parametrize("width,D,n", [(32, 8192, 200), (8, 24, 200)])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_embedding_gradient_of_runs_of_mixed_lengths(seed, width, D, n):
    g = R.gen(seed)
    lengths = torch.randint(1, 3 * width, (n,), generator=g, device="cuda").tolist()
    lengths[n // 2] = 40 * width
    t = runs(lengths, seed)
    assert t.numel() > 1024 and places(t.numel(), D) == width
    check(t, n, D, seed)


# ------------------------------------------------------------------ norm --

@pytest.mark.parametrize("T,D", [(12001, 256), (12001, 264), (12001, 512), (4001, 768),
                                 (4001, 1024), (4001, 2048), (2001, 4096), (1001, 8192),
                                 (601, 16384)])
def test_norm_gradient_with_more_rows_than_fit_at_once(T, D):
    """At least three rows for each group of threads that takes them in turn."""
    N.test_replay_and_gradient(T, D)


# -------------------------------------------------- side streams, graphs --

def everything(T, V, D):
    """Calls of the lookup, the norm, its replay and its gradient, and their outputs."""
    g = R.gen(T)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    table, w, dy = R.bf16(g, (V, D)), R.bf16(g, (D,)), R.bf16(g, (T, D))
    t = torch.randint(-1, V, (T,), generator=g, device="cuda")
    x, y, again, dx = (torch.zeros((T, D), **bf) for _ in range(4))
    dw = torch.zeros(D, **bf)
    codes = torch.zeros((T, D), dtype=torch.int8, device="cuda")
    scales, rstd = torch.zeros((T, -(-D // R.BLOCK)), device="cuda"), torch.zeros(T, device="cuda")
    scratch = torch.empty(z.zero_norm_grad_scratch_bytes(T, D), dtype=torch.uint8, device="cuda")

    def calls(stream=None):
        z.zero_embed(table, t, x, scale=2.0, stream=stream)
        z.zero_norm(x, w, y, codes, scales, rstd, stream=stream)
        z.zero_norm_replay(codes, scales, rstd, w, again, stream=stream)
        z.zero_norm_grad(dy, codes, scales, rstd, w, dx, dw, scratch, dsum=again, stream=stream)
    return calls, (x, y, codes, scales, rstd, again, dx, dw)


@pytest.mark.parametrize("T,V,D", [(5000, 3000, 768), (40, 100, 4096)])
def test_lookup_and_norm_on_another_stream_and_in_a_graph(T, V, D):
    calls, outputs = everything(T, V, D)
    calls()
    want = [x.clone() for x in outputs]

    def same():
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outputs, want))
        for x in outputs:
            x.zero_()
    same()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    calls(s)                                             # given by hand
    same()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls()                                          # the current one
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(2):
        graph.replay()
        same()
