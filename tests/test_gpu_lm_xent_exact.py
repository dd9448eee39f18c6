"""How exact the cross entropy and its gradients are, where the bounds of
test_gpu_lm_xent.py are too wide to tell."""
import pytest
import torch

from tests import lm_ref as R
from tests.test_gpu_lm_xent import backward, forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("weights", ["uniform", "random"])
@pytest.mark.parametrize("T,V,D", [(1000, 5003, 256), (64, 9001, 1024)])
def test_gradients_lose_no_more_than_their_own_rounding(T, V, D, weights):
    """Small logits over a large vocabulary: a row of dh is the target's entry,
    near -1 times the token's weight, times a row of the table.  Rounding the
    64-bit result is then the only error that dh may have (a tenth more for P's
    other entries, whose rounding is about 1 / sqrt(V) of it); the table's
    gradient has the rounding of P too, another one of that size."""
    g = R.gen(T + V)
    h, table = R.bf16(g, (T, D)), R.bf16(g, (V, D), 0.02)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    t[::9] = -1
    dloss = torch.rand(T, generator=g, device="cuda") + 0.1
    if weights == "uniform":
        dloss = torch.full((T,), 1.0 / T, device="cuda")
    lse = torch.logsumexp(h.to(R.F) @ table.to(R.F).T, 1).float()
    dh, dt = backward(h, table, t, lse, dloss)
    want_h, want_t, _, _ = R.xent_grad(h, table, t, lse, dloss)

    def rounding(x):
        return ((x.to(torch.bfloat16).to(R.F) - x).norm() / x.norm()).item()
    R.norm_close(dh, want_h, 1.1 * rounding(want_h), "dh")
    R.norm_close(dt, want_t, 1.1 * 2 ** 0.5 * rounding(want_t), "dtable")


@pytest.mark.parametrize("T,V", [(64, 200), (300, 5003)])
def test_a_small_loss_at_large_logits(T, V):
    """Whole numbers, so that every logit is exact, of magnitude 300 and more; the
    target is the largest logit or one of the next.  The loss then has the errors
    of the exponentials (2^-22 each), of their sums and joins and of one
    logarithm: below 2^-19 together, and two roundings of itself; none of the
    logits' own magnitude."""
    g = R.gen(V)
    h = torch.randint(-8, 9, (T, 64), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randint(-8, 9, (V, 64), generator=g, device="cuda").to(torch.bfloat16)
    logits = h.to(R.F) @ table.to(R.F).T
    top = logits.topk(3, 1)
    assert float(top.values[:, 0].median()) > 300
    t = top.indices.gather(1, (torch.arange(T, device="cuda") % 3)[:, None])[:, 0]
    loss, lse = forward(h, table, t)
    want_lse = torch.logsumexp(logits, 1)
    want = want_lse - logits.gather(1, t[:, None])[:, 0]
    assert int((want < 1).sum()) > T // 4
    R.within(loss, want, 2.0 ** -19 + 2 * R.U32 * want, "loss")
    R.within(lse, want_lse, 2.0 ** -19 + 2 * R.U32 * want_lse.abs(), "lse")


@pytest.mark.parametrize("T", [17, 300])
def test_ignored_rows_have_no_gradient_beside_a_table_that_is_not_finite(T):
    g = R.gen(T)
    h, table = R.bf16(g, (T, 64)), R.bf16(g, (1000, 64), 0.1)
    t = torch.randint(0, 1000, (T,), generator=g, device="cuda")
    t[::4] = -1
    t[1] = 1000                                          # past the table: no token either
    table[7, 3], table[500] = float("inf"), float("nan")
    _, lse = forward(h, table, t)
    dh, _ = backward(h, table, t, lse, torch.ones(T, device="cuda"))
    gone = (t < 0) | (t >= 1000)
    assert not dh[gone].any()                            # a NaN would count as true
    assert bool(torch.isnan(dh[~gone]).all())
