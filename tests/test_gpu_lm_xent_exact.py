"""How exact the cross entropy and its gradients are, where the bounds of
test_gpu_lm_xent.py are too wide to tell."""
import pytest
import torch

from tests import lm_ref as R
from tests.test_gpu_lm_xent import backward

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
