"""The layer norm's dweight and dbias where every row counts: small whole numbers, whose products and
sums (below 2^24) fp32 holds exactly in any order, so that the result is the exact sum rounded to
bf16 once.  A row that is lost or counted twice changes columns whose sum bf16 holds exactly."""
import pytest
import torch

import zero_optimizer_step_rs_gb300 as z
from tests import lm_ref as R

pytestmark = pytest.mark.gpu


def whole(g, shape, most, density=1.0):
    x = torch.randint(-most, most + 1, shape, generator=g, device="cuda").float()
    return (x * (torch.rand(shape, generator=g, device="cuda") < density)).to(torch.bfloat16)


# every form, with one row, fewer rows than fit at once, a few more and many more
WIDTHS = [8, 64, 72, 128, 136, 192, 200, 256, 264, 384, 392, 512, 520, 768, 776, 1024, 1032, 1304,
          2048, 2056, 2800, 4096, 4104, 5608, 8192, 8200, 12008, 16384]
ROWS = [1, 2, 151, 153, 1217, 5003, 20_001]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("T", ROWS)
@pytest.mark.parametrize("extra", [0, 8])
def test_every_row_is_in_the_sums(T, D, extra):
    if T * D > 1 << 27:
        T = (1 << 27) // D | 1
    g = R.gen(T + D)
    dy, x = whole(g, (T, D), 1, 0.25), whole(g, (T, D), 2)
    if extra:
        dy, x = R.strided(dy, extra), R.strided(x, extra)
    mean, rstd = torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")
    dx = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
    dw, db = (torch.empty(D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    scratch = torch.full((z.zero_layer_norm_grad_scratch_bytes(T, D),), 255, dtype=torch.uint8,
                         device="cuda")
    z.zero_layer_norm_grad(dy, x, mean, rstd, None, dx, dw, db, scratch)
    e, h = dy.double(), x.double()
    for got, terms in ((dw, e * h), (db, e)):
        total = terms.sum(0)
        assert float(terms.abs().sum(0).max()) < 2 ** 24
        assert torch.equal(got, total.float().to(torch.bfloat16))
        # and what the check is worth: without one row it would fail
        for t in {0, T // 3, T - 1}:
            if terms[t].any() and D >= 64:
                less = (total - terms[t]).float().to(torch.bfloat16)
                assert not torch.equal(got, less)


@pytest.mark.parametrize("T,D", [(3000, 2040), (5000, 1080), (3000, 4024), (3000, 2048), (40_000, 120)])
def test_the_sums_do_not_depend_on_the_rows_padding(T, D):
    """The same bits whatever the strides are, multiples of a cache line (64 elements) or not.  Each
    row comes back with the other sign, so that all that is left of the sums is what their order
    rounds away."""
    g = R.gen(D)
    dy = R.bf16(g, (T // 2, D)) * torch.randn((T // 2, 1), generator=g, device="cuda").mul(3).exp().to(torch.bfloat16)
    x, w = R.bf16(g, (T // 2, D)), R.bf16(g, (D,))
    back = torch.randperm(T // 2, generator=g, device="cuda")
    dy, x = torch.cat([dy, -dy[back]]), torch.cat([x, x[back]])
    mean, rstd = torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")
    want = None
    for extra in (0, 8, 64 - D % 64, 128 - D % 64 + 24):
        rows = [R.strided(t, extra) if extra else t for t in (dy, x, torch.zeros_like(x))]
        dw, db = (torch.empty(D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        scratch = torch.empty(z.zero_layer_norm_grad_scratch_bytes(T, D), dtype=torch.uint8, device="cuda")
        z.zero_layer_norm_grad(rows[0], rows[1], mean, rstd, w, rows[2], dw, db, scratch)
        got = (rows[2].clone(), dw, db)
        want = want or got
        assert dw.any()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), extra
