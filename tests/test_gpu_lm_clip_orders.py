"""What the gradient norm's order of additions depends on: the sizes, the types and the
addresses modulo 16 bytes, nothing else."""
import pytest
import torch

import zero_optimizer_step_rs_gb300 as z
from tests import lm_ref as R

pytestmark = pytest.mark.gpu
SIZES = [100_003, 1, 77, 0, 8_000, 40_961, 5, 1_000_007]
DEEP = 64 * R.U32                     # a sum of positive terms: under 64 roundings deep


def norms_at(values, dtype, shift):
    """The norms of tensors that lie `shift` elements behind a 16-byte boundary, one behind the
    other, in memory of their own."""
    n = sum(SIZES)
    flat = torch.empty(n + shift, dtype=dtype, device="cuda")[shift:]
    flat.copy_(values)
    t = list(flat.split(SIZES))
    norm, norms = torch.zeros(1, device="cuda"), torch.zeros(len(t), device="cuda")
    room = torch.full((z.zero_grad_norm_scratch_bytes(len(t)),), 255, dtype=torch.uint8, device="cuda")
    z.zero_grad_norm(t, norm, room, norms=norms)
    return norm, norms, flat


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_the_same_bits_at_the_same_remainder(dtype):
    values = torch.randn(sum(SIZES), generator=R.gen(4), device="cuda").to(dtype)
    per = 16 // values.element_size()
    want = torch.stack([t.double().norm() for t in values.split(SIZES)])
    for shift in range(per):
        first = norms_at(values, dtype, shift)
        for more in (per, 5 * per, 128 * per + 3 * per):
            again = norms_at(values, dtype, shift + more)
            assert again[2].data_ptr() != first[2].data_ptr()
            assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
        R.within(first[1], want, want * DEEP)
        R.within(first[0], want.norm().view(1), want.norm().view(1) * DEEP)
