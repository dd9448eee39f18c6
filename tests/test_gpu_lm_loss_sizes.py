"""The losses of packed sequences where their numbers are far apart: sequences by the million, most
of them empty, as a program with buffers of a fixed size has them."""
import math
import time

import pytest
import torch

import zero_optimizer_step_rs_gb300 as z
from tests.test_gpu_lm_loss import fresh, scratch_of

pytestmark = pytest.mark.gpu


def seconds(call):
    """Of the second call, from a GPU that has nothing to do until it has nothing to do again."""
    call()
    torch.cuda.synchronize()
    start = time.perf_counter()
    call()
    torch.cuda.synchronize()
    return time.perf_counter() - start


def test_many_sequences_without_tokens():
    """Their results in parallel: 2^22 of them in turn, 32 at a time, would wait for 2^17 loads of 0.3
    us each (40 ms); side by side they are 2^22 warps with two loads, under 1 ms."""
    S = 1 << 22
    e, ids = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    offsets = torch.zeros(S + 1, dtype=torch.int64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, kl, adv = fresh(S), fresh(S), torch.ones(S, device="cuda")
    clipped, counts = fresh(S, torch.int32), fresh(S, torch.int32)
    room = scratch_of(z.zero_policy_scratch_bytes, 0, S)
    assert seconds(lambda: z.zero_policy(e, e, e, adv, ids, offsets, loss, kl, clipped, counts, room,
                                         kl_coef=0.1, dev_status=status)) < 0.01
    assert status.item() == 0
    assert not (loss.any() or kl.any() or clipped.any() or counts.any())
    P = S // 2
    loss, slope, ratios, counts = fresh(P), fresh(P), fresh(S), fresh(S, torch.int32)
    room = scratch_of(z.zero_preference_scratch_bytes, 0, P)
    assert seconds(lambda: z.zero_preference(e, e, ids, offsets, loss, slope, ratios, counts, room,
                                             beta=0.5, dev_status=status)) < 0.01
    assert status.item() == 0 and not (ratios.any() or counts.any())
    assert bool((loss == loss[0]).all()) and abs(loss[0].item() - math.log(2)) < 1e-6
    assert bool((slope == -0.25).all())
    # one sequence that the tokens do not reach to
    offsets[-1] = 1
    z.zero_preference(e, e, ids, offsets, loss, slope, ratios, counts, room, dev_status=status)
    assert status.item() == z.ZERO_DEV_BAD_OFFSETS
