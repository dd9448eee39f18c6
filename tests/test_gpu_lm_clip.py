"""The norm of many tensors and their clipping on the GPU against 64-bit forms.

A thread adds up to 32 squares of a tile, the tiles without loss, and then come 5 halvings and 8
warps: all positive, so a sum of squares is off by under 64 U32 of itself (DEEP) and its root
by half of that and one rounding."""
import math

import pytest
import torch

import zero_optimizer_step_rs_gb300 as z
from tests import lm_ref as R

pytestmark = pytest.mark.gpu
TYPES = (torch.bfloat16, torch.float16, torch.float32)
DEEP = 64 * R.U32
STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def views(g, sizes, dtype, sigma=1.0, shift=0):
    """Tensors one behind the other in a flat buffer, `shift` elements from its start."""
    flat = (torch.randn(sum(sizes) + shift, generator=g, device="cuda") * sigma).to(dtype)
    return list(flat[shift:].split(sizes))


def norms_of(tensors, status=None):
    norm, norms = torch.full((1,), -1.0, device="cuda"), torch.full((len(tensors),), -1.0, device="cuda")
    scratch = torch.full((z.zero_grad_norm_scratch_bytes(len(tensors)),), 255, dtype=torch.uint8,
                         device="cuda")
    z.zero_grad_norm(tensors, norm, scratch, norms=norms, dev_status=status)
    alone = torch.empty(1, device="cuda")
    z.zero_grad_norm(tensors, alone, scratch)
    assert torch.equal(alone.view(torch.int32), norm.view(torch.int32))
    return norm, norms


def want_norms(tensors):
    each = torch.stack([t.to(R.F).norm() for t in tensors])
    return each.norm().view(1), each


SETS = {
    "one": [1], "few": [7, 1, 8, 9], "tile": [8192], "around": [8191, 8192, 8193, 16385],
    "odd": [100_003, 1, 77, 0, 8_000, 0, 0, 40_961, 5, 0], "empty": [0, 0],
    "many": [3] * 200 + [1000] * 300 + [0] * 100 + [8193] * 200,
    "some": [(k * 613) % 2999 for k in range(150)],
    "more than one launch": [k % 37 for k in range(2100)],
    "big": [30_000_001, 11, 5_000_000],
}


@pytest.mark.parametrize("name", SETS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift", [0, 1, 5])
def test_norm(name, dtype, shift):
    t = views(R.gen(len(name) + shift), SETS[name], dtype, shift=shift)
    norm, norms = norms_of(t)
    want, each = want_norms(t)
    R.within(norm, want, want * DEEP)
    R.within(norms, each, each * DEEP)
    again = norms_of(t)
    assert torch.equal(again[0], norm) and torch.equal(again[1], norms)


def test_tensors_of_several_types_and_orders():
    g = R.gen(3)
    t = [R.bf16(g, (33, 65)).t(), (torch.randn(5, 7, 9, generator=g, device="cuda")).permute(2, 0, 1),
         torch.randn(40, generator=g, device="cuda").half(), R.bf16(g, (1,))[0]]
    norm, norms = norms_of(tuple(t))
    want, each = want_norms(t)
    R.within(norm, want, want * DEEP)
    R.within(norms, each, each * DEEP)
    before = [x.clone() for x in t]
    z.zero_grad_clip(t, norm, 0.25)
    coef = coefficient(norm, 0.25)
    for x, b in zip(t, before):
        assert torch.equal(x, (b.float() * coef).to(b.dtype)) and x.stride() == b.stride()


@pytest.mark.parametrize("dtype,sigma", [(torch.float32, 1e30), (torch.float32, 1e-30),
                                         (torch.float32, 1e-42), (torch.bfloat16, 1e25),
                                         (torch.bfloat16, 1e-25), (torch.float16, 1e-6),
                                         (torch.float16, 3e4 / 5)])
def test_values_whose_squares_overflow_or_vanish(dtype, sigma):
    t = views(R.gen(8), [70_000, 3, 0, 9000], dtype, sigma, shift=1)
    t += [torch.zeros(20_000, dtype=dtype, device="cuda"), torch.ones(5, dtype=dtype, device="cuda")]
    norm, norms = norms_of(t)
    want, each = want_norms(t)
    # (the norm of subnormal values is itself rounded to a subnormal: half of 2^-149)
    R.within(norm, want, want * DEEP + 2.0 ** -150)
    R.within(norms, each, each * DEEP + 2.0 ** -150)
    assert norms[4].item() == 0.0


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", TYPES)
def test_values_that_are_not_finite(bad, dtype):
    t = views(R.gen(5), [9000, 20_001, 30], dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    clean = norms_of(t, status)
    assert status.item() == 0
    t[1][20_000] = bad
    norm, norms = norms_of(t, status)
    assert status.item() == z.ZERO_DEV_NONFINITE
    assert z.zero_get_device_status(status)[0] == -8     # ZERO_ERR_NONFINITE
    assert torch.equal(norms[::2], clean[1][::2])
    want = abs(bad)
    assert all(math.isnan(v) if math.isnan(want) else v == want for v in (norm.item(), norms[1].item()))
    # an infinite norm multiplies by 0, one that is NaN clips nothing
    before = [x.clone() for x in t]
    z.zero_grad_clip(t, norm, 1.0)
    for x, b in zip(t, before):
        want = b if math.isnan(bad) else (b.float() * 0.0).to(dtype)
        assert torch.equal(x.float().nan_to_num(7.0), want.float().nan_to_num(7.0))


def test_both_kinds_of_values_that_are_not_finite():
    t = [torch.tensor([1.0, float("inf"), float("nan")], device="cuda")]
    assert math.isnan(norms_of(t)[0].item())


def test_a_norm_past_fp32():
    t = [torch.full((9,), 3e38, device="cuda")]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    norm, _ = norms_of(t, status)
    assert math.isinf(norm.item()) and status.item() == z.ZERO_DEV_NONFINITE


def test_no_tensors():
    norm = torch.ones(1, device="cuda")
    z.zero_grad_norm([], norm, torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert norm.item() == 0.0
    z.zero_grad_clip([], norm, 1.0)


def coefficient(norm, most):
    """max_norm is taken in fp32, the quotient in 64 bits and rounded to fp32."""
    coef = torch.tensor(most, dtype=torch.float32).double() / (norm.cpu().double() + 1e-6)
    return coef.float().item() if coef < 1 else 1.0


PAIRS = [(d, d) for d in TYPES] + [(torch.float16, torch.bfloat16), (torch.float32, torch.bfloat16)]


@pytest.mark.parametrize("name", ["one", "around", "odd", "some", "many", "more than one launch"])
@pytest.mark.parametrize("dtype,to", PAIRS)
@pytest.mark.parametrize("shifts", [(0, 0), (3, 3), (1, 2), (0, 7)])
def test_clip(name, dtype, to, shifts):
    sizes = SETS[name]
    g = R.gen(len(name))
    t = views(g, sizes, dtype, shift=shifts[0])
    norm, _ = norms_of(t)
    for most in (0.37 * max(norm.item(), 1e-3), 2 * norm.item() + 1):
        coef = coefficient(norm, most)
        total = sum(sizes) + shifts[1]
        flat = torch.full((total + 9,), 5.0, dtype=to, device="cuda")
        outs = list(flat[shifts[1]:total].split(sizes))
        z.zero_grad_clip(t, norm, most, outs=outs)
        for x, o in zip(t, outs):
            # one fp32 product, one rounding: the same bits
            assert torch.equal(o, (x.float() * coef).to(to))
        assert bool((flat[:shifts[1]] == 5).all()) and bool((flat[total:] == 5).all())
        if dtype == to:
            own = [x.clone() for x in t]
            z.zero_grad_clip(own, norm, most)
            assert all(torch.equal(x, o) for x, o in zip(own, outs))


def test_clip_big():
    t = views(R.gen(1), SETS["big"], torch.float32, 1e-3, shift=1)
    norm, _ = norms_of(t)
    want = want_norms(t)[0]
    R.within(norm, want, want * DEEP)
    coef = coefficient(norm, 0.5)
    outs = [torch.empty_like(x, dtype=torch.bfloat16) for x in t]
    z.zero_grad_clip(t, norm, 0.5, outs=outs)
    assert all(torch.equal(o, (x * coef).to(torch.bfloat16)) for x, o in zip(t, outs))
    z.zero_grad_clip(t, norm, 0.5)
    # each element was rounded once more
    after = want_norms(t)[0].item()
    assert abs(after - 0.5) <= 0.5 * 2 * (DEEP + 1e-6)


def test_more_elements_than_32_bits_count():
    n = (1 << 31) + 8_195
    flat = torch.ones(n + 3, dtype=torch.bfloat16, device="cuda")
    flat[-1] = 3.0
    t = [flat[:3], flat[3:]]
    norm, norms = norms_of(t)
    want = (n + 3 + 8) ** 0.5
    assert abs(norm.item() - want) <= DEEP * want and norms[0].item() == pytest.approx(3 ** 0.5)
    z.zero_grad_clip(t, norm, 0.5 * norm.item())
    assert flat[0].item() == 0.5 and flat[-2].item() == 0.5 and flat[-1].item() == 1.5
    assert flat[1 << 31].item() == 0.5
    again = norms_of(t)[0].item()
    assert abs(again - 0.5 * want) <= DEEP * want


def test_the_same_tensor_twice():
    x = torch.full((1000,), 3.0, device="cuda")
    norm, norms = norms_of([x, x])
    assert norm.item() == pytest.approx((2000 * 9) ** 0.5, rel=1e-6)
    assert norms[0].item() == norms[1].item()


def test_two_calls_at_once():
    """On two streams, each with its own scratch and outputs."""
    sets = [views(R.gen(k), [200_003, 77, 1_000_001], torch.float32) for k in range(2)]
    want = [norms_of(t) for t in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    rooms = [torch.empty(z.zero_grad_norm_scratch_bytes(3), dtype=torch.uint8, device="cuda") for _ in sets]
    got = [(torch.zeros(1, device="cuda"), torch.zeros(3, device="cuda")) for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for t, s, room, (norm, norms) in zip(sets, streams, rooms, got):
            z.zero_grad_norm(t, norm, room, norms=norms, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_overlapping_outputs_are_refused():
    t = views(R.gen(1), [10, 20], torch.bfloat16)
    norm = torch.ones(1, device="cuda")
    for tensors, outs in (([t[0], t[0]], None), (t, [t[0], torch.empty_like(t[1])]),
                          (t, [torch.empty_like(t[0]), t[0].repeat(2)[:0]])):
        with pytest.raises((z.ZeroError, ValueError)):
            z.zero_grad_clip(tensors, norm, 1.0, outs=outs)


@pytest.mark.parametrize("count", [5, 150])
def test_another_stream_and_a_graph(count):
    t = views(R.gen(2), [1000 + k for k in range(count)], torch.float32)
    outs = [torch.empty_like(x) for x in t]
    norm = torch.zeros(1, device="cuda")
    scratch = torch.empty(z.zero_grad_norm_scratch_bytes(count), dtype=torch.uint8, device="cuda")

    def calls(stream=None):
        z.zero_grad_norm(t, norm, scratch, stream=stream)
        z.zero_grad_clip(t, norm, 1.0, outs=outs, stream=stream)
    calls()
    want = [x.clone() for x in outs]

    def same():
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        for x in (norm, *outs):
            x.zero_()
    same()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    calls(s)
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(2):
        graph.replay()
        same()
    # other values behind the same addresses
    for x, w in zip(t, want):
        x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    # twice the values with twice the norm: the same but for the 1e-6 and roundings
    for a, b in zip(outs, want):
        assert bool(((a - b).abs() <= b.abs() * (1e-6 + 8 * R.U32)).all())
