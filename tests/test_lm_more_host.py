"""Argument checks of the layer norm, the losses of packed sequences and the
gradient norm, which happen on the host before any CUDA call; their scratch
sizes; and tensors on different GPUs.  Needs no GPU."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import zero_optimizer_step_rs_gb300 as z
from tests.test_lm_host import ALIGN, CUDA, GAP, INVALID, NULL, OVERLAP, SIZE, Call, at, pointers
from zero_optimizer_step_rs_gb300 import binding as B

BIG = 1 << 38


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_rs_gb300 import build
    build.build()


LN = Call("zero_layer_norm", dict(
    x=at(0), x_ld=64, res=at(1), res_ld=64, weight=at(2), bias=at(3), T=50, D=64, eps=1e-5,
    y=at(4), y_ld=64, sum=at(5), sum_ld=64, mean=at(6), rstd=at(7), stream=None))
LN_GRAD = Call("zero_layer_norm_grad", dict(
    dy=at(0), dy_ld=64, dsum=at(1), dsum_ld=64, x=at(2), x_ld=64, mean=at(3), rstd=at(4),
    weight=at(5), T=50, D=64, dx=at(6), dx_ld=64, dweight=at(7), dbias=at(8), scratch=at(9),
    size=BIG, stream=None))
PREF = Call("zero_preference", dict(
    nll=at(0), ref_nll=at(1), targets=at(2), width=8, T=50, offsets=at(3), offset_width=8, P=3,
    kind=0, beta=0.1, smoothing=0.1, margin=0.5, average=1, loss=at(4), slope=at(5), ratios=at(6),
    counts=at(7), scratch=at(8), size=BIG, status=None, stream=None))
PREF_GRAD = Call("zero_preference_grad", dict(
    targets=at(0), width=4, T=50, offsets=at(1), offset_width=4, P=3, average=0, slope=at(2),
    counts=at(3), dloss=at(4), dnll=at(5), stream=None))
POLICY = Call("zero_policy", dict(
    nll=at(0), old_nll=at(1), ref_nll=at(2), advantages=at(3), per_token=0, targets=at(4), width=8,
    T=50, offsets=at(5), offset_width=4, S=3, clip_low=0.2, clip_high=0.2, kl_coef=0.1, average=1,
    loss=at(6), kl=at(7), clipped=at(8), counts=at(9), scratch=at(10), size=BIG, status=None,
    stream=None))
POLICY_GRAD = Call("zero_policy_grad", dict(
    nll=at(0), old_nll=at(1), ref_nll=at(2), advantages=at(3), per_token=1, targets=at(4), width=8,
    T=50, offsets=at(5), offset_width=8, S=3, clip_low=0.2, clip_high=0.2, kl_coef=0.1, average=0,
    counts=at(6), dloss=at(7), dnll=at(8), stream=None))
NORMS, LOSSES = (LN, LN_GRAD), (PREF, PREF_GRAD, POLICY, POLICY_GRAD)
ALL = NORMS + LOSSES
OPTIONAL = {"res", "sum", "dsum", "weight", "bias", "dweight", "dbias", "old_nll"}
OPTIONAL_OF = {PREF: {"ref_nll"}}
# pointers that need less than 16 bytes
SMALL = {"mean": 4, "rstd": 4, "nll": 4, "ref_nll": 4, "old_nll": 4, "advantages": 4, "loss": 4,
         "slope": 4, "ratios": 4, "counts": 4, "kl": 4, "clipped": 4, "dloss": 4, "dnll": 4}
OUTPUTS = {LN: ("y", "sum", "mean", "rstd"), LN_GRAD: ("dx", "dweight", "dbias", "scratch"),
           PREF: ("loss", "slope", "ratios", "counts", "scratch"), PREF_GRAD: ("dnll",),
           POLICY: ("loss", "kl", "clipped", "counts", "scratch"), POLICY_GRAD: ("dnll",)}
NAMES = dict(ids=lambda c: c.name)


@pytest.mark.parametrize("call", ALL, **NAMES)
def test_good_arguments_pass_the_checks(call):
    assert call() == CUDA                        # no GPU here: the launch is what fails


@pytest.mark.parametrize("call", ALL, **NAMES)
def test_null_and_misaligned_pointers(call):
    for k in pointers(call):
        if k not in OPTIONAL | OPTIONAL_OF.get(call, set()):
            assert call(**{k: None}) == NULL, k
        else:
            assert call(**{k: None}) == CUDA, k
        width = {"targets": "width", "offsets": "offset_width"}.get(k)
        need = call.good[width] if width else SMALL.get(k, 16)
        assert call(**{k: call.good[k] + need // 2}) == ALIGN, k
        if need < 16:
            assert call(**{k: call.good[k] + need}) == CUDA, k


@pytest.mark.parametrize("call", ALL, **NAMES)
def test_outputs_overlap_nothing(call):
    names = pointers(call)
    for out in OUTPUTS[call]:
        for other in names:
            if other != out:
                assert call(**{out: call.good[other]}) == OVERLAP, (out, other)
    if "status" in call.good:
        for other in names:
            assert call(status=call.good[other]) == OVERLAP, other
        assert call(status=at(20) + 2) == ALIGN


@pytest.mark.parametrize("call", NORMS, **NAMES)
def test_layer_norm_sizes(call):
    for bad in (dict(T=-1), dict(D=0), dict(D=60), dict(D=-8)):
        assert call(**bad) == INVALID
    assert call(T=1 << 31) == SIZE
    for k in call.good:
        if k.endswith("_ld"):
            assert call(**{k: 56}) == INVALID, k
            assert call(**{k: 68}) == INVALID, k
            assert call(**{k: 1 << 40}) == SIZE, k
    wide = {k: 1 << 15 for k in call.good if k.endswith("_ld")}
    assert call(D=z.ZERO_NORM_MAX_WIDTH + 8, **wide) == SIZE


def test_layer_norm_other_arguments():
    for eps in (-1.0, float("nan"), float("inf")):
        assert LN(eps=eps) == INVALID
    assert LN_GRAD(size=8) == SIZE
    assert LN_GRAD(dweight=None, dbias=None, scratch=None, size=0) == CUDA
    assert LN_GRAD(dbias=None, scratch=None) == NULL
    # no tokens: nothing per token is looked at, the weights' gradients are still written
    gone = {k: None for k in pointers(LN)}
    assert LN(T=0, **gone) == B.ZERO_OK
    gone = {k: None for k in pointers(LN_GRAD)}
    assert LN_GRAD(T=0, **gone) == B.ZERO_OK
    for k in ("dweight", "dbias"):
        assert LN_GRAD(T=0, **{**gone, k: at(1)}) == CUDA
    assert LN_GRAD(T=0, **{**gone, "dweight": at(1), "dbias": at(1)}) == OVERLAP


@pytest.mark.parametrize("call", LOSSES, **NAMES)
def test_loss_sizes(call):
    n = "P" if "P" in call.good else "S"
    for bad in (dict(T=-1), {n: -1}, dict(width=2), dict(offset_width=1), dict(average=2)):
        assert call(**bad) == INVALID, bad
    assert call(T=1 << 31) == SIZE
    assert call(**{n: (1 << 30) + 1}) == SIZE
    assert call(**{n: 1 << 62}) == SIZE
    if "size" in call.good:
        assert call(size=8) == SIZE
    gone = {k: None for k in pointers(call)}
    assert call(**{n: 0}, **gone) == B.ZERO_OK
    # without tokens the sequences' results are still written, and no gradient is
    if call in (PREF, POLICY):
        per_token = {"nll", "ref_nll", "old_nll", "targets"} & set(gone)
        assert call(T=0, **{k: None for k in per_token}) == CUDA
        assert call(T=0, offsets=None) == NULL
    else:
        assert call(T=0, **gone) == B.ZERO_OK


def test_loss_arguments():
    nan, inf = float("nan"), float("inf")
    for kind in (-1, 3):
        assert PREF(kind=kind) == INVALID
    for bad in ([dict(beta=b) for b in (0.0, -1.0, nan, inf)] +
                [dict(smoothing=s) for s in (-0.1, 0.5, nan)] +
                [dict(margin=m) for m in (nan, inf, -inf)] +
                [dict(kind=k, smoothing=0.1) for k in (1, 2)]):
        assert PREF(**bad) == INVALID, bad
    for kind in (1, 2):
        assert PREF(kind=kind, smoothing=0.0) == CUDA
    for call in (POLICY, POLICY_GRAD):
        for bad in ([dict(clip_low=c) for c in (-0.1, 1.1, nan)] +
                    [dict(clip_high=c) for c in (-0.1, nan, inf)] +
                    [dict(kl_coef=c) for c in (-0.1, nan, inf)] + [dict(per_token=2)]):
            assert call(**bad) == INVALID, bad
        assert call(clip_low=1.0, clip_high=10.0) == CUDA
        assert call(ref_nll=None, kl_coef=0.0) == CUDA
        assert call(ref_nll=None) == NULL


def test_inputs_may_be_the_same():
    assert LN(res=at(0), bias=at(2)) == CUDA
    assert LN_GRAD(dsum=at(0), x=at(0)) == CUDA
    assert PREF(ref_nll=at(0)) == CUDA
    assert POLICY(ref_nll=at(0), old_nll=at(0)) == CUDA


# ------------------------------------------------------- many tensors --

def table(*entries):
    """(address, elements, type) of each tensor as the C entry points take them."""
    return (B.zero_tensor * max(1, len(entries)))(*[B.zero_tensor(*e) for e in entries])


BF, FP16, FP32 = B.ZERO_TYPE_BF16, B.ZERO_TYPE_FP16, B.ZERO_TYPE_FP32
THREE = ((at(0), 1001, BF), (at(1), 7, FP16), (at(2), 500, FP32))


def norm(*entries, count=None, **other):
    good = dict(norm=at(10), norms=at(11), scratch=at(12), size=BIG, status=None, stream=None)
    if torch.cuda.is_available():
        pytest.skip("fake device addresses are used only on machines without a GPU")
    n = len(entries) if count is None else count
    return B.lib().zero_grad_norm(table(*entries), n, *{**good, **other}.values())


def clip(entries, outs=None, count=None, **other):
    good = dict(norm=at(10), max_norm=1.0, stream=None)
    if torch.cuda.is_available():
        pytest.skip("fake device addresses are used only on machines without a GPU")
    n = len(entries) if count is None else count
    return B.lib().zero_grad_clip(table(*entries), None if outs is None else table(*outs), n,
                                  *{**good, **other}.values())


def test_norm_arguments():
    assert norm(*THREE) == CUDA
    assert norm(*THREE, norms=None) == CUDA
    assert norm(count=-1) == INVALID
    assert norm(count=B.ZERO_MAX_TENSORS + 1) == SIZE
    assert B.lib().zero_grad_norm(None, 1, at(10), None, at(12), BIG, None, None) == NULL
    assert norm((at(0), -1, BF)) == INVALID
    assert norm((at(0), 5, 3)) == INVALID
    assert norm((at(0), 5, -1)) == INVALID
    assert norm((at(0), (1 << 40) + 1, BF)) == SIZE
    assert norm(*[(at(0), 1 << 40, BF)] * 9, norms=None, norm=1 << 60, scratch=1 << 61) == SIZE
    assert norm((None, 5, BF)) == NULL
    assert norm((at(0) + 1, 5, BF)) == ALIGN
    assert norm((at(0) + 2, 5, BF)) == CUDA              # aligned to its elements
    assert norm((at(0) + 2, 5, FP32)) == ALIGN
    for k, step in (("norm", 2), ("norms", 2), ("scratch", 8)):
        assert norm(*THREE, **{k: at(10) + step}) == ALIGN, k
    assert norm(*THREE, norm=None) == NULL and norm(*THREE, scratch=None) == NULL
    assert norm(*THREE, size=8) == SIZE
    assert norm(*THREE, status=at(13) + 2) == ALIGN
    for k in ("norm", "norms", "scratch"):
        assert norm(*THREE, **{k: at(1)}) == OVERLAP, k
    assert norm(*THREE, norm=at(12)) == OVERLAP
    assert norm(*THREE, status=at(2)) == OVERLAP
    # the same tensor twice counts twice; a call without tensors writes the norm alone
    assert norm(THREE[0], THREE[0]) == CUDA
    assert norm(norms=None, scratch=None) == CUDA
    assert norm((None, 0, BF)) == CUDA


def test_clip_arguments():
    outs = ((at(5), 1001, BF), (at(6), 7, BF), (at(7), 500, FP32))
    assert clip(THREE) == CUDA
    assert clip(THREE, outs) == CUDA
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert clip(THREE, max_norm=bad) == INVALID
    assert clip(THREE, norm=None) == NULL
    assert clip(THREE, norm=at(10) + 2) == ALIGN
    assert clip((), norm=None) == B.ZERO_OK
    assert clip(((None, 0, BF),)) == B.ZERO_OK           # nothing to launch for
    # sizes and types that do not match
    assert clip(THREE, (outs[0], outs[1], (at(7), 499, FP32))) == INVALID
    assert clip(THREE, ((at(5), 1001, FP16),) + outs[1:]) == INVALID
    assert clip(THREE, ((at(5), 1001, FP32),) + outs[1:]) == INVALID
    assert clip(THREE, ((None, 1001, BF),) + outs[1:]) == NULL
    # overlaps, in any order of addresses
    assert clip((THREE[0], THREE[0])) == OVERLAP
    assert clip((THREE[1], THREE[0], (at(0) + 2000, 1, BF))) == OVERLAP
    assert clip((THREE[1], THREE[0], (at(0) + 2002, 1, BF))) == CUDA
    assert clip(THREE, norm=at(1)) == OVERLAP
    assert clip(THREE, (outs[0], (at(0), 7, BF), outs[2])) == OVERLAP
    assert clip(THREE, (outs[0], outs[1], (at(5), 500, FP32))) == OVERLAP
    assert clip(THREE, outs, norm=at(7)) == OVERLAP
    assert clip((THREE[0], THREE[0]), ((at(5), 1001, BF), (at(6), 1001, BF))) == CUDA
    # a long tensor that starts first and reaches over several others
    assert clip(((at(0), 1 << 20, BF), (at(0) + (1 << 22), 4, BF), (at(0) + (1 << 19), 4, BF))) == OVERLAP


def test_scratch_sizes():
    L = B.lib()
    assert L.zero_layer_norm_grad_scratch_bytes(5, 12) == -1
    assert L.zero_preference_scratch_bytes(5, -1) == -1
    assert L.zero_preference_scratch_bytes(5, (1 << 29) + 1) == -1
    assert L.zero_policy_scratch_bytes(1 << 31, 5) == -1
    assert L.zero_grad_norm_scratch_bytes(-1) == -1
    assert L.zero_grad_norm_scratch_bytes(B.ZERO_MAX_TENSORS + 1) == -1
    with pytest.raises(ValueError):
        z.zero_policy_scratch_bytes(-1, 5)
    # what is enough for T tokens (or so many tensors) is enough for fewer
    for size in (lambda n: z.zero_layer_norm_grad_scratch_bytes(n, 1024),
                 lambda n: z.zero_preference_scratch_bytes(n, 7),
                 lambda n: z.zero_policy_scratch_bytes(1000, n),
                 lambda n: z.zero_grad_norm_scratch_bytes(n)):
        sizes = [size(n) for n in range(0, 5000, 7)]
        assert sizes == sorted(sizes) and sizes[0] >= 0


# ---------------------------------------------- the extension module --

T, D, S, P = 6, 64, 4, 2
M, ROW, PER = ((T, D), torch.bfloat16), ((D,), torch.bfloat16), ((T,), torch.float32)
IDS, OFF, SCRATCH = ((T,), torch.int64), ((S + 1,), torch.int32), ((1 << 20,), torch.int8)
WORD, SEQ, PAIR = ((1,), torch.int32), ((S,), torch.float32), ((P,), torch.float32)
COUNT, ONE = ((S,), torch.int32), ((1,), torch.float32)
CALLS = {
    "layer_norm": (M, ROW, ROW, M, PER, PER, M, M, 1e-5, None),
    "layer_norm_grad": (M, M, PER, PER, ROW, M, ROW, ROW, SCRATCH, M, None),
    "preference": (PER, PER, IDS, OFF, PAIR, PAIR, SEQ, COUNT, SCRATCH, 0, 0.1, 0.0, 0.0, True,
                   WORD, None),
    "preference_grad": (IDS, OFF, PAIR, COUNT, PAIR, PER, True, None),
    "policy": (PER, PER, PER, SEQ, IDS, OFF, SEQ, SEQ, COUNT, COUNT, SCRATCH, False, 0.2, 0.2, 0.1,
               True, WORD, None),
    "policy_grad": (PER, PER, PER, SEQ, IDS, OFF, COUNT, SEQ, PER, False, 0.2, 0.2, 0.1, True,
                    None),
}


@pytest.fixture(scope="module")
def lm(built):
    if torch.cuda.is_available():
        pytest.skip("the stand-ins for tensors are used only on machines without a GPU")
    from zero_optimizer_step_rs_gb300 import lm
    return lm._lm


def on(spec, device):
    return torch.empty(spec[0], dtype=spec[1], device=device) if isinstance(spec, tuple) else spec


@pytest.mark.parametrize("name", CALLS)
def test_tensors_on_two_gpus_are_refused(lm, name):
    tensors = [i for i, x in enumerate(CALLS[name]) if isinstance(x, tuple)]
    for other in tensors:
        with FakeTensorMode():
            args = [on(x, "cuda:1" if i == other else "cuda:0") for i, x in enumerate(CALLS[name])]
        with pytest.raises(ValueError, match="different devices"):
            getattr(lm, name)(*args)


@pytest.mark.parametrize("name", CALLS)
def test_types_and_shapes_are_checked(lm, name):
    for i, x in enumerate(CALLS[name]):
        if not isinstance(x, tuple) or x is SCRATCH or x is WORD:
            continue
        with FakeTensorMode():
            args = [on(y, "cuda:0") for y in CALLS[name]]
            args[i] = torch.empty(x[0], dtype=torch.float64, device="cuda:0")
        with pytest.raises(TypeError):
            getattr(lm, name)(*args)
        with FakeTensorMode():
            args[i] = torch.empty((*x[0], 2), dtype=x[1], device="cuda:0")[..., 0]
        with pytest.raises(ValueError):                      # strided columns
            getattr(lm, name)(*args)
        with FakeTensorMode():
            args[i] = torch.empty((3, *x[0]), dtype=x[1], device="cuda:0")
        with pytest.raises(ValueError):
            getattr(lm, name)(*args)


def test_numbers_of_sequences(lm):
    with FakeTensorMode():
        none = on(((0,), torch.int32), "cuda:0")
        even = on(((4,), torch.int32), "cuda:0")
        args = [on(x, "cuda:0") for x in CALLS["preference"]]
    for bad in (none, even):
        with pytest.raises(ValueError, match="offsets"):
            lm.preference(*args[:3], bad, *args[4:])
    with pytest.raises(OverflowError, match="kind"):
        lm.preference(*args[:9], 1 << 32, *args[10:])


def test_lists_of_tensors_are_checked(lm):
    with FakeTensorMode():
        a, b = (torch.empty(8, dtype=torch.bfloat16, device="cuda:0") for _ in range(2))
        far = torch.empty(8, dtype=torch.bfloat16, device="cuda:1")
        one, room = on(ONE, "cuda:0"), on(SCRATCH, "cuda:0")
        far_one = on(ONE, "cuda:1")
        gaps, wide = torch.empty(8, 2, dtype=torch.bfloat16, device="cuda:0")[:, 0], a.view(2, 4)
        broad = torch.empty(1, dtype=torch.bfloat16, device="cuda:0").expand(8)
        f64 = torch.empty(8, dtype=torch.float64, device="cuda:0")
        f32 = torch.empty(8, device="cuda:0")
        tall = torch.empty(4, 2, dtype=torch.bfloat16, device="cuda:0").t()
        two = torch.empty(2, device="cuda:0")
    for bad, error in (([a, far], ValueError), ([a, gaps], ValueError), ([broad], ValueError),
                       ([a, f64], TypeError), ([a, 3], TypeError), (3, TypeError),
                       ([a] * (B.ZERO_MAX_TENSORS + 1), ValueError)):
        with pytest.raises(error):
            lm.grad_norm(bad, one, room, None, None, None)
        with pytest.raises(error):
            lm.grad_clip(bad, one, 1.0, None, None)
        with pytest.raises((error, ValueError)):
            lm.grad_clip([a] * 2, one, 1.0, bad, None)
    with pytest.raises(ValueError, match="norms"):
        lm.grad_norm([a, b], one, room, one, None, None)
    for bad in (two, far_one):
        with pytest.raises(ValueError):
            lm.grad_norm([a, b], bad, room, None, None, None)
    with pytest.raises(ValueError, match="outs"):
        lm.grad_clip([a, b], one, 1.0, [a], None)
    with pytest.raises(TypeError, match="outs"):
        lm.grad_clip([a], one, 1.0, [f32], None)
    with pytest.raises(ValueError, match="strides"):
        lm.grad_clip([wide], one, 1.0, [tall], None)       # the same shape, other strides


def test_tensors_of_the_cpu_are_refused(lm):
    f = torch.zeros(4, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        z.zero_grad_norm([f], torch.zeros(1), torch.zeros(64))
    with pytest.raises(ValueError, match="CUDA"):
        z.zero_layer_norm(f.view(1, 4), None, None, f.view(1, 4), torch.zeros(1), torch.zeros(1))
    with pytest.raises(TypeError):
        z.zero_grad_norm(f[0].item(), torch.zeros(1), torch.zeros(64))
