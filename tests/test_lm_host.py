"""The language-model operators' argument checks, which happen on the host
before any CUDA call, and their scratch sizes.  Needs no GPU."""
import pytest
import torch

import zero_optimizer_step_rs_gb300 as z
from zero_optimizer_step_rs_gb300 import binding as B

INVALID, NULL, ALIGN, SIZE, OVERLAP, CUDA = (B.ZERO_ERR_INVALID_ARG, B.ZERO_ERR_NULL,
                                             B.ZERO_ERR_ALIGN, B.ZERO_ERR_SIZE,
                                             B.ZERO_ERR_OVERLAP, B.ZERO_ERR_CUDA)
GAP = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_rs_gb300 import build
    build.build()


def at(k):
    """The k-th of a set of fake, aligned addresses that are far apart."""
    return (k + 1) * GAP


class Call:
    """An entry point with good arguments, any of which a test replaces."""

    def __init__(self, name, good):
        self.name, self.good = name, good

    def __call__(self, **other):
        assert set(other) <= set(self.good)
        # a call that got past the checks by mistake must find no GPU to touch
        if torch.cuda.is_available():
            pytest.skip("fake device addresses are used only on machines without a GPU")
        return getattr(B.lib(), self.name)(*{**self.good, **other}.values())


BIG = 1 << 38
EMBED = Call("zero_embed", dict(table=at(0), V=1000, D=64, tokens=at(1), width=8, T=50, scale=1.0,
                                out=at(2), out_ld=64, status=None, stream=None))
EMBED_GRAD = Call("zero_embed_grad", dict(
    dy=at(0), dy_ld=64, tokens=at(1), width=4, T=50, scale=1.0, V=1000, D=64, grad=at(2),
    accumulate=0, scratch=at(3), size=BIG, status=None, stream=None))
NORM = Call("zero_norm", dict(
    x=at(0), x_ld=64, res=at(1), res_ld=64, weight=at(2), T=50, D=64, eps=1e-5, y=at(3), y_ld=64,
    sum=at(4), sum_ld=64, codes=at(5), scales=at(6), rstd=at(7), stream=None))
REPLAY = Call("zero_norm_replay", dict(codes=at(0), scales=at(1), rstd=at(2), weight=at(3), T=50,
                                       D=64, y=at(4), y_ld=64, stream=None))
NORM_GRAD = Call("zero_norm_grad", dict(
    dy=at(0), dy_ld=64, dsum=at(1), dsum_ld=64, codes=at(2), scales=at(3), rstd=at(4),
    weight=at(5), T=50, D=64, dx=at(6), dx_ld=64, dweight=at(7), scratch=at(8), size=BIG,
    stream=None))
XENT = Call("zero_xent", dict(
    h=at(0), h_ld=64, table=at(1), V=1000, D=64, targets=at(2), width=8, T=50, loss=at(3),
    lse=at(4), scratch=at(5), size=BIG, flags=0, status=None, stream=None))
XENT_GRAD = Call("zero_xent_grad", dict(
    h=at(0), h_ld=64, table=at(1), V=1000, D=64, targets=at(2), width=8, T=50, lse=at(3),
    dloss=at(4), dh=at(5), dh_ld=64, dtable=at(6), piece=0, scratch=at(7), size=BIG, flags=0,
    status=None, stream=None))
ALL = (EMBED, EMBED_GRAD, NORM, REPLAY, NORM_GRAD, XENT, XENT_GRAD)
OPTIONAL = {"res", "sum", "dsum", "status", "stream"}


def pointers(call):
    return [k for k, v in call.good.items() if isinstance(v, int) and v >= GAP and k != "size"]


@pytest.mark.parametrize("call", ALL, ids=lambda c: c.name)
def test_good_arguments_pass_the_checks(call):
    assert call() == CUDA                        # no GPU here: the launch is what fails


@pytest.mark.parametrize("call", ALL, ids=lambda c: c.name)
def test_null_and_misaligned_pointers(call):
    for k in pointers(call):
        if k in ("codes", "scales") and call is NORM:
            assert call(**{k: None}) == NULL     # one of the two alone
        elif k not in OPTIONAL:
            assert call(**{k: None}) == NULL, k
        step = {"tokens": 2, "targets": 2, "loss": 2, "lse": 2, "dloss": 2}.get(k, 8)
        assert call(**{k: call.good[k] + step}) == ALIGN, k


@pytest.mark.parametrize("call", ALL, ids=lambda c: c.name)
def test_sizes_and_strides(call):
    assert call(T=-1) == INVALID
    assert call(D=0) == INVALID
    assert call(D=60) == INVALID
    assert call(D=-8) == INVALID
    assert call(T=1 << 31) == SIZE
    for k in call.good:
        if k.endswith("_ld"):
            assert call(**{k: 56}) == INVALID, k
            assert call(**{k: 68}) == INVALID, k
            assert call(**{k: 1 << 40}) == SIZE, k
    if "V" in call.good:
        assert call(V=0) == INVALID
        assert call(V=1 << 31) == SIZE
    if "width" in call.good:
        assert call(width=2) == INVALID
    if "size" in call.good:
        assert call(size=8) == SIZE
    if call in (NORM, REPLAY, NORM_GRAD):
        wide = {k: 1 << 15 for k in call.good if k.endswith("_ld")}
        assert call(D=z.ZERO_NORM_MAX_WIDTH + 8, **wide) == SIZE


def test_other_arguments():
    assert EMBED_GRAD(accumulate=2) == INVALID
    assert NORM(eps=-1.0) == INVALID
    assert NORM(eps=float("nan")) == INVALID
    assert NORM(eps=float("inf")) == INVALID
    assert XENT_GRAD(piece=100) == INVALID
    assert XENT_GRAD(piece=-256) == INVALID
    for call in (XENT, XENT_GRAD):
        assert call(flags=1) == INVALID
        assert call(flags=z.ZERO_FLAG_DEBUG_EXPIRE_WAITS) == NULL        # needs the status word
    for call in (EMBED, EMBED_GRAD, XENT, XENT_GRAD):
        assert call(status=at(9) + 2) == ALIGN
    # optional arguments left out
    assert NORM(res=None, sum=None, codes=None, scales=None) == CUDA
    assert NORM_GRAD(dsum=None) == CUDA


OUTPUTS = {"zero_embed": ("out",), "zero_embed_grad": ("grad", "scratch"),
           "zero_norm": ("y", "sum", "codes", "scales", "rstd"), "zero_norm_replay": ("y",),
           "zero_norm_grad": ("dx", "dweight", "scratch"), "zero_xent": ("loss", "lse", "scratch"),
           "zero_xent_grad": ("dh", "dtable", "scratch")}


@pytest.mark.parametrize("call", ALL, ids=lambda c: c.name)
def test_outputs_overlap_nothing(call):
    names = pointers(call)
    for out in OUTPUTS[call.name]:
        for other in names:
            if other != out:
                assert call(**{out: call.good[other]}) == OVERLAP, (out, other)


def test_inputs_may_be_the_same():
    assert NORM(res=at(0)) == CUDA
    assert NORM_GRAD(dsum=at(0)) == CUDA


@pytest.mark.parametrize("call", ALL, ids=lambda c: c.name)
def test_no_tokens_need_no_buffers(call):
    """T = 0 returns before a per-token pointer is looked at; the gradients of
    tables and weights are still written."""
    gone = {k: None for k in pointers(call)}
    for k in ("grad", "dweight", "dtable"):
        if k in gone:
            assert call(T=0, **gone) == NULL
            gone[k] = call.good[k]
            assert call(T=0, **gone) == CUDA                   # the zero fill
            break
    else:
        assert call(T=0, **gone) == B.ZERO_OK
    if call is EMBED_GRAD:
        assert call(T=0, accumulate=1, **gone) == B.ZERO_OK


def test_scratch_sizes():
    L = B.lib()
    assert L.zero_embed_grad_scratch_bytes(-1, 10, 64) == -1
    assert L.zero_norm_grad_scratch_bytes(5, 12) == -1
    assert L.zero_xent_scratch_bytes(5, 0, 64) == -1
    assert L.zero_xent_grad_scratch_bytes(5, 10, 64, 100) == -1
    with pytest.raises(ValueError):
        z.zero_xent_grad_scratch_bytes(5, 10, 60)
    # the loss keeps 8 bytes per row and 128 (or more) vocabulary rows, not the logits
    assert z.zero_xent_scratch_bytes(8192, 128256, 2048) < 8192 * 128256 * 4 / 50
    # a smaller piece of the vocabulary takes less
    small = z.zero_xent_grad_scratch_bytes(8192, 128256, 2048, 1024)
    assert small < z.zero_xent_grad_scratch_bytes(8192, 128256, 2048) < 8192 * 128256 * 2
    assert z.zero_xent_grad_scratch_bytes(1, 1, 8) > 0


def test_binding_checks_tensors():
    """Types, shapes, strides and devices, before the library is called."""
    f = torch.zeros(4, 64, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        z.zero_embed(f, t, f)
    with pytest.raises(TypeError, match="tokens"):
        z.zero_embed(f, t.to(torch.int16), f)
    with pytest.raises(ValueError, match="matrix"):
        z.zero_embed(f[0], t, f)
    with pytest.raises(TypeError, match="x"):
        z.zero_norm(f.float(), f[0], f, None, None, torch.zeros(4))
    meta = torch.zeros(4, 64, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="CUDA"):
        z.zero_norm_replay(meta.to(torch.int8), torch.zeros(4, 1), torch.zeros(4), f[0], f)
