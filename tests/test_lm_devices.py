"""A call of the language-model operators with tensors on different GPUs is
refused before anything is launched.  Tensors without memory that only say
where they lie stand in for the GPUs, so this needs none."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="the stand-ins are used only on machines without a GPU")

T, V, D = 4, 10, 64
BF, F32, I64, I8 = torch.bfloat16, torch.float32, torch.int64, torch.int8
M, TABLE, ROW, SCRATCH, WORD = ((T, D), BF), ((V, D), BF), ((D,), BF), ((1 << 20,), I8), ((1,), torch.int32)
IDS, PER, CODES, SCALES = ((T,), I64), ((T,), F32), ((T, D), I8), ((T, 1), F32)
# the tensors of each call of the extension module by position, and its other arguments
CALLS = {
    "embed": (TABLE, IDS, M, 1.0, WORD, None),
    "embed_grad": (M, IDS, TABLE, SCRATCH, 1.0, False, WORD, None),
    "norm": (M, ROW, M, CODES, SCALES, PER, M, M, 1e-5, None),
    "norm_replay": (CODES, SCALES, PER, ROW, M, None),
    "norm_grad": (M, CODES, SCALES, PER, ROW, M, ROW, SCRATCH, M, None),
    "xent": (M, TABLE, IDS, PER, PER, SCRATCH, 0, WORD, None),
    "xent_grad": (M, TABLE, IDS, PER, PER, M, TABLE, SCRATCH, 0, 0, WORD, None),
}


@pytest.fixture(scope="module")
def lm():
    from zero_optimizer_step_rs_gb300 import build
    build.build()
    from zero_optimizer_step_rs_gb300 import lm
    return lm._lm


def on(spec, device):
    return torch.empty(spec[0], dtype=spec[1], device=device) if isinstance(spec, tuple) else spec


@pytest.mark.parametrize("name", CALLS)
def test_tensors_on_two_gpus_are_refused(lm, name):
    tensors = [i for i, x in enumerate(CALLS[name]) if isinstance(x, tuple)]
    assert len(tensors) >= 4
    for other in tensors:
        with FakeTensorMode():
            args = [on(x, "cuda:1" if i == other else "cuda:0") for i, x in enumerate(CALLS[name])]
        with pytest.raises(ValueError, match="different devices"):
            getattr(lm, name)(*args)


@pytest.mark.parametrize("name,at", [("xent", 6), ("xent_grad", 9)])
@pytest.mark.parametrize("flags", [1 << 32, -(1 << 33), 1 << 80])
def test_flags_past_32_bits_are_refused(lm, name, at, flags):
    with FakeTensorMode():
        args = [on(x, "cuda:0") for x in CALLS[name]]
    args[at] = flags
    with pytest.raises(OverflowError):
        getattr(lm, name)(*args)
