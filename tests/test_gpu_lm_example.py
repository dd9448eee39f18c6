"""examples/tied_lm_step.py: the operators together, from token ids to the step."""
import importlib.util
import os

import pytest
import torch

import zero_optimizer_step_rs_gb300 as z
from tests import lm_ref as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "tied_lm_step", os.path.join(ROOT, "examples", "tied_lm_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_against_autograd(example):
    """The flat gradient against 64-bit automatic differentiation of the model.
    The norm's gradient is taken from its checkpoint, whose values are off by up
    to half a code (amax / 254) and, over a block of 128 normal values, by about
    0.007 of their root mean square; with the activations and dh rounded to bf16
    on the way 0.03 in norm leaves room for both, and no wrong term would fit."""
    model = example.TiedModel(V=600, D=128, ctx=32, batch=4)
    tokens, targets = example.synthetic(model, 1)
    loss = model.backward(0, tokens, targets)
    table, wpe, w = (x.to(R.F).requires_grad_() for x in model.views(model.replicas[0]))
    s = table[tokens] * model.scale + wpe[model.pos]
    h = s / (s.square().mean(1, keepdim=True) + 1e-5).sqrt() * w
    l = h @ table.T
    ok = targets >= 0
    per = torch.logsumexp(l, 1) - l.gather(1, targets.clamp(min=0)[:, None])[:, 0]
    want = per[ok].mean()
    want.backward()
    assert abs(loss.item() - want.item()) <= 0.01 * want.item()
    for got, x in zip(model.views(model.grads[0]), (table, wpe, w)):
        R.norm_close(got, x.grad, 0.03)


def test_training_lowers_the_loss(example):
    model = example.TiedModel()
    losses = [model.step(t, [example.synthetic(model, 2 * t + r) for r in range(model.R)])
              for t in range(1, 61)]
    first, last = losses[0].item(), losses[-1].item()
    assert last < 0.8 * first
    assert z.zero_get_device_status(model.status) == (0, 0)
    assert torch.equal(model.replicas[0], model.replicas[1])
