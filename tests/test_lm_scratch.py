"""Scratch sizes of the language-model operators: a buffer made for the largest
batch serves the smaller ones."""
import pytest
import torch

import zero_optimizer_step_rs_gb300 as z
from zero_optimizer_step_rs_gb300 import binding as B


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_rs_gb300 import build
    build.build()


def lengths(most):
    """Around the multiples of 256 and of 1024, and others in between."""
    near = {m * k + d for m in (256, 1024) for k in range(most // m) for d in (-1, 0, 1)}
    return sorted(t for t in near | set(range(1, most, 97)) | {most} if 1 <= t <= most)


def never_falls():
    for V, D in ((1000, 64), (50257, 768), (128256, 2048), (5003, 8192)):
        sizes = {
            "embed_grad": lambda t: z.zero_embed_grad_scratch_bytes(t, V, D),
            "norm_grad": lambda t: z.zero_norm_grad_scratch_bytes(t, D),
            "xent": lambda t: z.zero_xent_scratch_bytes(t, V, D),
            "xent_grad": lambda t: z.zero_xent_grad_scratch_bytes(t, V, D),
            "xent_grad, piece": lambda t: z.zero_xent_grad_scratch_bytes(t, V, D, 1024),
        }
        for name, size in sizes.items():
            before = 0
            for t in lengths(30_000):
                n = size(t)
                assert n >= before, (name, V, D, t, n, before)
                before = n


def test_a_size_never_falls_as_tokens_are_added():
    never_falls()


@pytest.mark.parametrize("T,V,D", [((1 << 31) - 1024, 1000, 65536), (1 << 25, 1 << 26, 64),
                                   (1, (1 << 31) - 1024, 65536)])
def test_sizes_that_a_call_refuses_have_no_scratch_size(T, V, D):
    """Sizes within each limit whose product is past what a launch counts: -1,
    where the call says that it does not take them (before it looks at a buffer)."""
    L = B.lib()
    word = 1 << 40
    sizes_and_calls = [
        (L.zero_embed_grad_scratch_bytes(T, V, D), lambda: L.zero_embed_grad(
            word, D, word, 8, T, 1.0, V, D, word, 0, None, 0, None, None)),
        (L.zero_xent_scratch_bytes(T, V, D), lambda: L.zero_xent(
            word, D, word, V, D, word, 8, T, word, word, None, 0, 0, None, None)),
        (L.zero_xent_grad_scratch_bytes(T, V, D, 0), lambda: L.zero_xent_grad(
            word, D, word, V, D, word, 8, T, word, word, word, D, word, 0, None, 0, 0, None, None)),
    ]
    for size, call in sizes_and_calls:
        # (without scratch a call that takes the sizes stops at the missing buffer)
        assert call() == (B.ZERO_ERR_SIZE if size == -1 else B.ZERO_ERR_NULL)
    assert -1 in (size for size, _ in sizes_and_calls)


@pytest.mark.gpu
def test_a_size_never_falls_as_tokens_are_added_on_a_gpu():
    """Where the number of SMs is known, the sum of dh is split for few tokens."""
    never_falls()


@pytest.mark.gpu
@pytest.mark.parametrize("most", [257, 2100, 9728])
def test_calls_take_a_buffer_made_for_more_tokens(most):
    V, D = 4000, 2048
    bf = dict(dtype=torch.bfloat16, device="cuda")
    scratch = torch.empty(max(z.zero_embed_grad_scratch_bytes(most, V, D),
                              z.zero_xent_grad_scratch_bytes(most, V, D)), dtype=torch.uint8,
                          device="cuda")
    embed = scratch[: z.zero_embed_grad_scratch_bytes(most, V, D)]
    xent = scratch[: z.zero_xent_grad_scratch_bytes(most, V, D)]
    grad, table = torch.empty((V, D), **bf), torch.zeros((V, D), **bf)
    for T in (1, 128, 256, 1025, 2090, 9000):
        if T > most:
            continue
        t = torch.arange(T, device="cuda") % V
        dy, lse, one = torch.ones((T, D), **bf), torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")
        z.zero_embed_grad(dy, t, grad, embed)
        assert grad[:, 0].float().sum().item() == T
        z.zero_xent_grad(dy, table, t, lse, one, torch.empty_like(dy), grad, xent)
