"""The language-model operators of libzero_step.so around the optimizer step.

As in binding.py the caller owns every buffer, outputs and scratch among them,
status codes become ZeroError, and there is no fallback path; work goes to the
current torch stream of the tensors' device unless `stream` (a torch stream or
its address) says otherwise; that device (the same for all of a call's tensors) need
not be the current one.  Shapes, types, strides and devices are checked by
the extension module _lm (csrc/lm_binding.cpp; TypeError, ValueError), alignment,
sizes and overlaps by the library.

Activations are [T, D] bf16 matrices whose rows may be strided (columns
contiguous, strides multiples of 8); tables are contiguous [V, D] bf16, as
views of a replica or a gradient buffer at the tensor's offset:

    grad_table = grads[0][off:off + V * D].view(V, D)

Token ids are int32 or int64; negative ones take part in nothing.
"""
from __future__ import annotations

import ctypes

import torch  # noqa: F401  (its libraries are what the extension module links to)

from .binding import ZeroError, lib

try:
    from . import _lm
except ImportError as e:
    raise RuntimeError("the extension module _lm is missing or does not fit this torch: build it "
                       "with zero_optimizer_step_rs_gb300.build.build()") from e

_lm.bind(*(ctypes.cast(getattr(lib(), name), ctypes.c_void_p).value
           for name in ("zero_embed", "zero_embed_grad", "zero_norm", "zero_norm_replay",
                        "zero_norm_grad", "zero_xent", "zero_xent_grad")))


def _address(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def _bytes(n, where):
    if n < 0:
        raise ValueError(f"{where}: sizes out of range")
    return n


# ------------------------------------------------------------- embedding --

def zero_embed(table, tokens, out, scale: float = 1.0, dev_status=None, stream=None) -> None:
    """out[t] = scale * table[tokens[t]] (zeros for a negative id)."""
    code = _lm.embed(table, tokens, out, scale, dev_status, _address(stream))
    if code:
        raise ZeroError(code, "zero_embed")


def zero_embed_grad_scratch_bytes(T: int, V: int, D: int) -> int:
    return _bytes(lib().zero_embed_grad_scratch_bytes(T, V, D), "zero_embed_grad_scratch_bytes")


def zero_embed_grad(dy, tokens, grad, scratch, scale: float = 1.0, accumulate: bool = False,
                    dev_status=None, stream=None) -> None:
    """grad[v] = scale * sum of dy[t] over tokens[t] == v, in an order fixed by
    the sizes and the ids; with accumulate, added to what the rows met hold."""
    code = _lm.embed_grad(dy, tokens, grad, scratch, scale, accumulate, dev_status,
                          _address(stream))
    if code:
        raise ZeroError(code, "zero_embed_grad")


# ------------------------------------------------------------------ norm --

def zero_norm(x, weight, y, codes, scales, rstd, residual=None, sum_out=None, eps: float = 1e-5,
              stream=None) -> None:
    """y = norm(x + residual) * weight, the sum in bf16 where sum_out is given,
    and the 8-bit checkpoint (codes [T, D] int8, scales [T, ceil(D / 128)]
    fp32; None for both keeps none) with rstd [T] fp32."""
    code = _lm.norm(x, weight, y, codes, scales, rstd, residual, sum_out, eps, _address(stream))
    if code:
        raise ZeroError(code, "zero_norm")


def zero_norm_replay(codes, scales, rstd, weight, y, stream=None) -> None:
    """The normalised activation rebuilt from the checkpoint."""
    code = _lm.norm_replay(codes, scales, rstd, weight, y, _address(stream))
    if code:
        raise ZeroError(code, "zero_norm_replay")


def zero_norm_grad_scratch_bytes(T: int, D: int) -> int:
    return _bytes(lib().zero_norm_grad_scratch_bytes(T, D), "zero_norm_grad_scratch_bytes")


def zero_norm_grad(dy, codes, scales, rstd, weight, dx, dweight, scratch, dsum=None,
                   stream=None) -> None:
    """dx (the gradient of x and of the residual alike, dsum added) and
    dweight [D] bf16, from the checkpoint."""
    code = _lm.norm_grad(dy, codes, scales, rstd, weight, dx, dweight, scratch, dsum,
                         _address(stream))
    if code:
        raise ZeroError(code, "zero_norm_grad")


# --------------------------------------------------------- cross entropy --

def zero_xent_scratch_bytes(T: int, V: int, D: int) -> int:
    return _bytes(lib().zero_xent_scratch_bytes(T, V, D), "zero_xent_scratch_bytes")


def zero_xent(h, table, targets, loss, lse, scratch, flags: int = 0, dev_status=None,
              stream=None) -> None:
    """loss[t] and lse[t] (fp32) of the softmax over h @ table.T, whose
    logits are never stored; a negative target has no loss."""
    code = _lm.xent(h, table, targets, loss, lse, scratch, flags, dev_status, _address(stream))
    if code:
        raise ZeroError(code, "zero_xent")


def zero_xent_grad_scratch_bytes(T: int, V: int, D: int, piece: int = 0) -> int:
    return _bytes(lib().zero_xent_grad_scratch_bytes(T, V, D, piece),
                  "zero_xent_grad_scratch_bytes")


def zero_xent_grad(h, table, targets, lse, dloss, dh, dtable, scratch, piece: int = 0,
                   flags: int = 0, dev_status=None, stream=None) -> None:
    """dh [T, D] and dtable [V, D] from zero_xent's lse and the upstream
    gradient dloss [T] (fp32) of each token's loss; `piece` table rows at a
    time (a multiple of 256; 0: the library's choice)."""
    code = _lm.xent_grad(h, table, targets, lse, dloss, dh, dtable, scratch, piece, flags,
                         dev_status, _address(stream))
    if code:
        raise ZeroError(code, "zero_xent_grad")
