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

Token ids are int32 or int64; negative ones take part in nothing.  Losses of tokens and
sequences are fp32 vectors, gradients given as a list may be bf16, fp16 or fp32.
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
                        "zero_norm_grad", "zero_xent", "zero_xent_grad", "zero_layer_norm",
                        "zero_layer_norm_grad", "zero_preference", "zero_preference_grad",
                        "zero_policy", "zero_policy_grad", "zero_grad_norm", "zero_grad_clip")))


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


# ------------------------------------------------------------ layer norm --

def zero_layer_norm(x, weight, bias, y, mean, rstd, residual=None, sum_out=None,
                    eps: float = 1e-5, stream=None) -> None:
    """y = (s - mean) * rstd * weight + bias of s = x + residual, the sum in bf16
    where sum_out is given, and mean and rstd [T] fp32; weight and bias [D]
    bf16, or None for ones and zeros."""
    code = _lm.layer_norm(x, weight, bias, y, mean, rstd, residual, sum_out, eps,
                          _address(stream))
    if code:
        raise ZeroError(code, "zero_layer_norm")


def zero_layer_norm_grad_scratch_bytes(T: int, D: int) -> int:
    return _bytes(lib().zero_layer_norm_grad_scratch_bytes(T, D),
                  "zero_layer_norm_grad_scratch_bytes")


def zero_layer_norm_grad(dy, x, mean, rstd, weight, dx, dweight, dbias, scratch, dsum=None,
                         stream=None) -> None:
    """dx (the gradient of x and of the residual alike, dsum added), dweight and
    dbias [D] bf16 (None where not wanted; scratch may be None where neither is),
    from what was normalised: zero_layer_norm's x, or its sum_out where there
    was a residual."""
    code = _lm.layer_norm_grad(dy, x, mean, rstd, weight, dx, dweight, dbias, scratch, dsum,
                               _address(stream))
    if code:
        raise ZeroError(code, "zero_layer_norm_grad")


# --------------------------------------- losses of packed sequences --
#
# nll, ref_nll and old_nll [T] fp32 are zero_xent's losses of the tokens under the
# model that is trained, a reference model and the model that wrote them; dnll [T]
# is zero_xent_grad's dloss.  Sequence s holds the tokens offsets[s] <= t <
# offsets[s + 1] (int32 or int64, one more than there are sequences); a token with
# a negative target takes part in nothing and has dnll 0, and dnll of tokens in no
# sequence is left as it is.

def zero_preference_scratch_bytes(T: int, P: int) -> int:
    return _bytes(lib().zero_preference_scratch_bytes(T, P), "zero_preference_scratch_bytes")


def zero_preference(nll, ref_nll, targets, offsets, loss, slope, ratios, counts, scratch,
                    kind: int = 0, beta: float = 0.1, smoothing: float = 0.0,
                    margin: float = 0.0, average: bool = False, dev_status=None,
                    stream=None) -> None:
    """loss [P] of pairs of a chosen (2p) and a rejected (2p + 1) sequence, from their
    log ratios (ratios [2P], sums of ref_nll - nll, or with average means; ref_nll
    None: of -nll): kind ZERO_PREF_SIGMOID with label smoothing, _HINGE or _IPO.
    slope [P] (the loss's derivative by the ratios' difference) and counts [2P] int32
    (tokens that count) are what the gradient takes."""
    code = _lm.preference(nll, ref_nll, targets, offsets, loss, slope, ratios, counts, scratch,
                          kind, beta, smoothing, margin, average, dev_status, _address(stream))
    if code:
        raise ZeroError(code, "zero_preference")


def zero_preference_grad(targets, offsets, slope, counts, dloss, dnll, average: bool = False,
                         stream=None) -> None:
    """dnll [T] from zero_preference's slope and counts (and its `average`) and the
    upstream gradient dloss [P] of each pair's loss."""
    code = _lm.preference_grad(targets, offsets, slope, counts, dloss, dnll, average,
                               _address(stream))
    if code:
        raise ZeroError(code, "zero_preference_grad")


def zero_policy_scratch_bytes(T: int, S: int) -> int:
    return _bytes(lib().zero_policy_scratch_bytes(T, S), "zero_policy_scratch_bytes")


def zero_policy(nll, old_nll, ref_nll, advantages, targets, offsets, loss, kl, clipped, counts,
                scratch, per_token: bool = False, clip_low: float = 0.2, clip_high: float = 0.2,
                kl_coef: float = 0.0, average: bool = True, dev_status=None,
                stream=None) -> None:
    """loss [S] of each sequence: -min(r A, clip(r) A) + kl_coef k, summed over its
    tokens, or with average their mean, with r = exp(old_nll - nll) (1 for old_nll
    None), A = advantages [S] (or [T], per_token), and k the estimate of the KL
    divergence from the reference, whose sums or means go to kl [S].  clipped and
    counts [S] int32: the tokens that are clipped, and those that count."""
    code = _lm.policy(nll, old_nll, ref_nll, advantages, targets, offsets, loss, kl, clipped,
                      counts, scratch, per_token, clip_low, clip_high, kl_coef, average,
                      dev_status, _address(stream))
    if code:
        raise ZeroError(code, "zero_policy")


def zero_policy_grad(nll, old_nll, ref_nll, advantages, targets, offsets, counts, dloss, dnll,
                     per_token: bool = False, clip_low: float = 0.2, clip_high: float = 0.2,
                     kl_coef: float = 0.0, average: bool = True, stream=None) -> None:
    """dnll [T] from zero_policy's arguments and counts, and the upstream gradient
    dloss [S] of each sequence's loss."""
    code = _lm.policy_grad(nll, old_nll, ref_nll, advantages, targets, offsets, counts, dloss,
                           dnll, per_token, clip_low, clip_high, kl_coef, average,
                           _address(stream))
    if code:
        raise ZeroError(code, "zero_policy_grad")


# ------------------------------------------------- norm of many tensors --

def zero_grad_norm_scratch_bytes(count: int) -> int:
    return _bytes(lib().zero_grad_norm_scratch_bytes(count), "zero_grad_norm_scratch_bytes")


def zero_grad_norm(grads, norm, scratch, norms=None, dev_status=None, stream=None) -> None:
    """norm [1] fp32 = the 2-norm of all of `grads`, a sequence of bf16, fp16 or fp32
    tensors that fill their memory (any order of dimensions, any alignment), and
    norms [len(grads)] fp32 each one's."""
    code = _lm.grad_norm(grads, norm, scratch, norms, dev_status, _address(stream))
    if code:
        raise ZeroError(code, "zero_grad_norm")


def zero_grad_clip(grads, norm, max_norm: float, outs=None, stream=None) -> None:
    """outs[i] = grads[i] * min(1, max_norm / (norm + 1e-6)), with zero_grad_norm's norm; each
    out has its tensor's type or is bf16.  outs None: in place."""
    code = _lm.grad_clip(grads, norm, max_norm, outs, _address(stream))
    if code:
        raise ZeroError(code, "zero_grad_clip")
