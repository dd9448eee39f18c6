"""The language-model operators of libzero_step.so around the optimizer step.

Argument marshalling, as in binding.py: shapes, types and strides are checked
here, everything else in the library; status codes become ZeroError.  The
caller owns every buffer, outputs and scratch among them; work goes to the
current torch stream of the current device unless `stream` says otherwise.

Activations are [T, D] bf16 matrices whose rows may be strided (columns
contiguous, strides multiples of 8); tables are contiguous [V, D] bf16, as
views of a replica or a gradient buffer at the tensor's offset:

    grad_table = grads[0][off:off + V * D].view(V, D)

Token ids are int32 or int64; negative ones take part in nothing.
"""
from __future__ import annotations

import torch

from .binding import (ZERO_NORM_BLOCK, ZERO_OK, ZeroError, _check, lib)

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_bf16, _f32, _i8 = torch.bfloat16, torch.float32, torch.int8
_ID_BYTES = {torch.int32: 4, torch.int64: 8}


def _stream(stream, t):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(t.get_device())
        return torch.cuda.current_stream(t.device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _refuse(t, dtype, shape, name):
    """Says why a tensor was refused.  (The checks themselves are one condition:
    for a small call they are a good part of its time.)"""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: " + ("columns" if t.dim() == 2 else "elements") +
                     " must be contiguous")


def _rows(t, shape, name):
    """Address and row stride of a [T, D] bf16 matrix with contiguous columns."""
    if t.dtype is _bf16 and t.is_cuda and t.shape == shape:
        ld, step = t.stride()
        if step == 1:
            return t.data_ptr(), ld if shape[0] > 1 else shape[1]
    _refuse(t, _bf16, shape, name)


def _dense(t, dtype, shape, name):
    """Address of a contiguous tensor of that type and shape."""
    if t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, dtype, shape, name)


def _ids(t, name):
    """Address, bytes an id, and number of the token ids."""
    width = _ID_BYTES.get(t.dtype)
    if width is None:
        raise TypeError(f"{name}: expected int32 or int64, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous vector")
    return t.data_ptr(), width, t.shape[0]


def _scratch(t):
    if not t.is_cuda:
        raise ValueError("scratch: must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("scratch: tensor must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def _status(t):
    if t is None:
        return None
    if t.dtype is not torch.int32 or not t.is_cuda or t.numel() < 1:
        raise ValueError("dev_status: expected an int32 CUDA tensor")
    return t.data_ptr()


def _table(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a matrix, got shape {tuple(t.shape)}")
    return t.shape


def _bytes(n, where):
    if n < 0:
        raise ValueError(f"{where}: sizes out of range")
    return n


# ------------------------------------------------------------- embedding --

def zero_embed(table, tokens, out, scale: float = 1.0, dev_status=None, stream=None) -> None:
    """out[t] = scale * table[tokens[t]] (zeros for a negative id)."""
    V, D = _table(table, "table")
    ids, width, T = _ids(tokens, "tokens")
    dst, ld = _rows(out, (T, D), "out")
    code = lib().zero_embed(_dense(table, _bf16, (V, D), "table"), V, D, ids, width, T, scale, dst,
                            ld, _status(dev_status), _stream(stream, table))
    if code != ZERO_OK:
        raise ZeroError(code, "zero_embed")


def zero_embed_grad_scratch_bytes(T: int, V: int, D: int) -> int:
    return _bytes(lib().zero_embed_grad_scratch_bytes(T, V, D), "zero_embed_grad_scratch_bytes")


def zero_embed_grad(dy, tokens, grad, scratch, scale: float = 1.0, accumulate: bool = False,
                    dev_status=None, stream=None) -> None:
    """grad[v] = scale * sum of dy[t] over tokens[t] == v, in ascending t;
    with accumulate, added to what the rows met hold."""
    V, D = _table(grad, "grad")
    ids, width, T = _ids(tokens, "tokens")
    src, ld = _rows(dy, (T, D), "dy")
    room, size = _scratch(scratch)
    _check(lib().zero_embed_grad(src, ld, ids, width, T, scale, V, D,
                                 _dense(grad, _bf16, (V, D), "grad"), 1 if accumulate else 0, room,
                                 size, _status(dev_status), _stream(stream, grad)),
           "zero_embed_grad")


# ------------------------------------------------------------------ norm --

def zero_norm(x, weight, y, codes, scales, rstd, residual=None, sum_out=None, eps: float = 1e-5,
              stream=None) -> None:
    """y = norm(x + residual) * weight, the sum in bf16 where sum_out is given,
    and the 8-bit checkpoint (codes [T, D] int8, scales [T, ceil(D / 128)]
    fp32; None for both keeps none) with rstd [T] fp32."""
    T, D = _table(x, "x")
    src, x_ld = _rows(x, (T, D), "x")
    dst, y_ld = _rows(y, (T, D), "y")
    res, res_ld = _rows(residual, (T, D), "residual") if residual is not None else (None, 0)
    total, sum_ld = _rows(sum_out, (T, D), "sum_out") if sum_out is not None else (None, 0)
    blocks = (T, -(-D // ZERO_NORM_BLOCK))
    _check(lib().zero_norm(src, x_ld, res, res_ld, _dense(weight, _bf16, (D,), "weight"), T, D, eps,
                           dst, y_ld, total, sum_ld,
                           None if codes is None else _dense(codes, _i8, (T, D), "codes"),
                           None if scales is None else _dense(scales, _f32, blocks, "scales"),
                           _dense(rstd, _f32, (T,), "rstd"), _stream(stream, x)), "zero_norm")


def _checkpoint(codes, scales, rstd, weight):
    T, D = _table(codes, "codes")
    return T, D, (_dense(codes, _i8, (T, D), "codes"),
                  _dense(scales, _f32, (T, -(-D // ZERO_NORM_BLOCK)), "scales"),
                  _dense(rstd, _f32, (T,), "rstd"), _dense(weight, _bf16, (D,), "weight"))


def zero_norm_replay(codes, scales, rstd, weight, y, stream=None) -> None:
    """The normalised activation rebuilt from the checkpoint."""
    T, D, kept = _checkpoint(codes, scales, rstd, weight)
    dst, ld = _rows(y, (T, D), "y")
    _check(lib().zero_norm_replay(*kept, T, D, dst, ld, _stream(stream, y)), "zero_norm_replay")


def zero_norm_grad_scratch_bytes(T: int, D: int) -> int:
    return _bytes(lib().zero_norm_grad_scratch_bytes(T, D), "zero_norm_grad_scratch_bytes")


def zero_norm_grad(dy, codes, scales, rstd, weight, dx, dweight, scratch, dsum=None,
                   stream=None) -> None:
    """dx (the gradient of x and of the residual alike, dsum added) and
    dweight [D] bf16, from the checkpoint."""
    T, D, kept = _checkpoint(codes, scales, rstd, weight)
    src, dy_ld = _rows(dy, (T, D), "dy")
    dst, dx_ld = _rows(dx, (T, D), "dx")
    extra, dsum_ld = _rows(dsum, (T, D), "dsum") if dsum is not None else (None, 0)
    room, size = _scratch(scratch)
    _check(lib().zero_norm_grad(src, dy_ld, extra, dsum_ld, *kept, T, D, dst, dx_ld,
                                _dense(dweight, _bf16, (D,), "dweight"), room, size,
                                _stream(stream, dx)), "zero_norm_grad")


# --------------------------------------------------------- cross entropy --

def zero_xent_scratch_bytes(T: int, V: int, D: int) -> int:
    return _bytes(lib().zero_xent_scratch_bytes(T, V, D), "zero_xent_scratch_bytes")


def zero_xent(h, table, targets, loss, lse, scratch, flags: int = 0, dev_status=None,
              stream=None) -> None:
    """loss[t] and lse[t] (fp32) of the softmax over h @ table.T, whose
    logits are never stored; a negative target has no loss."""
    V, D = _table(table, "table")
    ids, width, T = _ids(targets, "targets")
    src, ld = _rows(h, (T, D), "h")
    room, size = _scratch(scratch)
    _check(lib().zero_xent(src, ld, _dense(table, _bf16, (V, D), "table"), V, D, ids, width, T,
                           _dense(loss, _f32, (T,), "loss"), _dense(lse, _f32, (T,), "lse"), room,
                           size, flags, _status(dev_status), _stream(stream, table)), "zero_xent")


def zero_xent_grad_scratch_bytes(T: int, V: int, D: int, piece: int = 0) -> int:
    return _bytes(lib().zero_xent_grad_scratch_bytes(T, V, D, piece),
                  "zero_xent_grad_scratch_bytes")


def zero_xent_grad(h, table, targets, lse, dloss, dh, dtable, scratch, piece: int = 0,
                   flags: int = 0, dev_status=None, stream=None) -> None:
    """dh [T, D] and dtable [V, D] from zero_xent's lse and the upstream
    gradient dloss [T] (fp32) of each token's loss; `piece` table rows at a
    time (a multiple of 256; 0: the library's choice)."""
    V, D = _table(table, "table")
    ids, width, T = _ids(targets, "targets")
    src, h_ld = _rows(h, (T, D), "h")
    dst, dh_ld = _rows(dh, (T, D), "dh")
    room, size = _scratch(scratch)
    _check(lib().zero_xent_grad(src, h_ld, _dense(table, _bf16, (V, D), "table"), V, D, ids, width,
                                T, _dense(lse, _f32, (T,), "lse"),
                                _dense(dloss, _f32, (T,), "dloss"), dst, dh_ld,
                                _dense(dtable, _bf16, (V, D), "dtable"), piece, room, size, flags,
                                _status(dev_status), _stream(stream, table)), "zero_xent_grad")
