"""8-bit integer operators (include/exl3_int8.h): quantise, dequantise, a norm that
quantises, products.

Tensors:
  codes  : int8 [..., n], n a multiple of 16
  scales : float32 [...], one for each row of codes
  x      : float16, bfloat16 or float32 [m, n_in]; its rows may be a slice of wider ones
A code c stands for c times its row's scale; a weight's rows are its outputs, so a
weight is codes [n_out, n_in] and scales [n_out].  With offsets (int32 [groups + 1])
there is one per group, [groups, n_out, ...], and rows offsets[g] .. offsets[g + 1] - 1
go through weight g.

    codes, scales, x = int8_rms_norm(y, norm_weight, x)             # x + y, and its norm in 8 bits
    q, k, v = (int8_matmul(codes, scales, *w) for w in (wq, wk, wv))

Nothing here is recorded by autograd and there are no gradients: a tensor that requires
grad is refused where grad mode is on.  int8_quantize takes one (a layer's parameter,
say): its scales depend on it, but are meant to be constants of what follows.
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd import forward_ad

from . import Exl3Error, _check
from ._args import (I32, I64, INDEX, SIZE, VOID, FLOATS, Function, call, dtype_code, need, need_rows, no_gradient,
                    on_device, on_stream, result, scratch, too_large)

PIECE = 16  # EXL3_INT8_PIECE
_CODES = {torch.int8: None}
_SCALES = {torch.float32: None}

_quantize = Function("exl3_int8_quantize", VOID, I32, I64, I32, I64, VOID, VOID, VOID)
_dequantize = Function("exl3_int8_dequantize", VOID, VOID, I64, I32, VOID, I32, VOID)
_norm = Function("exl3_int8_rms_norm", VOID, I32, I64, I32, I64, VOID, I64, VOID, I32, ctypes.c_double, VOID, VOID, VOID, VOID)
_bytes = Function("exl3_int8_workspace_bytes", I32, I32, I32, restype=I64)
_matmul = Function("exl3_int8_matmul", VOID, VOID, I32, VOID, I32, VOID, VOID, I32, I32, VOID, I32, VOID)
_linear = Function("exl3_int8_linear", VOID, I32, I32, I64, VOID, I32, VOID, VOID, I32, I32, VOID, VOID, SIZE, VOID)


def _whole(n: int, name: str) -> None:
    if n < PIECE or n % PIECE:
        raise Exl3Error(f"{name}: {n} columns, expected a positive multiple of {PIECE}")


def int8_quantize(x, codes=None, scales=None, stream=None):
    """x [rows, n] to (codes [rows, n], scales [rows])."""
    if stream is not None:
        return on_stream(stream, int8_quantize, x, codes, scales)
    rows, n, ld, code, at = need_rows(x, "x")
    _whole(n, "x")
    codes, c = result(codes, "codes", x, torch.int8, (rows, n))
    scales, s = result(scales, "scales", x, torch.float32, (rows,), 4)
    dev = x.get_device()
    if not dev == codes.get_device() == scales.get_device() >= 0:
        on_device(dev, x=x, codes=codes, scales=scales)
    call(_quantize, dev, at, code, rows, n, ld, c, s)
    return codes, scales


def int8_dequantize(codes, scales, dtype=torch.bfloat16, out=None, stream=None):
    """The values of codes [rows, n] and scales [rows], as dtype [rows, n]."""
    if stream is not None:
        return on_stream(stream, int8_dequantize, codes, scales, dtype, out)
    code = dtype_code(dtype, "dtype")
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise Exl3Error("codes: expected a torch tensor of two dimensions")
    rows, n = codes.shape
    if n >> 31:
        too_large("codes", codes.shape)
    _whole(n, "codes")
    c, s = need(codes, "codes", _CODES, (rows, n)), _scales(scales, "scales", (rows,))
    out, o = result(out, "out", codes, dtype, (rows, n))
    dev = codes.get_device()
    if not dev == scales.get_device() == out.get_device() >= 0:
        on_device(dev, codes=codes, scales=scales, out=out)
    call(_dequantize, dev, c, s, rows, n, o, code)
    return out


def int8_rms_norm(x, weight, residual=None, eps: float = 1e-6, codes=None, scales=None, added=None, stream=None):
    """The root-mean-square norm of h = x + residual (rounded to x's type), quantised.

    Returns (codes [rows, n], scales [rows], added): codes times scales stand for
    h * weight / sqrt(mean(h^2) + eps), and added is h, the next residual.  Without a
    residual h is x and the result (codes, scales).  weight [n] may be of another type
    than x.
    """
    if stream is not None:
        return on_stream(stream, int8_rms_norm, x, weight, residual, eps, codes, scales, added)
    rows, n, ld, code, at = need_rows(x, "x")
    _whole(n, "x")
    if x.requires_grad or forward_ad._current_level >= 0:
        no_gradient(x, "x")
    w = need(weight, "weight", FLOATS, (n,))
    if weight.requires_grad or forward_ad._current_level >= 0:
        no_gradient(weight, "weight")
    if not 0 <= eps < float("inf"):
        raise Exl3Error(f"eps: {eps}, expected a finite number that is not negative")
    ldr, r, h = 0, None, None
    if residual is not None:
        rrows, rn, ldr, rcode, r = need_rows(residual, "residual")
        if rrows != rows or rn != n:
            raise Exl3Error(f"residual: shape {tuple(residual.shape)}, expected {tuple(x.shape)}")
        if rcode != code:
            raise Exl3Error(f"residual: dtype {residual.dtype}, expected {x.dtype}")
        if residual.requires_grad or forward_ad._current_level >= 0:
            no_gradient(residual, "residual")
        added, h = result(added, "added", x, x.dtype, (rows, n))
    elif added is not None:
        raise Exl3Error("added: given without a residual")
    codes, c = result(codes, "codes", x, torch.int8, (rows, n))
    scales, s = result(scales, "scales", x, torch.float32, (rows,), 4)
    dev = x.get_device()
    if not (dev == weight.get_device() == codes.get_device() == scales.get_device() >= 0
            and (r is None or dev == residual.get_device() == added.get_device())):
        on_device(dev, x=x, weight=weight, residual=residual, codes=codes, scales=scales, added=added)
    call(_norm, dev, at, code, rows, n, ld, r, ldr, w, FLOATS[weight.dtype], eps, c, s, h)
    return (codes, scales) if r is None else (codes, scales, added)


@functools.lru_cache(maxsize=1024)  # a size, of sizes alone
def int8_workspace_bytes(rows: int, n_in: int, groups: int = 1) -> int:
    """Bytes of device scratch that int8_linear needs (0: none)."""
    if max(rows, n_in, groups) >> 31 or min(rows, n_in, groups) < -1 << 31:
        too_large("int8_workspace_bytes", (rows, n_in, groups))
    n = (_bytes.bound or _bytes.load())(rows, groups, n_in)
    if n < 0:
        _check(n, "exl3_int8_workspace_bytes")
    return n


def _scales(t, name: str, shape) -> int:
    """The address of scales, which need be no more than 4-byte aligned."""
    at = need(t, name, _SCALES, shape, 4)
    if t.requires_grad or forward_ad._current_level >= 0:
        no_gradient(t, name)
    return at


def _weight(codes, scales, offsets, n_in: int):
    """Addresses of a weight and its offsets, with the group count and n_out."""
    shape = codes.shape if isinstance(codes, torch.Tensor) else ()
    if len(shape) != (2 if offsets is None else 3):
        raise Exl3Error("codes: expected a torch tensor [n_out, n_in], or [groups, n_out, n_in] with offsets")
    n_out, groups = shape[-2], 1 if offsets is None else shape[0]
    if (n_out | groups) >> 31:
        too_large("codes", shape)
    if offsets is None:
        return need(codes, "codes", _CODES, (n_out, n_in)), _scales(scales, "scales", (n_out,)), None, 1, n_out
    return (need(codes, "codes", _CODES, (groups, n_out, n_in)), _scales(scales, "scales", (groups, n_out)),
            need(offsets, "offsets", INDEX, (groups + 1,)), groups, n_out)


def int8_matmul(x_codes, x_scales, codes, scales, dtype=torch.bfloat16, offsets=None, y=None, stream=None):
    """y [m, n_out] = X @ W^T for quantised rows X (x_codes [m, n_in], x_scales [m]):
    several projections of one input quantise it once."""
    if stream is not None:
        return on_stream(stream, int8_matmul, x_codes, x_scales, codes, scales, dtype, offsets, y)
    code = dtype_code(dtype, "dtype")
    if not isinstance(x_codes, torch.Tensor) or x_codes.dim() != 2:
        raise Exl3Error("x_codes: expected a torch tensor of two dimensions")
    m, n_in = x_codes.shape
    if (m | n_in) >> 31:
        too_large("x_codes", x_codes.shape)
    _whole(n_in, "x_codes")
    xc, xs = need(x_codes, "x_codes", _CODES, (m, n_in)), _scales(x_scales, "x_scales", (m,))
    c, s, at, groups, n_out = _weight(codes, scales, offsets, n_in)
    y, o = result(y, "y", x_codes, dtype, (m, n_out))
    dev = x_codes.get_device()
    if not (dev == x_scales.get_device() == codes.get_device() == scales.get_device() == y.get_device() >= 0
            and (at is None or offsets.get_device() == dev)):
        on_device(dev, x_codes=x_codes, x_scales=x_scales, codes=codes, scales=scales, offsets=offsets, y=y)
    call(_matmul, dev, xc, xs, m, at, groups, c, s, n_in, n_out, o, code)
    return y


def int8_linear(x, codes, scales, offsets=None, workspace=None, y=None, stream=None):
    """y [m, n_out] = Q(x) @ W^T in x's type, Q(x) the 8-bit quantisation of x.

    workspace: a uint8 device tensor of int8_workspace_bytes(m, n_in, groups); by
    default new scratch where that is not 0.
    """
    if stream is not None:
        return on_stream(stream, int8_linear, x, codes, scales, offsets, workspace, y)
    m, n_in, ld, code, src = need_rows(x, "x")
    if m >> 31:
        too_large("x", x.shape)
    _whole(n_in, "x")
    if x.requires_grad or forward_ad._current_level >= 0:
        no_gradient(x, "x")
    c, s, at, groups, n_out = _weight(codes, scales, offsets, n_in)
    y, o = result(y, "y", x, x.dtype, (m, n_out))
    dev = x.get_device()
    if not (dev == codes.get_device() == scales.get_device() == y.get_device() >= 0
            and (at is None or offsets.get_device() == dev)):
        on_device(dev, x=x, codes=codes, scales=scales, offsets=offsets, y=y)
    ws, nbytes, held = scratch(workspace, 0 if workspace is not None else int8_workspace_bytes(m, n_in, groups), x)
    call(_linear, dev, src, code, m, ld, at, groups, c, s, n_in, n_out, o, ws, nbytes)
    return y
