"""MXFP4 operators (include/exl3_mxfp4.h): quantise, dequantise, products.

Tensors:
  codes  : uint8 [..., n / 2], two codes a byte, the lower column in the low half
  scales : uint8 [..., n / 32], 2^(b - 127) for each block of 32 columns
  x      : float16, bfloat16 or float32 [m, n_in]; its rows may be a slice of wider ones
A weight is codes [n_out, n_in / 2] and scales [n_out, n_in / 32]; with offsets
(int32 [groups + 1]) there is one per group, [groups, n_out, ...], and rows
offsets[g] .. offsets[g + 1] - 1 go through weight g.

Nothing here is recorded by autograd and the products have no gradient:
mxfp4_linear refuses an x that requires grad where grad mode is on.  mxfp4_quantize
takes one (a layer's parameter, say), as its results are integers.
"""
from __future__ import annotations

import functools

import torch
from torch.autograd import forward_ad

from . import Exl3Error, _check
from ._args import (BYTES, I32, I64, INDEX, SIZE, VOID, Function, call, dtype_code, need, need_rows, no_gradient,
                    on_device, on_stream, result, scratch, too_large)

BLOCK = 32  # EXL3_MXFP4_BLOCK

_quantize = Function("exl3_mxfp4_quantize", VOID, I32, I64, I32, I64, VOID, VOID, VOID)
_dequantize = Function("exl3_mxfp4_dequantize", VOID, VOID, I64, I32, VOID, I32, VOID)
_bytes = Function("exl3_mxfp4_workspace_bytes", I32, I32, I32, restype=I64)
_matmul = Function("exl3_mxfp4_matmul", VOID, VOID, I32, VOID, I32, VOID, VOID, I32, I32, VOID, I32, VOID)
_linear = Function("exl3_mxfp4_linear", VOID, I32, I32, I64, VOID, I32, VOID, VOID, I32, I32, VOID, VOID, SIZE, VOID)


def _blocks(n: int, name: str) -> int:
    if n < BLOCK or n % BLOCK:
        raise Exl3Error(f"{name}: {n} columns, expected a positive multiple of {BLOCK}")
    return n // BLOCK


def mxfp4_quantize(x, codes=None, scales=None, stream=None):
    """x [rows, n] to (codes [rows, n / 2], scales [rows, n / 32])."""
    if stream is not None:
        return on_stream(stream, mxfp4_quantize, x, codes, scales)
    rows, n, ld, code, at = need_rows(x, "x")
    blocks = _blocks(n, "x")
    codes, c = result(codes, "codes", x, torch.uint8, (rows, n // 2))
    scales, s = result(scales, "scales", x, torch.uint8, (rows, blocks))
    dev = x.get_device()
    if not dev == codes.get_device() == scales.get_device() >= 0:
        on_device(dev, x=x, codes=codes, scales=scales)
    call(_quantize, dev, at, code, rows, n, ld, c, s)
    return codes, scales


def mxfp4_dequantize(codes, scales, dtype=torch.bfloat16, out=None, stream=None):
    """The values of codes [rows, n / 2] and scales [rows, n / 32], as dtype [rows, n]."""
    if stream is not None:
        return on_stream(stream, mxfp4_dequantize, codes, scales, dtype, out)
    code = dtype_code(dtype, "dtype")
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise Exl3Error("codes: expected a torch tensor of two dimensions")
    rows, n = codes.shape[0], codes.shape[1] * 2
    if n >> 31:
        too_large("codes", codes.shape)
    blocks = _blocks(n, "codes")
    c, s = need(codes, "codes", BYTES, (rows, n // 2)), need(scales, "scales", BYTES, (rows, blocks))
    out, o = result(out, "out", codes, dtype, (rows, n))
    dev = codes.get_device()
    if not dev == scales.get_device() == out.get_device() >= 0:
        on_device(dev, codes=codes, scales=scales, out=out)
    call(_dequantize, dev, c, s, rows, n, o, code)
    return out


@functools.lru_cache(maxsize=1024)  # a size, of sizes alone: 0.6 us of a call otherwise
def mxfp4_workspace_bytes(rows: int, n_in: int, groups: int = 1) -> int:
    """Bytes of device scratch that mxfp4_linear needs (0: none)."""
    if max(rows, n_in, groups) >> 31 or min(rows, n_in, groups) < -1 << 31:
        too_large("mxfp4_workspace_bytes", (rows, n_in, groups))
    n = (_bytes.bound or _bytes.load())(rows, groups, n_in)
    if n < 0:
        _check(n, "exl3_mxfp4_workspace_bytes")
    return n


def _weight(codes, scales, offsets, n_in: int, blocks: int):
    """Addresses of a weight and its offsets, with the group count and n_out."""
    shape = codes.shape if isinstance(codes, torch.Tensor) else ()
    if len(shape) != (2 if offsets is None else 3):
        raise Exl3Error("codes: expected a torch tensor [n_out, n_in / 2], or [groups, n_out, n_in / 2] with offsets")
    n_out, groups = shape[-2], 1 if offsets is None else shape[0]
    if (n_out | groups) >> 31:
        too_large("codes", shape)
    if offsets is None:
        return need(codes, "codes", BYTES, (n_out, n_in // 2)), need(scales, "scales", BYTES, (n_out, blocks)), None, 1, n_out
    return (need(codes, "codes", BYTES, (groups, n_out, n_in // 2)), need(scales, "scales", BYTES, (groups, n_out, blocks)),
            need(offsets, "offsets", INDEX, (groups + 1,)), groups, n_out)


def mxfp4_matmul(x_codes, x_scales, codes, scales, dtype=torch.bfloat16, offsets=None, y=None, stream=None):
    """y [m, n_out] = X @ W^T for quantised rows X (x_codes [m, n_in / 2], x_scales
    [m, n_in / 32]): several projections of one input quantise it once."""
    if stream is not None:
        return on_stream(stream, mxfp4_matmul, x_codes, x_scales, codes, scales, dtype, offsets, y)
    code = dtype_code(dtype, "dtype")
    if not isinstance(x_codes, torch.Tensor) or x_codes.dim() != 2:
        raise Exl3Error("x_codes: expected a torch tensor of two dimensions")
    m, n_in = x_codes.shape[0], x_codes.shape[1] * 2
    if (m | n_in) >> 31:
        too_large("x_codes", x_codes.shape)
    blocks = _blocks(n_in, "x_codes")
    xc, xs = need(x_codes, "x_codes", BYTES, (m, n_in // 2)), need(x_scales, "x_scales", BYTES, (m, blocks))
    c, s, at, groups, n_out = _weight(codes, scales, offsets, n_in, blocks)
    y, o = result(y, "y", x_codes, dtype, (m, n_out))
    dev = x_codes.get_device()
    if not (dev == x_scales.get_device() == codes.get_device() == scales.get_device() == y.get_device() >= 0
            and (at is None or offsets.get_device() == dev)):
        on_device(dev, x_codes=x_codes, x_scales=x_scales, codes=codes, scales=scales, offsets=offsets, y=y)
    call(_matmul, dev, xc, xs, m, at, groups, c, s, n_in, n_out, o, code)
    return y


def mxfp4_linear(x, codes, scales, offsets=None, workspace=None, y=None, stream=None):
    """y [m, n_out] = Q(x) @ W^T in x's type, Q(x) the MXFP4 quantisation of x.

    workspace: a uint8 device tensor of mxfp4_workspace_bytes(m, n_in, groups); by
    default new scratch where that is not 0.
    """
    if stream is not None:
        return on_stream(stream, mxfp4_linear, x, codes, scales, offsets, workspace, y)
    m, n_in, ld, code, src = need_rows(x, "x")
    if m >> 31:
        too_large("x", x.shape)
    if x.requires_grad or forward_ad._current_level >= 0:
        no_gradient(x, "x")
    c, s, at, groups, n_out = _weight(codes, scales, offsets, n_in, _blocks(n_in, "x"))
    y, o = result(y, "y", x, x.dtype, (m, n_out))
    dev = x.get_device()
    if not (dev == codes.get_device() == scales.get_device() == y.get_device() >= 0
            and (at is None or offsets.get_device() == dev)):
        on_device(dev, x=x, codes=codes, scales=scales, offsets=offsets, y=y)
    ws, nbytes, held = scratch(workspace, 0 if workspace is not None else mxfp4_workspace_bytes(m, n_in, groups), x)
    call(_linear, dev, src, code, m, ld, at, groups, c, s, n_in, n_out, o, ws, nbytes)
    return y
