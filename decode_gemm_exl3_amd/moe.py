"""Mixture-of-experts routing (include/exl3_moe.h).

    order, position, offsets = moe_sort(expert_ids, n_experts)
    rows = moe_gather(x, position, offsets)
    rows = mxfp4_linear(rows, codes, scales, offsets=offsets)     # one weight per expert
    y = moe_combine(rows, position, offsets, weights)

Tensors:
  expert_ids, position : [tokens, top_k]; ids outside 0 .. n_experts - 1 are dropped slots,
                         position holds each of 0 .. slots - 1 once, as moe_sort makes it
                         (a row that no entry names is not written)
  order                : int32 [tokens * top_k]
  offsets              : int32 [n_experts + 1]
  x, y                 : float16, bfloat16 or float32 [tokens, n]
  rows                 : the same type, [tokens * top_k, n], in the experts' order, dropped slots last
  weights              : float32, float16 or bfloat16 [tokens, top_k]

Nothing here is recorded by autograd: the gradients are calls of their own,
moe_gather_backward and moe_combine_backward.  A tensor that requires grad is
refused where grad mode is on (an autograd.Function's forward and backward run with
it off).
"""
from __future__ import annotations

import functools

import torch
from torch.autograd import forward_ad

from . import Exl3Error
from ._args import (FLOATS, I32, I64, INDEX, SIZE, VOID, Function, call, need, no_gradient, on_device,
                    on_stream, result, scratch, too_large)

MAX_EXPERTS = 1024  # EXL3_MOE_MAX_EXPERTS
_IDS = {torch.int32: 4, torch.int64: 8}

_bytes = Function("exl3_moe_workspace_bytes", I32, I32, restype=I64)
_sort = Function("exl3_moe_sort", VOID, I32, I32, I32, VOID, VOID, VOID, VOID, SIZE, VOID)
_gather = Function("exl3_moe_gather", VOID, I32, I32, I32, I32, VOID, VOID, VOID, VOID)
_combine = Function("exl3_moe_combine", VOID, I32, I32, I32, I32, VOID, VOID, VOID, I32, VOID, VOID)
_backward = Function("exl3_moe_combine_backward", VOID, VOID, I32, I32, I32, I32, VOID, VOID, VOID, I32, VOID, VOID, VOID)


@functools.lru_cache(maxsize=1024)  # a size, of sizes alone
def _workspace_bytes(slots: int, n_experts: int) -> int:
    return (_bytes.bound or _bytes.load())(slots, n_experts)


def moe_sort(expert_ids, n_experts: int, order=None, position=None, offsets=None, workspace=None, stream=None):
    """The slots sorted by expert, stable: (order, position, offsets).

    workspace: a uint8 device tensor of exl3_moe_workspace_bytes; by default new
    scratch where that is not 0.
    """
    if stream is not None:
        return on_stream(stream, moe_sort, expert_ids, n_experts, order, position, offsets, workspace)
    if not isinstance(expert_ids, torch.Tensor) or expert_ids.dim() != 2:
        raise Exl3Error("expert_ids: expected a torch tensor [tokens, top_k]")
    shape, slots = expert_ids.shape, expert_ids.numel()
    if slots >> 31:
        too_large("expert_ids", shape)
    ids = need(expert_ids, "expert_ids", _IDS, shape)
    if not 1 <= n_experts <= MAX_EXPERTS:
        raise Exl3Error(f"n_experts: {n_experts}, expected 1 to {MAX_EXPERTS}")
    order, o = result(order, "order", expert_ids, torch.int32, (slots,))
    position, p = result(position, "position", expert_ids, torch.int32, shape)
    offsets, f = result(offsets, "offsets", expert_ids, torch.int32, (n_experts + 1,))
    dev = expert_ids.get_device()
    if not dev == order.get_device() == position.get_device() == offsets.get_device() >= 0:
        on_device(dev, expert_ids=expert_ids, order=order, position=position, offsets=offsets)
    ws, nbytes, held = scratch(workspace, 0 if workspace is not None else _workspace_bytes(slots, n_experts), expert_ids)
    call(_sort, dev, ids, _IDS[expert_ids.dtype], slots, n_experts, o, p, f, ws, nbytes)
    return order, position, offsets


def _places(position, offsets):
    """Tokens, top_k, the address of position and that of the number of kept slots."""
    if not isinstance(position, torch.Tensor) or len(shape := position.shape) != 2 or shape[1] < 1:
        raise Exl3Error("position: expected a torch tensor [tokens, top_k]")
    if not isinstance(offsets, torch.Tensor) or len(ends := offsets.shape) != 1 or ends[0] < 2:
        raise Exl3Error("offsets: expected a torch tensor [n_experts + 1]")
    if shape[0] * shape[1] >> 31:
        too_large("position", shape)
    at, kept = position.data_ptr(), offsets.data_ptr()
    if not (position.dtype is offsets.dtype is torch.int32 and position.is_contiguous() and offsets.is_contiguous()) or (at | kept) & 15:
        need(position, "position", INDEX, shape)
        need(offsets, "offsets", INDEX, ends)
    return shape[0], shape[1], at, kept + 4 * (ends[0] - 1)


def _matrix(t, name: str, rows: int):
    """A floating tensor of `rows` rows: columns, exl3_dtype and address."""
    if not isinstance(t, torch.Tensor) or len(shape := t.shape) != 2 or shape[1] < 1:
        raise Exl3Error(f"{name}: expected a torch tensor of two dimensions")
    n, code, at = shape[1], FLOATS.get(t.dtype), t.data_ptr()
    if n >> 31:
        too_large(name, shape)
    if code is None or shape[0] != rows or not t.is_contiguous() or at & 15:
        need(t, name, FLOATS, (rows, n))
    if t.requires_grad or forward_ad._current_level >= 0:
        no_gradient(t, name)
    return n, code, at


def _weights(t, shape):
    """The address of the router's weights."""
    at = need(t, "weights", FLOATS, shape)
    if t.requires_grad or forward_ad._current_level >= 0:
        no_gradient(t, "weights")
    return at


def moe_gather(x, position, offsets, rows=None, stream=None):
    """rows[position[t, j]] = x[t]; the rows of dropped slots are zero."""
    if stream is not None:
        return on_stream(stream, moe_gather, x, position, offsets, rows)
    tokens, top_k, at, kept = _places(position, offsets)
    n, code, src = _matrix(x, "x", tokens)
    rows, dst = result(rows, "rows", x, x.dtype, (tokens * top_k, n))
    dev = x.get_device()
    if not dev == position.get_device() == offsets.get_device() == rows.get_device() >= 0:
        on_device(dev, x=x, position=position, offsets=offsets, rows=rows)
    call(_gather, dev, src, code, tokens, top_k, n, at, kept, dst)
    return rows


def moe_combine(rows, position, offsets, weights=None, y=None, stream=None):
    """y[t] = sum over j of weights[t, j] * rows[position[t, j]] (no weights: ones)."""
    if stream is not None:
        return on_stream(stream, moe_combine, rows, position, offsets, weights, y)
    tokens, top_k, at, kept = _places(position, offsets)
    n, code, src = _matrix(rows, "rows", tokens * top_k)
    w = None if weights is None else _weights(weights, (tokens, top_k))
    y, dst = result(y, "y", rows, rows.dtype, (tokens, n))
    dev = rows.get_device()
    if not (dev == position.get_device() == offsets.get_device() == y.get_device() >= 0
            and (w is None or weights.get_device() == dev)):
        on_device(dev, rows=rows, position=position, offsets=offsets, weights=weights, y=y)
    call(_combine, dev, src, code, tokens, top_k, n, at, kept, w, 0 if w is None else FLOATS[weights.dtype], dst)
    return y


def moe_gather_backward(drows, position, offsets, dx=None, stream=None):
    """The gradient of moe_gather: dx[t] = sum over j of drows[position[t, j]]."""
    return moe_combine(drows, position, offsets, None, dx, stream)


def moe_combine_backward(dy, rows, position, offsets, weights, drows=None, dweights=None, stream=None):
    """The gradients of moe_combine: (drows, dweights)."""
    if stream is not None:
        return on_stream(stream, moe_combine_backward, dy, rows, position, offsets, weights, drows, dweights)
    tokens, top_k, at, kept = _places(position, offsets)
    n, code, src = _matrix(rows, "rows", tokens * top_k)
    grad = need(dy, "dy", (rows.dtype,), (tokens, n))
    if dy.requires_grad or forward_ad._current_level >= 0:
        no_gradient(dy, "dy")
    w = _weights(weights, (tokens, top_k))
    drows, dst = result(drows, "drows", rows, rows.dtype, (tokens * top_k, n))
    dweights, dw = result(dweights, "dweights", weights, weights.dtype, (tokens, top_k))
    dev = rows.get_device()
    if not (dev == dy.get_device() == position.get_device() == offsets.get_device() == weights.get_device() == drows.get_device()
            == dweights.get_device() >= 0):
        on_device(dev, rows=rows, dy=dy, position=position, offsets=offsets, weights=weights, drows=drows, dweights=dweights)
    call(_backward, dev, grad, src, code, tokens, top_k, n, at, kept, w, FLOATS[weights.dtype], dst, dw)
    return drows, dweights
