"""Mixture-of-experts routing (include/exl3_moe.h).

    order, position, offsets = moe_sort(expert_ids, n_experts)
    rows = moe_gather(x, position, offsets)
    rows = mxfp4_linear(rows, codes, scales, offsets=offsets)     # one weight per expert
    y = moe_combine(rows, position, offsets, weights)

Tensors:
  expert_ids, position : [tokens, top_k]; ids outside 0 .. n_experts - 1 are dropped slots
  order                : int32 [tokens * top_k]
  offsets              : int32 [n_experts + 1]
  x, y                 : float16, bfloat16 or float32 [tokens, n]
  rows                 : the same type, [tokens * top_k, n], in the experts' order, dropped slots last
  weights              : float32, float16 or bfloat16 [tokens, top_k]
"""
from __future__ import annotations

import torch

from . import Exl3Error
from ._args import FLOATS, I32, I64, INDEX, SIZE, VOID, call, declare, dtype_code, need, on_device, scratch

MAX_EXPERTS = 1024  # EXL3_MOE_MAX_EXPERTS
_IDS = {torch.int32: 4, torch.int64: 8}

_bytes = declare("exl3_moe_workspace_bytes", I32, I32, restype=I64)
_sort = declare("exl3_moe_sort", VOID, I32, I32, I32, VOID, VOID, VOID, VOID, SIZE, VOID)
_gather = declare("exl3_moe_gather", VOID, I32, I32, I32, I32, VOID, VOID, VOID, VOID)
_combine = declare("exl3_moe_combine", VOID, I32, I32, I32, I32, VOID, VOID, VOID, I32, VOID, VOID)
_backward = declare("exl3_moe_combine_backward", VOID, VOID, I32, I32, I32, I32, VOID, VOID, VOID, I32, VOID, VOID, VOID)


def moe_sort(expert_ids, n_experts: int, order=None, position=None, offsets=None, workspace=None, stream=None):
    """The slots sorted by expert, stable: (order, position, offsets)."""
    if not isinstance(expert_ids, torch.Tensor) or expert_ids.dim() != 2:
        raise Exl3Error("expert_ids: expected a torch tensor [tokens, top_k]")
    ids = need(expert_ids, "expert_ids", _IDS, expert_ids.shape)
    if not 1 <= n_experts <= MAX_EXPERTS:
        raise Exl3Error(f"n_experts: {n_experts}, expected 1 to {MAX_EXPERTS}")
    slots, like = expert_ids.numel(), {"dtype": torch.int32, "device": expert_ids.device}
    if order is None:
        order = torch.empty((slots,), **like)
    if position is None:
        position = torch.empty(expert_ids.shape, **like)
    if offsets is None:
        offsets = torch.empty((n_experts + 1,), **like)
    o, p = need(order, "order", INDEX, (slots,)), need(position, "position", INDEX, expert_ids.shape)
    f = need(offsets, "offsets", INDEX, (n_experts + 1,))
    dev = expert_ids.get_device()
    on_device(dev, expert_ids=expert_ids, order=order, position=position, offsets=offsets, workspace=workspace)
    ws = scratch(workspace, int(_bytes()(slots, n_experts)) if workspace is None else 0, expert_ids, stream)
    call(_sort, "exl3_moe_sort", dev, stream, ids, _IDS[expert_ids.dtype], slots, n_experts, o, p, f,
         None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel())
    return order, position, offsets


def _places(position, offsets):
    """Tokens, top_k, the address of position and that of the number of kept slots."""
    if not isinstance(position, torch.Tensor) or position.dim() != 2 or position.shape[1] < 1:
        raise Exl3Error("position: expected a torch tensor [tokens, top_k]")
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise Exl3Error("offsets: expected a torch tensor [n_experts + 1]")
    at, kept = need(position, "position", INDEX, position.shape), need(offsets, "offsets", INDEX, offsets.shape)
    return (*position.shape, at, kept + 4 * (offsets.shape[0] - 1))


def _width(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.shape[1] < 1:
        raise Exl3Error(f"{name}: expected a torch tensor of two dimensions")
    return t.shape[1]


def moe_gather(x, position, offsets, rows=None, stream=None):
    """rows[position[t, j]] = x[t]; the rows of dropped slots are zero."""
    tokens, top_k, at, kept = _places(position, offsets)
    n, code = _width(x, "x"), dtype_code(x, "x")
    src = need(x, "x", FLOATS, (tokens, n))
    if rows is None:
        rows = torch.empty((tokens * top_k, n), dtype=x.dtype, device=x.device)
    dst = need(rows, "rows", (x.dtype,), (tokens * top_k, n))
    dev = x.get_device()
    on_device(dev, x=x, position=position, offsets=offsets, rows=rows)
    call(_gather, "exl3_moe_gather", dev, stream, src, code, tokens, top_k, n, at, kept, dst)
    return rows


def moe_combine(rows, position, offsets, weights=None, y=None, stream=None):
    """y[t] = sum over j of weights[t, j] * rows[position[t, j]] (no weights: ones)."""
    tokens, top_k, at, kept = _places(position, offsets)
    n, code = _width(rows, "rows"), dtype_code(rows, "rows")
    src = need(rows, "rows", FLOATS, (tokens * top_k, n))
    w = None if weights is None else need(weights, "weights", FLOATS, (tokens, top_k))
    if y is None:
        y = torch.empty((tokens, n), dtype=rows.dtype, device=rows.device)
    dst = need(y, "y", (rows.dtype,), (tokens, n))
    dev = rows.get_device()
    on_device(dev, rows=rows, position=position, offsets=offsets, weights=weights, y=y)
    call(_combine, "exl3_moe_combine", dev, stream, src, code, tokens, top_k, n, at, kept, w,
         0 if weights is None else FLOATS[weights.dtype], dst)
    return y


def moe_gather_backward(drows, position, offsets, dx=None, stream=None):
    """The gradient of moe_gather: dx[t] = sum over j of drows[position[t, j]]."""
    return moe_combine(drows, position, offsets, None, dx, stream)


def moe_combine_backward(dy, rows, position, offsets, weights, drows=None, dweights=None, stream=None):
    """The gradients of moe_combine: (drows, dweights)."""
    tokens, top_k, at, kept = _places(position, offsets)
    n, code = _width(rows, "rows"), dtype_code(rows, "rows")
    src, grad = need(rows, "rows", FLOATS, (tokens * top_k, n)), need(dy, "dy", (rows.dtype,), (tokens, n))
    w = need(weights, "weights", FLOATS, (tokens, top_k))
    if drows is None:
        drows = torch.empty((tokens * top_k, n), dtype=rows.dtype, device=rows.device)
    if dweights is None:
        dweights = torch.empty((tokens, top_k), dtype=weights.dtype, device=rows.device)
    dst, dw = need(drows, "drows", (rows.dtype,), (tokens * top_k, n)), need(dweights, "dweights", (weights.dtype,), (tokens, top_k))
    dev = rows.get_device()
    on_device(dev, rows=rows, dy=dy, position=position, offsets=offsets, weights=weights, drows=drows, dweights=dweights)
    call(_backward, "exl3_moe_combine_backward", dev, stream, grad, src, code, tokens, top_k, n, at, kept, w,
         FLOATS[weights.dtype], dst, dw)
    return drows, dweights
