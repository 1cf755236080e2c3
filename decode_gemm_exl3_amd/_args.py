"""Argument checks shared by the bindings of the MXFP4, 8-bit and expert operators.

The library reads and writes raw device memory, so every tensor is checked for
element type, shape, contiguity, 16-byte alignment and device before a call
reaches it.  The calls run on the device of their first tensor, on `stream` or on
that device's current stream.  Results are outside autograd's graph: a tensor that
would have to pass a gradient on is refused.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd import forward_ad

from . import Exl3Error, _check, load

VOID, I32, I64, SIZE = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
FLOATS = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}  # enum exl3_dtype
BYTES = {torch.uint8: None}
INDEX = {torch.int32: None}


class Function:
    """A function of the library, its types set on the first use."""
    __slots__ = ("name", "argtypes", "restype", "bound")

    def __init__(self, name: str, *argtypes, restype=ctypes.c_int):
        self.name, self.argtypes, self.restype, self.bound = name, argtypes, restype, None

    def load(self):
        f = getattr(load(), self.name)
        f.argtypes, f.restype = self.argtypes, self.restype
        self.bound = f
        return f


def dtype_code(t, name: str) -> int:
    """exl3_dtype of a floating tensor (or dtype)."""
    dtype = t if isinstance(t, torch.dtype) else getattr(t, "dtype", None)
    code = FLOATS.get(dtype)
    if code is None:
        if dtype is None:
            raise Exl3Error(f"{name}: expected a torch tensor")
        raise Exl3Error(f"{name}: dtype {dtype}, expected one of {tuple(str(d) for d in FLOATS)}")
    return code


def too_large(name: str, shape):
    """The library takes its sizes as 32-bit numbers, and ctypes would cut longer ones."""
    raise Exl3Error(f"{name}: shape {tuple(shape)}, sizes must be below 2^31 and not negative")


def need(t, name: str, dtypes, shape, align: int = 16) -> int:
    """Checks all but the device; returns the address."""
    if not isinstance(t, torch.Tensor):
        raise Exl3Error(f"{name}: expected a torch tensor")
    at = t.data_ptr()
    if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and not at & (align - 1):
        return at
    if t.dtype not in dtypes:
        raise Exl3Error(f"{name}: dtype {t.dtype}, expected one of {tuple(str(d) for d in dtypes)}")
    if t.shape != shape:
        raise Exl3Error(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise Exl3Error(f"{name}: must be contiguous")
    raise Exl3Error(f"{name}: data must be {align}-byte aligned (a view at an offset is not)")


def no_gradient(t, name: str) -> None:
    """Raises where t asks for a gradient or carries a tangent: nothing would flow
    through the call, and nothing else would say so.  (Callers come here only if t
    requires grad or a level of forward mode is open: 0.1 us of a call, not 0.4.)"""
    if t.requires_grad and torch.is_grad_enabled():
        raise Exl3Error(f"{name}: requires grad, but the results are outside autograd's graph: pass it detached or call under "
                        "torch.no_grad() (moe_gather_backward, moe_combine_backward and moe_balance_loss_backward are the gradients there are)")
    if forward_ad.unpack_dual(t).tangent is not None:
        raise Exl3Error(f"{name}: carries a tangent, but the results are outside autograd's graph")


def result(t, name: str, like, dtype, shape, align: int = 16):
    """A given output, checked, or a new one beside `like`; with its address."""
    if t is None:
        # sizes one by one, and no dtype where it is the same: 1.2 us against 1.6
        t = like.new_empty(*shape) if dtype is like.dtype else like.new_empty(*shape, dtype=dtype)
        return t, t.data_ptr()
    at = need(t, name, (dtype,), shape, align)
    if t.requires_grad or forward_ad._current_level >= 0:
        no_gradient(t, name)
    return t, at


def need_rows(t, name: str):
    """A 2-dimensional floating tensor whose rows are contiguous and start at
    multiples of 16 bytes: (rows, columns, row stride in elements, exl3_dtype, address)."""
    code = FLOATS.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None:
        dtype_code(t, name)
    shape = t.shape
    if len(shape) != 2:
        raise Exl3Error(f"{name}: expected two dimensions, got shape {tuple(shape)}")
    rows, n = shape
    if n >> 31:
        too_large(name, shape)
    ld, inner = t.stride()
    if rows <= 1:
        ld = n
    if (inner != 1 and n > 1) or ld < n:
        raise Exl3Error(f"{name}: the values of a row must be contiguous and rows must not overlap")
    at = t.data_ptr()
    if (at | ld * (4 if code == 2 else 2)) & 15:
        raise Exl3Error(f"{name}: rows must start at multiples of 16 bytes")
    return rows, n, ld, code, at


def on_device(dev: int, **tensors) -> None:
    """Raises unless every tensor is on GPU `dev`, the device of the first (the
    callers compare the devices themselves and come here to name the odd one)."""
    for name, t in tensors.items():
        if t is None:
            continue
        at = t.get_device()
        if at < 0:
            raise Exl3Error(f"{name}: must be on a GPU device")
        if at != dev:
            raise Exl3Error(f"{name}: on GPU {at}, the first tensor is on GPU {dev}")


# The current device without the check for a first use (0.1 us against 0.25: tensors
# on it are there already), and the handle of its current stream without a Stream
# object made for it (0.1 against 1.1 us, of about 7 for a whole call).
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def call(fn: Function, dev: int, *args) -> None:
    """fn(*args, stream) on GPU `dev` and its current stream."""
    if dev != _device():
        with torch.cuda.device(dev):
            return call(fn, dev, *args)
    status = (fn.bound or fn.load())(*args, _current(dev))
    if status != 0:
        _check(status, fn.name)


def on_stream(stream, fn, first, *args):
    """fn(first, *args) with `stream` the current one, so that results and scratch
    come from its memory as well and nothing of another stream is written early.  The
    tensors are marked as used there: one that is dropped right after the call (a
    temporary, say) keeps its memory until `stream` has passed it."""
    if isinstance(first, torch.Tensor) and first.get_device() >= 0 and first.get_device() != stream.device_index:
        raise Exl3Error(f"{fn.__name__}: the stream is of GPU {stream.device_index}, the tensors are on GPU {first.get_device()}")
    with torch.cuda.stream(stream):
        out = fn(first, *args)
    for t in (first, *args):
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    return out


def scratch(workspace, nbytes: int, like):
    """Address and size of `workspace` when given, else of scratch of the caching
    allocator; the third value keeps it alive for the call."""
    if workspace is None and nbytes == 0:
        return None, 0, None
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor):
            raise Exl3Error("workspace: expected a torch tensor")
        at = need(workspace, "workspace", BYTES, workspace.shape)
        if workspace.get_device() != like.get_device():
            on_device(like.get_device(), workspace=workspace)
        return at, workspace.numel(), workspace
    buf = like.new_empty(nbytes, dtype=torch.uint8)
    return buf.data_ptr(), nbytes, buf
