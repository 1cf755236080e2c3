"""Calls of the MXFP4 and expert operators that are refused, at the C ABI and in the
binding, and the package without torch.  CPU only: every case returns before
anything is launched."""
import contextlib
import os
import subprocess
import sys

import pytest
import torch

import decode_gemm_exl3_amd as ex

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # stand-ins for device addresses: no call below reaches the device
F16, BF16, F32 = 0, 1, 2
EINVAL = -1


@pytest.fixture(scope="module")
def lib():
    from decode_gemm_exl3_amd import moe, mxfp4
    for f in (mxfp4._quantize, mxfp4._dequantize, mxfp4._bytes, mxfp4._matmul, mxfp4._linear, moe._bytes, moe._sort,
              moe._gather, moe._combine, moe._backward):
        f.load()
    return ex.load()


def touching(at, nbytes, mine):
    """Addresses, 16 apart, of `mine` bytes that share a byte with `nbytes` bytes at `at`: the
    first, one in the middle and the last."""
    last = (nbytes - 1) // 16 * 16
    return [at + last, at + last // 32 * 16, at, at - (mine - 1) // 16 * 16]


# ---- results that share bytes with an argument, wherever the two begin ----

def test_mxfp4_results_that_touch_arguments(lib):
    rows, n, n_out, groups, f32 = 40, 64, 48, 3, 4
    x_bytes, codes, scales = rows * n * f32, rows * n // 2, rows * n // 32

    def quantize(x=A, c=4 * A, s=8 * A, ld=n):
        return lib.exl3_mxfp4_quantize(x, F32, rows, n, ld, c, s, None)
    for at in touching(A, x_bytes, codes):
        assert quantize(c=at) == EINVAL
    for at in touching(A, x_bytes, scales) + touching(4 * A, codes, scales):
        assert quantize(s=at) == EINVAL
    assert quantize(ld=2 * n, c=A + 39 * 2 * n * f32) == EINVAL         # the last of rows further apart
    assert quantize(ld=2 * n, c=A + 5 * 2 * n * f32 - 16) == EINVAL     # from the space before row 5 into it
    for at in touching(A, codes, x_bytes) + touching(4 * A, scales, x_bytes):
        assert lib.exl3_mxfp4_dequantize(A, 4 * A, rows, n, at, F32, None) == EINVAL

    y_bytes, w_codes, w_scales = rows * n_out * f32, groups * n_out * n // 2, groups * n_out * n // 32

    def matmul(y):
        return lib.exl3_mxfp4_matmul(A, 2 * A, rows, 3 * A, groups, 4 * A, 5 * A, n, n_out, y, F32, None)
    for at, nbytes in ((A, codes), (2 * A, scales), (3 * A, 4 * groups + 4), (4 * A, w_codes), (5 * A, w_scales)):
        for y in touching(at, nbytes, y_bytes):
            assert matmul(y) == EINVAL

    def linear(y=6 * A, ws=7 * A, given=1 << 30):
        return lib.exl3_mxfp4_linear(A, F32, rows, n, 3 * A, groups, 4 * A, 5 * A, n, n_out, y, ws, given, None)
    need = lib.exl3_mxfp4_workspace_bytes(rows, groups, n)
    assert need > 0
    for at, nbytes in ((A, x_bytes), (3 * A, 4 * groups + 4), (4 * A, w_codes), (5 * A, w_scales)):
        for y in touching(at, nbytes, y_bytes):
            assert linear(y=y) == EINVAL
        for ws in touching(at, nbytes, need):
            assert linear(ws=ws) == EINVAL
    for ws in touching(6 * A, y_bytes, need):
        assert linear(ws=ws) == EINVAL


def test_moe_results_that_touch_arguments(lib):
    tokens, k, n, f32 = 20, 2, 24, 4
    slots = tokens * k
    x, rows, index, w = tokens * n * f32, slots * n * f32, slots * 4, slots * 4

    def combine(y, weights=8 * A):
        return lib.exl3_moe_combine(A, F32, tokens, k, n, 2 * A, 3 * A, weights, F32, y, None)
    for at, nbytes in ((A, rows), (2 * A, index), (3 * A, 4), (8 * A, w)):
        for y in touching(at, nbytes, x):
            assert combine(y) == EINVAL
    assert combine(A + 16 * n, weights=None) == EINVAL

    for at, nbytes in ((A, x), (2 * A, index), (3 * A, 4)):
        for r in touching(at, nbytes, rows):
            assert lib.exl3_moe_gather(A, F32, tokens, k, n, 2 * A, 3 * A, r, None) == EINVAL

    def backward(drows=6 * A, dweights=7 * A):
        return lib.exl3_moe_combine_backward(A, 2 * A, F32, tokens, k, n, 3 * A, 4 * A, 5 * A, F32, drows, dweights, None)
    for at, nbytes in ((A, x), (2 * A, rows), (3 * A, index), (4 * A, 4), (5 * A, w)):
        for r in touching(at, nbytes, rows):
            assert backward(drows=r) == EINVAL
        for r in touching(at, nbytes, w):
            assert backward(dweights=r) == EINVAL
    for r in touching(6 * A, rows, w):
        assert backward(dweights=r) == EINVAL

    slots, experts = 3000, 20
    need, offsets = lib.exl3_moe_workspace_bytes(slots, experts), 4 * (experts + 1)
    assert need > 0

    def sort(order=2 * A, position=3 * A, offs=4 * A, ws=5 * A):
        return lib.exl3_moe_sort(A, 8, slots, experts, order, position, offs, ws, 1 << 30, None)
    for at in touching(A, 8 * slots, 4 * slots) + touching(3 * A, 4 * slots, 4 * slots):
        assert sort(order=at) == EINVAL
    for at in touching(A, 8 * slots, 4 * slots) + touching(4 * A, offsets, 4 * slots):
        assert sort(position=at) == EINVAL
    for at in touching(A, 8 * slots, offsets) + touching(2 * A, 4 * slots, offsets):
        assert sort(offs=at) == EINVAL
    for at, nbytes in ((A, 8 * slots), (2 * A, 4 * slots), (3 * A, 4 * slots), (4 * A, offsets)):
        for ws in touching(at, nbytes, need):
            assert sort(ws=ws) == EINVAL


# ---- tensors that ask for a gradient: it would be lost without a word ----

def differentiable_calls():
    """(call of its floating tensors, those tensors), on the CPU: past the checks of types and sizes
    the next refusal is that of the device."""
    ids, at = torch.zeros((3, 2), dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    c, s = torch.zeros((5, 32), dtype=torch.uint8), torch.zeros((5, 2), dtype=torch.uint8)
    x, rows, w, y = torch.zeros((3, 8)), torch.zeros((6, 8)), torch.zeros((3, 2)), torch.zeros((3, 5))
    return {
        "moe_gather": (lambda x, r: ex.moe_gather(x, ids, at, rows=r), (x, rows)),
        "moe_gather_backward": (lambda r, d: ex.moe_gather_backward(r, ids, at, dx=d), (rows, x)),
        "moe_combine": (lambda r, w, y: ex.moe_combine(r, ids, at, w, y=y), (rows, w, x)),
        "moe_combine_backward": (lambda d, r, w, dr, dw: ex.moe_combine_backward(d, r, ids, at, w, drows=dr, dweights=dw),
                                 (x, rows, w, rows.clone(), w.clone())),
        "mxfp4_linear": (lambda x, y: ex.mxfp4_linear(x, c, s, y=y), (torch.zeros((3, 64)), y)),
        "mxfp4_matmul": (lambda y: ex.mxfp4_matmul(c[:3], s[:3], c, s, torch.float32, y=y), (y,)),
        "mxfp4_dequantize": (lambda out: ex.mxfp4_dequantize(c, s, torch.float32, out=out), (torch.zeros((5, 64)),)),
    }


@pytest.mark.parametrize("name", differentiable_calls())
def test_gradients_are_refused_and_not_lost(name):
    from torch.autograd import forward_ad
    call, tensors = differentiable_calls()[name]
    for i, t in enumerate(tensors):
        asks = [u.clone() for u in tensors]
        asks[i].requires_grad_()
        with pytest.raises(ex.Exl3Error, match="requires grad"):
            call(*asks)
        with torch.no_grad(), pytest.raises(ex.Exl3Error, match="must be on a GPU"):
            call(*asks)
        with pytest.raises(ex.Exl3Error, match="must be on a GPU"):
            call(*(u.detach() for u in asks))
        with forward_ad.dual_level():
            asks = [u.clone() for u in tensors]
            asks[i] = forward_ad.make_dual(asks[i], torch.ones_like(t))
            with pytest.raises(ex.Exl3Error, match="tangent"):
                call(*asks)
            with pytest.raises(ex.Exl3Error, match="must be on a GPU"):
                call(*tensors)


def test_quantize_takes_a_parameter():
    with pytest.raises(ex.Exl3Error, match="must be on a GPU"):
        ex.mxfp4_quantize(torch.nn.Parameter(torch.zeros((3, 64))))


def test_an_autograd_function_calls_the_operators():
    """Inside one grad mode is off: the tensors that require grad outside are taken."""
    ids, at = torch.zeros((3, 2), dtype=torch.int32), torch.zeros(5, dtype=torch.int32)

    class Gather(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return ex.moe_gather(x, ids, at)
    with pytest.raises(ex.Exl3Error, match="must be on a GPU"):
        Gather.apply(torch.zeros((3, 8), requires_grad=True))


# ---- the package without torch ----

def in_a_new_process(code, blocked=True):
    """Runs code where torch cannot be imported (or only is not yet)."""
    block = """
import sys
class Block:
    def find_spec(self, name, path=None, target=None):
        if name.split(".")[0] == "torch":
            raise ModuleNotFoundError("No module named 'torch'", name="torch")
sys.meta_path.insert(0, Block())
""" if blocked else "import sys\n"
    r = subprocess.run([sys.executable, "-c", block + code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_import_star_needs_no_torch():
    in_a_new_process("""
from decode_gemm_exl3_amd import *
assert pack_info(256, 32, 3)["n_in"] == 256 and "torch" not in sys.modules
assert mxfp4_linear.__name__ == "mxfp4_linear"
try:
    mxfp4_linear(None, None, None)
except ModuleNotFoundError:
    pass
else:
    raise AssertionError
""")


def test_names_taken_before_torch_is_imported_work_after():
    in_a_new_process("""
import decode_gemm_exl3_amd as ex
from decode_gemm_exl3_amd import mxfp4_workspace_bytes, moe_sort
assert "torch" not in sys.modules
import torch
assert mxfp4_workspace_bytes(100, 512) == ex.mxfp4_workspace_bytes(100, 512) > 0
from decode_gemm_exl3_amd import mxfp4
assert ex.mxfp4_linear is mxfp4.mxfp4_linear and ex.mxfp4_workspace_bytes is mxfp4.mxfp4_workspace_bytes
try:
    moe_sort(torch.zeros((3, 2), dtype=torch.int32), n_experts=4)
except ex.Exl3Error as e:
    assert "must be on a GPU" in str(e)
else:
    raise AssertionError
""", blocked=False)


def test_workspace_of_sizes_far_below_zero():
    # cut to 32 bits these would be 0 and 64
    for bad in ((-1 << 32, 64, 1), (100, 64 - (1 << 32), 1), (100, 64, 1 - (1 << 32)), (-1 << 33, 1 << 31, 1)):
        with pytest.raises(ex.Exl3Error, match="below 2.31 and not negative"):
            ex.mxfp4_workspace_bytes(*bad)


def test_tensors_of_a_call_on_a_given_stream_are_marked(monkeypatch):
    """Each tensor is recorded on the stream that uses it: its memory is not handed out again before."""
    from decode_gemm_exl3_amd import _args

    class Stream:
        device_index = 0
    marked, stream = [], Stream()
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: marked.append((t, s)))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    a, b, c = torch.zeros(1), torch.zeros(2), torch.zeros(3)
    assert _args.on_stream(stream, lambda *args: len(args), a, None, b, 7, torch.float16, c) == 6
    assert [(t is u, s is stream) for (t, s), u in zip(marked, (a, b, c))] == [(True, True)] * 3 and len(marked) == 3
