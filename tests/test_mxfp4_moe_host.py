"""Host-side checks of the MXFP4 and expert operators: the library exports what
the headers declare, refuses bad arguments before touching the GPU, and the
binding refuses bad tensors.  No kernel is launched here."""
import os
import re

import numpy as np
import pytest
import torch

import decode_gemm_exl3_amd as ex
import _mxfp4_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # stand-ins for device addresses: no call below reaches the device
F16, BF16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from decode_gemm_exl3_amd import moe, mxfp4
    for f in (mxfp4._quantize, mxfp4._dequantize, mxfp4._bytes, mxfp4._matmul, mxfp4._linear, moe._bytes, moe._sort,
              moe._gather, moe._combine, moe._backward):
        f.load()
    return ex.load()


@pytest.mark.parametrize("header, prefix, names", [
    ("exl3_mxfp4.h", "exl3_mxfp4_", {"quantize", "dequantize", "workspace_bytes", "matmul", "linear"}),
    ("exl3_moe.h", "exl3_moe_", {"workspace_bytes", "sort", "gather", "combine", "combine_backward"})])
def test_exports_every_declared_symbol(lib, header, prefix, names):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    assert set(re.findall(rf"\b{prefix}([a-z0-9_]+)\s*\(", src)) == names
    for n in names:
        assert hasattr(lib, prefix + n), n


def test_names_are_public():
    for n in ("mxfp4_quantize", "mxfp4_dequantize", "mxfp4_linear", "mxfp4_matmul", "mxfp4_workspace_bytes", "moe_sort",
              "moe_gather", "moe_gather_backward", "moe_combine", "moe_combine_backward"):
        assert n in ex.__all__ and callable(getattr(ex, n))
    with pytest.raises(AttributeError):
        ex.mxfp4_nothing


def test_reference_quantisation_by_hand():
    # amax 6 -> scale 1: codes 0 .. 7, ties to the even code, saturation below 8
    x = torch.zeros((3, 32))
    x[0, :11] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 7.9, -3, -0.0])
    x[1, 0], x[2, 0] = 2.0 ** -149, float("inf")
    codes, scales = R.quantize(x)
    assert scales[:, 0].tolist() == [127, 0, 255]
    code = np.stack([codes & 15, codes >> 4], -1).reshape(3, 32)
    assert code[0, :11].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 7, 13, 8]
    assert not code[1:].any()
    assert np.isnan(R.dequantize(codes, scales)[2]).all()


def test_workspace_sizes():
    assert ex.mxfp4_workspace_bytes(0, 32) == 0
    assert ex.mxfp4_workspace_bytes(1, 4096) == 0 and ex.mxfp4_workspace_bytes(64, 4096, 64) == 0  # quantised inside
    # codes and scales, each from a 256-byte border
    assert ex.mxfp4_workspace_bytes(2048, 4096) == 2048 * 2048 + 2048 * 128
    assert ex.mxfp4_workspace_bytes(333, 2080) >= 333 * 1040 + 333 * 65
    for bad in ((-1, 32, 1), (1, 0, 1), (1, 48, 1), (1, 32, 0)):
        with pytest.raises(ex.Exl3Error):
            ex.mxfp4_workspace_bytes(*bad)


def test_quantize_argument_errors(lib):
    def q(x=A, dtype=F16, rows=4, n=64, ld=64, codes=2 * A, scales=3 * A):
        return lib.exl3_mxfp4_quantize(x, dtype, rows, n, ld, codes, scales, None)
    assert q(dtype=3) == -1 and q(dtype=-1) == -1
    assert q(rows=-1) == -1 and q(n=0, ld=0) == -1 and q(n=48) == -1 and q(n=-32) == -1
    assert q(ld=63) == -1 and q(ld=68) == -1 and q(dtype=F32, ld=66) == -1   # rows off 16 bytes
    assert q(x=None) == -1 and q(codes=None) == -1 and q(scales=None) == -1
    assert q(x=A + 8) == -1 and q(codes=A + 4) == -1 and q(scales=A + 1) == -1
    assert q(rows=0, x=None, codes=None, scales=None) == 0
    assert q(rows=1 << 41) == -2 and q(rows=1 << 32) == -2

    def d(codes=A, scales=2 * A, rows=4, n=64, out=3 * A, dtype=F16):
        return lib.exl3_mxfp4_dequantize(codes, scales, rows, n, out, dtype, None)
    assert d(dtype=5) == -1 and d(rows=-1) == -1 and d(n=31) == -1
    assert d(codes=None) == -1 and d(scales=None) == -1 and d(out=None) == -1
    assert d(codes=A + 2) == -1 and d(scales=A + 2) == -1 and d(out=A + 8) == -1
    assert d(rows=0, codes=None, scales=None, out=None) == 0


def test_product_argument_errors(lib):
    def m(xc=A, xs=2 * A, rows=4, at=None, groups=1, c=3 * A, s=4 * A, n_in=64, n_out=5, y=5 * A, dtype=BF16):
        return lib.exl3_mxfp4_matmul(xc, xs, rows, at, groups, c, s, n_in, n_out, y, dtype, None)

    def f(x=A, dtype=BF16, rows=4, ld=64, at=None, groups=1, c=3 * A, s=4 * A, n_in=64, n_out=5, y=5 * A, ws=6 * A, wsb=1 << 40):
        return lib.exl3_mxfp4_linear(x, dtype, rows, ld, at, groups, c, s, n_in, n_out, y, ws, wsb, None)
    for g in (m, f):
        assert g(dtype=3) == -1 and g(rows=-1) == -1 and g(n_in=32 + 16) == -1 and g(n_in=0) == -1 and g(n_out=0) == -1
        assert g(groups=0) == -1 and g(groups=2) == -1                     # groups without offsets
        assert g(c=None) == -1 and g(s=None) == -1 and g(y=None) == -1
        assert g(c=A + 8) == -1 and g(s=A + 8) == -1 and g(y=A + 8) == -1 and g(at=A + 2) == -1
        assert g(groups=4097, at=7 * A) == -2 and g(rows=(1 << 23) + 1) == -2 and g(n_out=(1 << 24) + 1) == -2
        assert g(rows=1 << 23, n_out=1 << 14) == -2                      # 2^37 outputs
        assert g(rows=0, c=None, s=None, y=None) == 0
    assert m(n_in=(1 << 20) + 32) == -2 and f(n_in=(1 << 20) + 32, ld=(1 << 20) + 32) == -2
    assert m(xc=None) == -1 and m(xs=None) == -1 and m(xc=A + 1) == -1 and m(xs=A + 1) == -1 and m(xc=5 * A) == -1
    assert f(x=None) == -1 and f(x=A + 2) == -1 and f(x=5 * A) == -1 and f(ld=32) == -1 and f(ld=65) == -1 and f(ws=6 * A + 8) == -1
    assert f(rows=100, ws=None) == -3 and f(rows=100, wsb=100) == -3
    assert f(rows=1000, at=7 * A, groups=3, ws=None) == -3


def test_moe_argument_errors(lib):
    def s(ids=A, nbytes=4, slots=8, experts=4, order=2 * A, pos=3 * A, offs=4 * A, ws=5 * A, wsb=1 << 40):
        return lib.exl3_moe_sort(ids, nbytes, slots, experts, order, pos, offs, ws, wsb, None)
    assert s(nbytes=2) == -1 and s(slots=-1) == -1 and s(experts=0) == -1 and s(experts=1025) == -1
    assert s(ids=None) == -1 and s(order=None) == -1 and s(pos=None) == -1 and s(offs=None) == -1
    assert s(ids=A + 4) == -1 and s(order=A + 4) == -1 and s(pos=A + 4) == -1 and s(offs=A + 4) == -1 and s(ws=A + 4) == -1
    assert s(slots=1 << 20, ws=None) == -3 and s(slots=1 << 20, wsb=64) == -3
    assert s(slots=(1 << 30) + 1) == -2
    assert lib.exl3_moe_workspace_bytes(64, 8) == 0 and lib.exl3_moe_workspace_bytes(1 << 20, 8) > 0
    assert lib.exl3_moe_workspace_bytes(-1, 8) == -1 and lib.exl3_moe_workspace_bytes(8, 0) == -1

    def g(x=A, dtype=F16, tokens=4, k=2, n=10, pos=2 * A, kept=3 * A, rows=4 * A):
        return lib.exl3_moe_gather(x, dtype, tokens, k, n, pos, kept, rows, None)

    def c(x=A, dtype=F16, tokens=4, k=2, n=10, pos=2 * A, kept=3 * A, rows=4 * A, w=5 * A, wd=F32):
        return lib.exl3_moe_combine(x, dtype, tokens, k, n, pos, kept, w, wd, rows, None)

    def b(x=A, dtype=F16, tokens=4, k=2, n=10, pos=2 * A, kept=3 * A, rows=4 * A, w=5 * A, wd=F32, src=6 * A, dw=7 * A):
        return lib.exl3_moe_combine_backward(x, src, dtype, tokens, k, n, pos, kept, w, wd, rows, dw, None)
    for f in (g, c, b):
        assert f(dtype=3) == -1 and f(tokens=-1) == -1 and f(k=0) == -1 and f(n=0) == -1
        assert f(x=None) == -1 and f(pos=None) == -1 and f(kept=None) == -1 and f(rows=None) == -1 and f(rows=A) == -1
        assert f(x=A + 8) == -1 and f(pos=A + 8) == -1 and f(kept=A + 2) == -1 and f(rows=A + 8) == -1
        assert f(tokens=1 << 24) == -2 and f(tokens=1 << 20, k=64) == -2 and f(n=(1 << 24) + 1) == -2
        assert f(tokens=0, x=None) == 0
    for f in (c, b):
        assert f(wd=4) == -1 and f(w=A + 8) == -1
    assert b(w=None) == -1 and b(src=None) == -1 and b(dw=None) == -1 and b(src=4 * A) == -1 and b(dw=5 * A) == -1


def test_results_over_arguments_are_refused(lib):
    # every workgroup reads what others write: the same pointer twice is an error, not a race
    q = lambda x, c, s: lib.exl3_mxfp4_quantize(x, F16, 4, 64, 64, c, s, None)  # noqa: E731
    assert q(A, A, 2 * A) == -1 and q(A, 2 * A, A) == -1 and q(A, 2 * A, 2 * A) == -1
    d = lambda c, s, o: lib.exl3_mxfp4_dequantize(c, s, 4, 64, o, F16, None)  # noqa: E731
    assert d(A, 2 * A, A) == -1 and d(A, 2 * A, 2 * A) == -1
    m = lambda y, at=None: lib.exl3_mxfp4_matmul(A, 2 * A, 4, at, 1, 3 * A, 4 * A, 64, 5, y, BF16, None)  # noqa: E731
    assert [m(k * A) for k in (1, 2, 3, 4)] == [-1] * 4 and m(5 * A, 5 * A) == -1
    f = lambda y, ws: lib.exl3_mxfp4_linear(A, BF16, 100, 64, None, 1, 3 * A, 4 * A, 64, 5, y, ws, 1 << 40, None)  # noqa: E731
    assert [f(k * A, 6 * A) for k in (1, 3, 4)] == [-1] * 3 and f(5 * A, 5 * A) == -1 and f(5 * A, A) == -1
    s = lambda i, o, p, f: lib.exl3_moe_sort(i, 4, 8, 4, o, p, f, None, 0, None)  # noqa: E731
    for args in ((1, 1, 3, 4), (1, 2, 1, 4), (1, 2, 2, 4), (1, 2, 3, 1), (1, 2, 3, 2), (1, 2, 3, 3)):
        assert s(*(k * A for k in args)) == -1
    b = lambda dr, dw: lib.exl3_moe_combine_backward(A, 2 * A, F32, 4, 2, 8, 3 * A, 4 * A, 5 * A, F32, dr, dw, None)  # noqa: E731
    assert [b(k * A, 7 * A) for k in (1, 2, 3, 4, 5, 7)] == [-1] * 6 and [b(6 * A, k * A) for k in (1, 2, 3, 5)] == [-1] * 4
    g = lambda rows: lib.exl3_moe_gather(A, F32, 4, 2, 8, 2 * A, 3 * A, rows, None)  # noqa: E731
    assert [g(k * A) for k in (1, 2, 3)] == [-1] * 3


def test_mxfp4_binding_rejects_bad_tensors():
    x = torch.zeros((3, 64), dtype=torch.bfloat16)
    c, s = torch.zeros((5, 32), dtype=torch.uint8), torch.zeros((5, 2), dtype=torch.uint8)
    at = torch.zeros(3, dtype=torch.int32)
    bad = [
        (lambda: ex.mxfp4_quantize(x.double()), "x: dtype"),
        (lambda: ex.mxfp4_quantize([1.0]), "x: expected a torch tensor"),
        (lambda: ex.mxfp4_quantize(x[0]), "x: expected two dimensions"),
        (lambda: ex.mxfp4_quantize(x[:, :40]), "x: 40 columns"),
        (lambda: ex.mxfp4_quantize(torch.zeros((64, 64), dtype=torch.bfloat16).t()[:, ::2]), "x: the values of a row"),
        (lambda: ex.mxfp4_quantize(torch.zeros((3, 68), dtype=torch.bfloat16)[:, :64]), "x: rows must start"),
        (lambda: ex.mxfp4_quantize(x, codes=c), "codes: shape"),
        (lambda: ex.mxfp4_quantize(x), "x: must be on a GPU"),
        (lambda: ex.mxfp4_dequantize(c, s[:4]), "scales: shape"),
        (lambda: ex.mxfp4_dequantize(c, s, torch.float64), "dtype: dtype"),
        (lambda: ex.mxfp4_dequantize(c, s), "codes: must be on a GPU"),
        (lambda: ex.mxfp4_linear(x, c[:, :16], s), "codes: shape"),
        (lambda: ex.mxfp4_linear(x, c.int(), s), "codes: dtype"),
        (lambda: ex.mxfp4_linear(x, c, s, offsets=at), "codes: expected"),
        (lambda: ex.mxfp4_linear(x, c[None], s[None], offsets=at), "offsets: shape"),
        (lambda: ex.mxfp4_linear(x, c[None], s[None], offsets=at[:2].long()), "offsets: dtype"),
        (lambda: ex.mxfp4_linear(x, c, s, y=torch.zeros((3, 5))), "y: dtype"),
        (lambda: ex.mxfp4_linear(x, c, s), "x: must be on a GPU"),
        (lambda: ex.mxfp4_matmul(c, s, c, s[:, :1]), "scales: (shape|must be contiguous)"),
        (lambda: ex.mxfp4_matmul(c, s, c, s, torch.int8), "dtype: dtype"),
        (lambda: ex.mxfp4_matmul(c, s, c, s), "x_codes: must be on a GPU"),
    ]
    for f, match in bad:
        with pytest.raises(ex.Exl3Error, match=match):
            f()


def test_moe_binding_rejects_bad_tensors():
    ids = torch.zeros((3, 2), dtype=torch.int32)
    at = torch.zeros(5, dtype=torch.int32)
    x, rows, w = torch.zeros((3, 8)), torch.zeros((6, 8)), torch.zeros((3, 2))
    bad = [
        (lambda: ex.moe_sort(ids[0], 4), "expert_ids: expected"),
        (lambda: ex.moe_sort(ids.short(), 4), "expert_ids: dtype"),
        (lambda: ex.moe_sort(ids, 0), "n_experts"),
        (lambda: ex.moe_sort(ids, 1025), "n_experts"),
        (lambda: ex.moe_sort(ids, 4, offsets=at[:4]), "offsets: shape"),
        (lambda: ex.moe_sort(ids, 4), "expert_ids: must be on a GPU"),
        (lambda: ex.moe_gather(x, ids.long(), at), "position: dtype"),
        (lambda: ex.moe_gather(x[:2], ids, at), "x: shape"),
        (lambda: ex.moe_gather(x.double(), ids, at), "x: dtype"),
        (lambda: ex.moe_gather(x, ids, at[:1]), "offsets: expected"),
        (lambda: ex.moe_gather(x, ids, at, rows=rows.half()), "rows: dtype"),
        (lambda: ex.moe_gather(x, ids, at), "x: must be on a GPU"),
        (lambda: ex.moe_combine(x, ids, at, w), "rows: shape"),
        (lambda: ex.moe_combine(rows, ids, at, w[:2]), "weights: shape"),
        (lambda: ex.moe_combine(rows, ids, at, w), "rows: must be on a GPU"),
        (lambda: ex.moe_combine_backward(x.half(), rows, ids, at, w), "dy: dtype"),
        (lambda: ex.moe_combine_backward(x, rows, ids, at, None), "weights: expected"),
        (lambda: ex.moe_combine_backward(x, rows, ids, at, w), "rows: must be on a GPU"),
        (lambda: ex.moe_gather_backward(rows[:5], ids, at), "rows: shape"),
    ]
    for f, match in bad:
        with pytest.raises(ex.Exl3Error, match=match):
            f()


def test_binding_rejects_sizes_beyond_32_bits():
    # ctypes cuts a size to 32 bits without an error; meta tensors stand for ones too large to allocate
    def t(*shape, dtype=torch.uint8):
        return torch.empty(shape, dtype=dtype, device="meta")
    big, f16, i32 = 2 ** 32 + 32, torch.float16, torch.int32
    ids, at = t(3, 2, dtype=i32), t(5, dtype=i32)
    bad = [
        lambda: ex.mxfp4_quantize(t(1, big, dtype=f16)),
        lambda: ex.mxfp4_dequantize(t(1, big // 2), t(1, big // 32)),
        lambda: ex.mxfp4_linear(t(big, 64, dtype=f16), t(5, 32), t(5, 2)),
        lambda: ex.mxfp4_linear(t(3, big, dtype=f16), t(5, big // 2), t(5, big // 32)),
        lambda: ex.mxfp4_linear(t(3, 64, dtype=f16), t(big, 32), t(big, 2)),
        lambda: ex.mxfp4_linear(t(3, 64, dtype=f16), t(big, 5, 32), t(big, 5, 2), offsets=t(big + 1, dtype=i32)),
        lambda: ex.mxfp4_linear(t(3, 64, dtype=f16), t(2, big, 32), t(2, big, 2), offsets=t(3, dtype=i32)),
        lambda: ex.mxfp4_matmul(t(big, 32), t(big, 2), t(5, 32), t(5, 2)),
        lambda: ex.mxfp4_matmul(t(3, big // 2), t(3, big // 32), t(5, big // 2), t(5, big // 32)),
        lambda: ex.mxfp4_matmul(t(3, 32), t(3, 2), t(big, 32), t(big, 2)),
        lambda: ex.mxfp4_workspace_bytes(big, 64),
        lambda: ex.mxfp4_workspace_bytes(64, big),
        lambda: ex.mxfp4_workspace_bytes(64, 64, big),
        lambda: ex.moe_sort(t(big // 2, 2, dtype=i32), 4),
        lambda: ex.moe_gather(t(big // 2, 1, dtype=f16), t(big // 2, 2, dtype=i32), at),
        lambda: ex.moe_gather(t(3, big, dtype=f16), ids, at),
        lambda: ex.moe_combine(t(6, big, dtype=f16), ids, at),
        lambda: ex.moe_combine_backward(t(3, big, dtype=f16), t(6, big, dtype=f16), ids, at, t(3, 2, dtype=f16)),
    ]
    for f in bad:
        with pytest.raises(ex.Exl3Error, match="below 2.31"):
            f()
