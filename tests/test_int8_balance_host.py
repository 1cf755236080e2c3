"""Host-side checks of the 8-bit operators and the balance loss: what the headers declare is
exported, bad arguments are refused before the GPU is touched, and the CPU definitions that the
GPU tests use are right.  No kernel is launched here."""
import os
import re

import numpy as np
import pytest
import torch

import decode_gemm_exl3_amd as ex
import _int8_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 24  # stand-ins for device addresses: no call below reaches the device
F16, BF16, F32 = 0, 1, 2
EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3
INT8 = ("int8_quantize", "int8_dequantize", "int8_rms_norm", "int8_linear", "int8_matmul", "int8_workspace_bytes")


@pytest.fixture(scope="module")
def lib():
    from decode_gemm_exl3_amd import int8, moe
    for f in (int8._quantize, int8._dequantize, int8._norm, int8._bytes, int8._matmul, int8._linear, moe._balance_bytes, moe._balance,
              moe._balance_backward):
        f.load()
    return ex.load()


@pytest.mark.parametrize("header, prefix, names", [
    ("exl3_int8.h", "exl3_int8_", {"quantize", "dequantize", "rms_norm", "workspace_bytes", "matmul", "linear"}),
    ("exl3_balance.h", "exl3_moe_balance_", {"workspace_bytes", "loss", "loss_backward"})])
def test_exports_every_declared_symbol(lib, header, prefix, names):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    assert set(re.findall(rf"\b{prefix}([a-z0-9_]+)\s*\(", src)) == names
    for n in names:
        assert hasattr(lib, prefix + n), n


def test_names_are_public():
    for n in INT8 + ("moe_balance_loss", "moe_balance_loss_backward"):
        assert n in ex.__all__ and callable(getattr(ex, n))


# ---- the definitions that the GPU tests use ----

def test_reference_quantisation_by_hand():
    x = torch.zeros((4, 16))
    x[0, :8] = torch.tensor([127, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, -127])  # scale 1: ties to the even code
    x[1, :4] = torch.tensor([2.0, 1.0, -1.0, 0.0])                          # half of the largest: 63.5 to 64
    x[2, 3] = float("inf")
    codes, scales = R.quantize(x)
    assert codes[0, :8].tolist() == [127, 0, 2, 2, 0, -2, 126, -127] and codes[1, :4].tolist() == [127, 64, -64, 0]
    assert scales[0] == 1 and scales[1] == np.float32(2 / 127) and np.isnan(scales[2]) and scales[3] == 0
    assert not codes[2:].any()


def test_reference_norm_by_hand():
    x, r, w = torch.full((1, 16), 1.0), torch.full((1, 16), 2.0), torch.ones(16)
    w[0] = 0.5
    codes, scales, h = R.norm(x, w, r, 0.0)  # h = 3, u = 3 (1.5), rms 3
    assert (h == 3).all() and codes[0, :2].tolist() == [64, 127] and scales[0] == pytest.approx(1 / 127, rel=1e-15)


def test_reference_gradient_is_that_of_the_loss():
    rng = np.random.default_rng(1)
    logits, ids = rng.standard_normal((7, 5)), rng.integers(-1, 5, (7, 3))
    ids[2] = -1
    _, counts, gradient, _, _ = R.balance(logits, ids, 0.3)
    g, step = gradient(2.0), 1e-5
    assert counts[-1] == 6 and counts[:-1].sum() == (ids >= 0).sum()
    for t in range(7):
        for e in range(5):
            up, down = logits.copy(), logits.copy()
            up[t, e] += step
            down[t, e] -= step
            slope = 2 * (R.balance(up, ids, 0.3)[0] - R.balance(down, ids, 0.3)[0]) / (2 * step)
            assert abs(slope - g[t, e]) < 1e-9


def test_reference_loss_of_an_even_and_a_collapsed_router():
    even = np.arange(12).reshape(6, 2) % 4
    assert R.balance(np.zeros((6, 4)), even)[0] == pytest.approx(1.0)
    one = np.full((6, 4), -50.0)
    one[:, 2] = 0
    assert R.balance(one, np.full((6, 1), 2))[0] == pytest.approx(4.0)


# ---- arguments at the C ABI ----

def test_quantize_argument_errors(lib):
    def q(x=A, dtype=F16, rows=4, n=64, ld=64, codes=2 * A, scales=3 * A):
        return lib.exl3_int8_quantize(x, dtype, rows, n, ld, codes, scales, None)
    assert q(dtype=3) == q(dtype=-1) == q(rows=-1) == q(n=0, ld=0) == q(n=40) == q(n=-16) == EINVAL
    assert q(ld=63) == q(ld=68) == q(dtype=F32, ld=66) == EINVAL   # rows off 16 bytes
    assert q(x=None) == q(codes=None) == q(scales=None) == q(x=A + 8) == q(codes=2 * A + 8) == q(scales=3 * A + 2) == EINVAL
    assert q(rows=0, x=None, codes=None, scales=None) == 0
    assert q(n=(1 << 24) + 16, ld=(1 << 24) + 16) == q(rows=(1 << 40) + 1) == EUNSUPPORTED

    def d(codes=A, scales=2 * A, rows=4, n=64, out=3 * A, dtype=F16):
        return lib.exl3_int8_dequantize(codes, scales, rows, n, out, dtype, None)
    assert d(dtype=5) == d(rows=-1) == d(n=24) == d(codes=None) == d(scales=None) == d(out=None) == EINVAL
    assert d(codes=A + 8) == d(scales=2 * A + 1) == d(out=3 * A + 8) == EINVAL
    assert d(rows=0, codes=None, scales=None, out=None) == 0
    assert d(rows=1 << 40) == d(rows=1 << 34) == EUNSUPPORTED


def test_norm_argument_errors(lib):
    def f(x=A, dtype=BF16, rows=4, n=64, ld=64, r=2 * A, ldr=64, w=3 * A, wt=F32, eps=1e-6, codes=4 * A, scales=5 * A, added=6 * A):
        return lib.exl3_int8_rms_norm(x, dtype, rows, n, ld, r, ldr, w, wt, eps, codes, scales, added, None)
    assert f(dtype=3) == f(wt=3) == f(wt=-1) == f(rows=-1) == f(n=8) == f(n=72, ld=72) == f(ld=56) == f(ldr=56) == f(ldr=65) == EINVAL
    assert f(eps=-1e-9) == f(eps=float("nan")) == f(eps=float("inf")) == EINVAL
    assert f(r=None) == f(added=None) == EINVAL                    # one without the other
    assert f(x=None) == f(w=None) == f(codes=None) == f(scales=None) == EINVAL
    assert f(x=A + 8) == f(r=2 * A + 8) == f(w=3 * A + 8) == f(codes=4 * A + 8) == f(scales=5 * A + 2) == f(added=6 * A + 8) == EINVAL
    assert f(rows=0, x=None, w=None, codes=None, scales=None) == 0
    assert f(n=(1 << 24) + 16, ld=(1 << 24) + 16, ldr=(1 << 24) + 16) == f(rows=(1 << 40) + 1) == EUNSUPPORTED


def test_product_argument_errors(lib):
    def m(xc=A, xs=2 * A, rows=4, at=None, groups=1, c=3 * A, s=4 * A, n_in=64, n_out=5, y=5 * A, dtype=BF16):
        return lib.exl3_int8_matmul(xc, xs, rows, at, groups, c, s, n_in, n_out, y, dtype, None)

    def f(x=A, dtype=BF16, rows=4, ld=64, at=None, groups=1, c=3 * A, s=4 * A, n_in=64, n_out=5, y=5 * A, ws=6 * A, wsb=1 << 40):
        return lib.exl3_int8_linear(x, dtype, rows, ld, at, groups, c, s, n_in, n_out, y, ws, wsb, None)
    for g in (m, f):
        assert g(dtype=3) == g(rows=-1) == g(n_in=24) == g(n_in=0) == g(n_out=0) == g(groups=0) == g(groups=2) == EINVAL
        assert g(c=None) == g(s=None) == g(y=None) == EINVAL
        assert g(c=3 * A + 8) == g(s=4 * A + 2) == g(y=5 * A + 8) == g(at=7 * A + 2) == EINVAL
        assert g(groups=4097, at=7 * A) == g(rows=(1 << 23) + 1) == g(n_out=(1 << 24) + 1) == EUNSUPPORTED
        assert g(rows=1 << 23, n_out=1 << 14) == EUNSUPPORTED            # 2^37 outputs
        assert g(rows=0, c=None, s=None, y=None) == 0
    assert m(n_in=1 << 17) == f(n_in=1 << 17, ld=1 << 17) == EUNSUPPORTED  # a sum might pass 32 bits
    assert m(xc=None) == m(xs=None) == m(xc=A + 1) == m(xs=2 * A + 1) == EINVAL
    assert f(x=None) == f(x=A + 2) == f(ld=48) == f(ld=65) == f(ws=6 * A + 8) == EINVAL
    assert f(rows=200, ws=None) == f(rows=200, wsb=100) == EWORKSPACE
    assert f(rows=2000, at=7 * A, groups=3, ws=None) == EWORKSPACE


def test_workspace_sizes():
    assert ex.int8_workspace_bytes(0, 64) == 0
    assert ex.int8_workspace_bytes(333, 2064) >= 333 * 2064 + 333 * 4
    for bad in ((-1, 64, 1), (1, 0, 1), (1, 40, 1), (1, 64, 0), (1 << 31, 64, 1), (1, 64, -1 << 33)):
        with pytest.raises(ex.Exl3Error):
            ex.int8_workspace_bytes(*bad)


def test_balance_argument_errors(lib):
    def f(x=A, dtype=F32, ids=2 * A, nb=4, tokens=4, k=2, e=10, co=1.0, loss=3 * A, counts=4 * A, ws=5 * A, wsb=1 << 40):
        return lib.exl3_moe_balance_loss(x, dtype, ids, nb, tokens, k, e, co, loss, counts, ws, wsb, None)

    def b(x=A, dtype=F32, ids=2 * A, nb=4, tokens=4, k=2, e=10, co=1.0, d=3 * A, counts=4 * A, out=5 * A):
        return lib.exl3_moe_balance_loss_backward(d, x, dtype, ids, nb, tokens, k, e, counts, co, out, None)
    for g in (f, b):
        assert g(dtype=3) == g(nb=2) == g(tokens=-1) == g(k=0) == g(e=0) == g(e=1025) == EINVAL
        assert g(co=float("nan")) == g(co=float("inf")) == EINVAL
        assert g(x=None) == g(ids=None) == g(counts=None) == g(x=A + 8) == g(ids=2 * A + 4) == g(counts=4 * A + 4) == EINVAL
        assert g(tokens=1 << 24) == g(tokens=1 << 20, k=1 << 11) == EUNSUPPORTED
    assert f(loss=None) == f(loss=3 * A + 2) == f(ws=5 * A + 8) == EINVAL
    assert f(tokens=100000, ws=None) == f(tokens=100000, wsb=64) == EWORKSPACE
    assert b(d=None) == b(d=3 * A + 2) == b(out=None) == b(out=5 * A + 8) == EINVAL
    assert b(tokens=0, x=None, ids=None, d=None, counts=None, out=None) == 0
    assert lib.exl3_moe_balance_workspace_bytes(64, 8) == 0 and lib.exl3_moe_balance_workspace_bytes(1 << 20, 8) > 0
    for bad in ((-1, 8), (8, 0), (8, 1025)):
        assert lib.exl3_moe_balance_workspace_bytes(*bad) == EINVAL


# ---- results that share bytes with an argument, wherever the two begin ----

def touching(at, nbytes, mine):
    """Addresses, 16 apart, of `mine` bytes that share a byte with `nbytes` bytes at `at`."""
    last = (nbytes - 1) // 16 * 16
    return [at + last, at + last // 32 * 16, at, at - (mine - 1) // 16 * 16]


def refuse(call, results, arguments):
    """Each result over each argument and each other result; both given as {name: (address, bytes)}."""
    for name, (_, mine) in results.items():
        for other, (at, nbytes) in {**arguments, **results}.items():
            if other == name:
                continue
            for where in touching(at, nbytes, mine):
                assert call(**{name: where}) == EINVAL, (name, other, where)


def test_results_that_touch_arguments(lib):
    rows, n, n_out, groups = 40, 64, 48, 3
    x, codes, scales = rows * n * 4, rows * n, rows * 4

    def quantize(c=4 * A, s=8 * A, ld=n):
        return lib.exl3_int8_quantize(A, F32, rows, n, ld, c, s, None)
    refuse(quantize, {"c": (4 * A, codes), "s": (8 * A, scales)}, {"x": (A, x)})
    assert quantize(ld=2 * n, c=A + 39 * 2 * n * 4) == EINVAL and quantize(ld=2 * n, c=A + 5 * 2 * n * 4 - 16) == EINVAL

    def dequantize(o=8 * A):
        return lib.exl3_int8_dequantize(A, 4 * A, rows, n, o, F32, None)
    refuse(dequantize, {"o": (8 * A, x)}, {"c": (A, codes), "s": (4 * A, scales)})

    def norm(c=4 * A, s=5 * A, h=6 * A, r=2 * A, ldr=n):
        return lib.exl3_int8_rms_norm(A, F32, rows, n, n, r, ldr, 3 * A, F16, 0.0, c, s, h, None)
    refuse(norm, {"c": (4 * A, codes), "s": (5 * A, scales), "h": (6 * A, x)}, {"x": (A, x), "r": (2 * A, x), "w": (3 * A, 2 * n)})
    assert norm(h=2 * A + 64, ldr=2 * n) == EINVAL

    y, wc, ws = rows * n_out * 4, groups * n_out * n, groups * n_out * 4

    def matmul(y=7 * A):
        return lib.exl3_int8_matmul(A, 2 * A, rows, 3 * A, groups, 4 * A, 5 * A, n, n_out, y, F32, None)
    refuse(matmul, {"y": (7 * A, y)}, {"xc": (A, codes), "xs": (2 * A, scales), "at": (3 * A, 4 * groups + 4), "wc": (4 * A, wc), "ws": (5 * A, ws)})

    many = 400
    need = lib.exl3_int8_workspace_bytes(many, groups, n)
    assert need > 0

    def linear(y=7 * A, w=8 * A):
        return lib.exl3_int8_linear(A, F32, many, n, 3 * A, groups, 4 * A, 5 * A, n, n_out, y, w, 1 << 30, None)
    refuse(linear, {"y": (7 * A, many * n_out * 4), "w": (8 * A, need)},
           {"x": (A, many * n * 4), "at": (3 * A, 4 * groups + 4), "wc": (4 * A, wc), "ws": (5 * A, ws)})


def test_balance_results_that_touch_arguments(lib):
    tokens, k, e = 3000, 2, 20
    need = lib.exl3_moe_balance_workspace_bytes(tokens, e)
    assert need > 0
    logits, ids, counts = tokens * e * 4, tokens * k * 8, 4 * e + 4

    def loss(l=3 * A, c=4 * A, w=5 * A):
        return lib.exl3_moe_balance_loss(A, F32, 2 * A, 8, tokens, k, e, 1.0, l, c, w, 1 << 30, None)
    refuse(loss, {"l": (3 * A, 4), "c": (4 * A, counts), "w": (5 * A, need)}, {"x": (A, logits), "ids": (2 * A, ids)})

    def backward(o=5 * A):
        return lib.exl3_moe_balance_loss_backward(3 * A, A, F32, 2 * A, 8, tokens, k, e, 4 * A, 1.0, o, None)
    refuse(backward, {"o": (5 * A, logits)}, {"x": (A, logits), "ids": (2 * A, ids), "d": (3 * A, 4), "c": (4 * A, counts)})


# ---- the binding ----

def test_int8_binding_rejects_bad_tensors():
    x, w = torch.zeros((3, 64), dtype=torch.bfloat16), torch.ones(64)
    c, s = torch.zeros((5, 64), dtype=torch.int8), torch.zeros(5)
    at = torch.zeros(3, dtype=torch.int32)
    bad = [
        (lambda: ex.int8_quantize(x.double()), "x: dtype"),
        (lambda: ex.int8_quantize([1.0]), "x: expected a torch tensor"),
        (lambda: ex.int8_quantize(x[0]), "x: expected two dimensions"),
        (lambda: ex.int8_quantize(x[:, :40]), "x: 40 columns"),
        (lambda: ex.int8_quantize(torch.zeros((64, 64), dtype=torch.bfloat16).t()[:, ::2]), "x: the values of a row"),
        (lambda: ex.int8_quantize(torch.zeros((3, 68), dtype=torch.bfloat16)[:, :64]), "x: rows must start"),
        (lambda: ex.int8_quantize(x, codes=c), "codes: shape"),
        (lambda: ex.int8_quantize(x, scales=s[:3].double()), "scales: dtype"),
        (lambda: ex.int8_quantize(x), "x: must be on a GPU"),
        (lambda: ex.int8_dequantize(c, s[:4]), "scales: shape"),
        (lambda: ex.int8_dequantize(c.view(torch.uint8), s), "codes: dtype"),
        (lambda: ex.int8_dequantize(c[:, :24], s), "codes: 24 columns"),
        (lambda: ex.int8_dequantize(c, s, torch.float64), "dtype: dtype"),
        (lambda: ex.int8_dequantize(c, s), "codes: must be on a GPU"),
        (lambda: ex.int8_rms_norm(x, w[:32]), "weight: shape"),
        (lambda: ex.int8_rms_norm(x, w.double()), "weight: dtype"),
        (lambda: ex.int8_rms_norm(x, w, x[:2]), "residual: shape"),
        (lambda: ex.int8_rms_norm(x, w, x.half()), "residual: dtype"),
        (lambda: ex.int8_rms_norm(x, w, x, eps=-1.0), "eps"),
        (lambda: ex.int8_rms_norm(x, w, x, eps=float("nan")), "eps"),
        (lambda: ex.int8_rms_norm(x, w, added=x.clone()), "added: given without"),
        (lambda: ex.int8_rms_norm(x, w, x, added=x.float()), "added: dtype"),
        (lambda: ex.int8_rms_norm(x, w, x), "x: must be on a GPU"),
        (lambda: ex.int8_linear(x, c[:, :16], s), "codes: shape"),
        (lambda: ex.int8_linear(x, c.int(), s), "codes: dtype"),
        (lambda: ex.int8_linear(x, c, s, offsets=at), "codes: expected"),
        (lambda: ex.int8_linear(x, c[None], s[None], offsets=at), "offsets: shape"),
        (lambda: ex.int8_linear(x, c[None], s[None], offsets=at[:2].long()), "offsets: dtype"),
        (lambda: ex.int8_linear(x, c[None], s, offsets=at[:2]), "scales: shape"),
        (lambda: ex.int8_linear(x, c, s, y=torch.zeros((3, 5))), "y: dtype"),
        (lambda: ex.int8_linear(x, c, s), "x: must be on a GPU"),
        (lambda: ex.int8_matmul(c, s, c, s[:4]), "scales: shape"),
        (lambda: ex.int8_matmul(c, s[:3], c, s), "x_scales: shape"),
        (lambda: ex.int8_matmul(c[:, 16:], s, c[:, 16:], s), "x_codes: must be contiguous"),
        (lambda: ex.int8_matmul(c, s, c, s, torch.int8), "dtype: dtype"),
        (lambda: ex.int8_matmul(c, s, c, s), "x_codes: must be on a GPU"),
    ]
    for f, match in bad:
        with pytest.raises(ex.Exl3Error, match=match):
            f()


def test_balance_binding_rejects_bad_tensors():
    x, ids, d, c = torch.zeros((3, 8)), torch.zeros((3, 2), dtype=torch.int32), torch.ones(()), torch.zeros(9, dtype=torch.int32)
    bad = [
        (lambda f: f(x.double(), ids), "logits: dtype"), (lambda f: f(x[:2], ids), "logits: shape"), (lambda f: f(x[0], ids), "logits: expected"),
        (lambda f: f(torch.zeros((3, 1025)), ids), "logits: 1025 experts"), (lambda f: f(torch.zeros((3, 16))[:, :8], ids), "logits: must be contiguous"),
        (lambda f: f(x, ids[0]), "expert_ids: expected"), (lambda f: f(x, ids[:, :0]), "expert_ids: expected"), (lambda f: f(x, ids.short()), "expert_ids: dtype"),
        (lambda f: f(x, ids, float("inf")), "coefficient"), (lambda f: f(x, ids, float("nan")), "coefficient"), (lambda f: f(x, ids), "logits: must be on a GPU")]
    for f, match in bad:
        with pytest.raises(ex.Exl3Error, match=match):
            f(ex.moe_balance_loss)
        with pytest.raises(ex.Exl3Error, match=match):
            f(lambda x, i, co=1.0: ex.moe_balance_loss_backward(d, x, i, c, co))
    for f, match in [(lambda: ex.moe_balance_loss(x, ids, loss=torch.zeros(1)), "loss: shape"), (lambda: ex.moe_balance_loss(x, ids, counts=c[:8]), "counts: shape"),
                     (lambda: ex.moe_balance_loss_backward(d.double(), x, ids, c), "dloss: dtype"), (lambda: ex.moe_balance_loss_backward(1.0, x, ids, c), "dloss: expected"),
                     (lambda: ex.moe_balance_loss_backward(d, x, ids, c.long()), "counts: dtype"), (lambda: ex.moe_balance_loss_backward(d, x, ids, c, dlogits=x.half()), "dlogits: dtype")]:
        with pytest.raises(ex.Exl3Error, match=match):
            f()


def differentiable_calls():
    """(call of its floating tensors, those tensors), on the CPU: past the other checks the next refusal is that of the device."""
    c, s, ids, n = torch.zeros((5, 64), dtype=torch.int8), torch.zeros(5), torch.zeros((3, 2), dtype=torch.int32), torch.zeros(9, dtype=torch.int32)
    x, w, y, logits = torch.zeros((3, 64)), torch.ones(64), torch.zeros((3, 5)), torch.zeros((3, 8))
    return {
        "int8_rms_norm": (lambda x, w, r, h: ex.int8_rms_norm(x, w, r, added=h), (x, w, x.clone(), x.clone())),
        "int8_linear": (lambda x, s, y: ex.int8_linear(x, c, s, y=y), (x, s, y)),
        "int8_matmul": (lambda xs, s, y: ex.int8_matmul(c[:3], xs, c, s, torch.float32, y=y), (s[:3].clone(), s, y)),
        "int8_dequantize": (lambda s, out: ex.int8_dequantize(c, s, torch.float32, out=out), (s, torch.zeros((5, 64)))),
        "moe_balance_loss": (lambda x, l: ex.moe_balance_loss(x, ids, loss=l), (logits, torch.zeros(()))),
        "moe_balance_loss_backward": (lambda d, x, o: ex.moe_balance_loss_backward(d, x, ids, n, dlogits=o), (torch.ones(()), logits, logits.clone())),
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


def test_quantize_takes_a_parameter():
    with pytest.raises(ex.Exl3Error, match="must be on a GPU"):
        ex.int8_quantize(torch.nn.Parameter(torch.zeros((3, 64))))


def test_binding_rejects_sizes_beyond_32_bits():
    def t(*shape, dtype=torch.int8):
        return torch.empty(shape, dtype=dtype, device="meta")
    big, f16, f32, i32 = 2 ** 32 + 32, torch.float16, torch.float32, torch.int32
    bad = [
        lambda: ex.int8_quantize(t(1, big, dtype=f16)),
        lambda: ex.int8_dequantize(t(1, big), t(1, dtype=f32)),
        lambda: ex.int8_rms_norm(t(1, big, dtype=f16), t(big, dtype=f32)),
        lambda: ex.int8_linear(t(big, 64, dtype=f16), t(5, 64), t(5, dtype=f32)),
        lambda: ex.int8_linear(t(3, big, dtype=f16), t(5, big), t(5, dtype=f32)),
        lambda: ex.int8_linear(t(3, 64, dtype=f16), t(big, 64), t(big, dtype=f32)),
        lambda: ex.int8_linear(t(3, 64, dtype=f16), t(big, 5, 64), t(big, 5, dtype=f32), offsets=t(big + 1, dtype=i32)),
        lambda: ex.int8_matmul(t(big, 64), t(big, dtype=f32), t(5, 64), t(5, dtype=f32)),
        lambda: ex.int8_matmul(t(3, big), t(3, dtype=f32), t(5, big), t(5, dtype=f32)),
        lambda: ex.int8_workspace_bytes(64, big),
        lambda: ex.moe_balance_loss(t(big // 2, 8, dtype=f16), t(big // 2, 2, dtype=i32)),
        lambda: ex.moe_balance_loss(t(3, big, dtype=f16), t(3, 2, dtype=i32)),
    ]
    for f in bad:
        with pytest.raises(ex.Exl3Error, match="below 2.31"):
            f()
