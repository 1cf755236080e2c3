"""MXFP4 and expert routing from their definitions, in float64 on the CPU."""
import numpy as np
import torch

VALUES = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def quantize(x):
    """x: torch [rows, n] on any device; codes and scales as NumPy uint8."""
    v = x.detach().cpu().double().numpy()
    rows, n = v.shape
    v = v.reshape(rows, n // 32, 32)
    bad = ~np.isfinite(v).all(-1)
    a = np.where(bad[..., None], 0.0, np.abs(v))
    amax = a.max(-1)
    exponent = np.frexp(amax)[1] - 1
    shared = np.where(amax == 0, -127, np.maximum(exponent - 2, -127))
    q = np.ldexp(a, -shared[..., None])
    code = np.zeros(q.shape, np.uint8)
    for k in range(7):  # the border between codes k and k + 1; a tie goes to the even one
        middle = (VALUES[k] + VALUES[k + 1]) / 2
        code[(q >= middle) if k % 2 else (q > middle)] = k + 1
    code += np.where(np.signbit(v), 8, 0).astype(np.uint8)
    code[bad] = 0
    scales = np.where(bad, 255, shared + 127).astype(np.uint8)
    code = code.reshape(rows, n)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def dequantize(codes, scales):
    """float64 [..., n] of NumPy or torch codes and scales."""
    codes, scales = (t.cpu().numpy() if isinstance(t, torch.Tensor) else t for t in (codes, scales))
    code = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = VALUES[code & 7] * np.where(code & 8, -1.0, 1.0)
    power = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return v * np.repeat(power, 32, axis=-1)


def weight(rng, *shape):
    """A random weight: codes [..., n / 2] and scales [..., n / 32], values of order 1."""
    *lead, n = shape
    return (rng.integers(0, 256, (*lead, n // 2), dtype=np.uint8),
            rng.integers(122, 128, (*lead, n // 32), dtype=np.uint8))


def rows(rng, m, n, dtype, pad=0):
    """Activations whose rows and blocks differ in size, as a CPU tensor (a slice of a wider one with pad)."""
    x = rng.standard_normal((m, n + pad)) * np.exp2(rng.integers(-3, 4, (m, 1)))
    x[:, rng.random(n + pad) < 0.03] *= 16
    return torch.from_numpy(x).to(dtype)[:, :n]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def assert_product(y, x, w, dtype, what=""):
    """y against x @ w.T for float64 x [m, k] and w [n, k].  The products of two codes
    and their scales are exact; the sum over k runs in fp32: k / 128 steps of the
    matrix core, each off by at most two half steps (its own sum and the addition), and the
    sums of up to 16 waves, relative to the sum of magnitudes; then one rounding
    to the output type (a half step, or half of fp16's smallest subnormal)."""
    ref, size = x @ w.T, np.abs(x) @ np.abs(w).T
    tol = (2 * -(-x.shape[1] // 128) + 16) * 2.0 ** -24 * size
    tol = tol + half_step(dtype) * (np.abs(ref) + tol) + (2.0 ** -25 if dtype == torch.float16 else 0)
    got = y.detach().cpu().double().numpy()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert (np.isnan(got) == np.isnan(ref)).all(), (what, "NaN in other places")
    off = np.abs(got - ref) - tol
    worst = np.unravel_index(np.nanargmax(np.where(np.isnan(off), -np.inf, off)), off.shape) if off.size else None
    assert worst is None or not off[worst] > 0, (what, worst, got[worst], ref[worst], tol[worst])


def sort(ids, experts):
    """order, position, offsets of the stable sort, dropped slots last."""
    flat = np.asarray(ids).reshape(-1)
    group = np.where((flat < 0) | (flat >= experts), experts, flat)
    order = np.argsort(group, kind="stable")
    position = np.empty_like(order)
    position[order] = np.arange(order.size)
    offsets = np.searchsorted(group[order], np.arange(experts + 1))
    return order, position.reshape(np.asarray(ids).shape), offsets
