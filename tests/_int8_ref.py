"""8-bit rows, their norm and products, and the balance loss from their definitions, on the CPU."""
import numpy as np
import torch

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def codes_of(u):
    """Codes int8 [rows, n] and the largest magnitudes (float64) of fp32 values u; a row that is not finite: 0 and NaN.
    127 u / A in 64 bits is exact enough: 127 u has at most 31 bits, and a quotient that is no tie is at
    least 2^-25 of its size away from one."""
    u = u.astype(np.float64)
    bad = ~np.isfinite(u).all(1, keepdims=True)
    a = np.where(bad, 0.0, u)
    largest = np.abs(a).max(1, keepdims=True)
    q = np.rint(127 * a / np.where(largest == 0, 1, largest))
    return q.astype(np.int8), np.where(bad, np.nan, largest)[:, 0]


def quantize(x):
    """x: torch [rows, n] on any device."""
    codes, largest = codes_of(x.detach().cpu().float().numpy())
    return codes, (largest / 127).astype(np.float32)


def norm(x, weight, residual, eps):
    """codes, scales (float64, not rounded), h; x, weight, residual: torch tensors."""
    x, weight = x.detach().cpu(), weight.detach().cpu()
    h = x if residual is None else (x.float() + residual.detach().cpu().float()).to(x.dtype)
    with np.errstate(over="ignore", invalid="ignore"):
        codes, largest = codes_of(h.float().numpy() * weight.float().numpy())
        mean = (h.double().numpy() ** 2).mean(1)
        scales = np.where(largest == 0, 0.0, largest / (127 * np.sqrt(np.where(largest == 0, 1.0, mean) + eps)))
    return codes, scales, h


def product(xc, xs, wc, ws, dtype):
    """What the definition says, bit for bit: whole sums, converted to fp32, times the row's scale, times the output's."""
    acc = xc.astype(np.float64) @ wc.astype(np.float64).T  # below 2^53: exact
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        y = acc.astype(np.float32) * xs[:, None] * ws[None, :]
    return torch.from_numpy(y).to(dtype)


def weight(rng, *shape):
    """A random weight: codes [..., n_out, n] over the whole range and scales [..., n_out]."""
    return rng.integers(-128, 128, shape, dtype=np.int8), (0.01 * np.exp2(rng.uniform(-3, 3, shape[:-1]))).astype(np.float32)


def rows(rng, m, n, dtype):
    """Activations whose rows and columns differ in size, as a CPU tensor."""
    x = rng.standard_normal((m, n)) * np.exp2(rng.integers(-3, 4, (m, 1)))
    x[:, rng.random(n) < 0.03] *= 16
    return torch.from_numpy(x).to(dtype)


def equal(a, b):
    """Bit for bit, any NaN equal to any other."""
    a, b = (t.detach().cpu() for t in (a, b))
    return a.dtype == b.dtype and a.shape == b.shape and bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


# ---- balance loss ----

def balance(logits, ids, coefficient=1.0):
    """loss, counts and a gradient function dloss -> dlogits, in 64 bits (logits: float64 NumPy)."""
    tokens, experts = logits.shape
    kept = (ids >= 0) & (ids < experts)
    live = kept.any(1)
    c = np.bincount(ids[kept].astype(np.int64), minlength=experts)
    v = int(live.sum())
    with np.errstate(invalid="ignore"):
        top = logits.max(1, keepdims=True, initial=-np.inf)
        e = np.exp(logits - np.where(top == -np.inf, 0, top))
        total = e.sum(1, keepdims=True)
        p = np.where(live[:, None], np.where(total == 0, 0.0, e / np.where(total == 0, 1, total)), 0.0)
    s = c / (max(v, 1) * ids.shape[1])
    loss = coefficient * experts * (s * p.sum(0)).sum() / max(v, 1)

    def gradient(dloss):
        return dloss * coefficient * experts / max(v, 1) * p * (s - (p * s).sum(1, keepdims=True))
    return loss, np.append(c, v).astype(np.int32), gradient, p, s


def balance_tolerances(logits, ids, p, s, scale, dtype):
    """Bounds on the error of the loss and of each gradient, from the steps in fp32 (u = 2^-24, half a step).

    A probability: the difference to the largest logit is rounded (its size times u; below -120 exp is 0), exp is good to one step (2 u), the sum of
    `experts` terms adds at most `experts` u and each term's own error, the inverse and the product 2 u.
    The sum over tokens: a chain of at most tokens / 4 + 280 additions (four waves; 256 workgroups and the joins).
    The gradient: `along` is a sum of `experts` products; then a difference, two products and the conversion of s and the factor.
    """
    u, (tokens, experts) = 2.0 ** -24, logits.shape
    live = ((ids >= 0) & (ids < experts)).any(1)
    finite = np.where(np.isfinite(logits), logits, -np.inf)[live]
    below = finite.max(1, keepdims=True, initial=-1e300) - finite
    spread = below[below < 120].max(initial=0.0)
    dp = (2 * spread + 4 + experts + 3) * u
    loss = (dp + (min(tokens, tokens // 4 + 280) + 4) * u) * scale * experts * (s * p.sum(0)).sum() / max(int(live.sum()), 1)
    along = (p * s).sum(1, keepdims=True)
    factor = scale * experts / max(int(live.sum()), 1)
    grad = factor * p * ((dp + 6 * u) * np.abs(s - along) + (dp + (experts + 4) * u) * along + 2 * u * s)
    return 1.01 * loss, 1.01 * grad
