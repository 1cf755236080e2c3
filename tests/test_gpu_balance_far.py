"""Probabilities of logits far below their token's largest."""
import numpy as np
import pytest
import torch

import _int8_ref as R

pytestmark = pytest.mark.gpu
DTYPES = R.DTYPES


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import decode_gemm_exl3_amd as ex
    ex.load()
    return ex


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("top", [0.0, 3.5])
@pytest.mark.parametrize("experts", [62, 250])
def test_logits_80_to_110_below(ex, dtype, top, experts):
    """Each probability as the gradient shows it: dloss is 2^100, so that 2^-149 of it is far above the types' smallest values.
    Down to 2^-126 of the largest a probability has its relative error; below it counts as 0, which is off by 2^-126 at most."""
    tokens = 40
    rng = np.random.default_rng([51, experts])
    below = rng.integers(160, 221, (tokens, experts)) / 2.0  # exact in all types
    below[:, 0] = 0
    below[:, 1] = rng.integers(0, 8, tokens) / 2.0
    logits = torch.from_numpy(top - below).to(DTYPES[dtype])
    wide = logits.double().numpy()
    assert top != 0 or (wide == -below).all()
    ids = rng.integers(0, 2, (tokens, 1)).astype(np.int32)
    x, i = logits.cuda(), torch.from_numpy(ids).cuda()
    loss, counts = ex.moe_balance_loss(x, i)
    dloss, scale = (2.0 ** 100, 2.0 ** 100) if dtype != "fp16" else (2.0 ** 110, 2.0 ** 110)
    got = ex.moe_balance_loss_backward(torch.tensor(dloss, device="cuda"), x, i, counts).cpu().double().numpy()
    ref, _, gradient, p, s = R.balance(wide, ids)
    _, tol = R.balance_tolerances(wide, ids, p, s, scale, DTYPES[dtype])
    g = gradient(dloss)
    along = (p * s).sum(1, keepdims=True)
    tol = tol + 1.01 * scale * experts / tokens * np.abs(s - along) * 2.0 ** -126
    eps, info = torch.finfo(DTYPES[dtype]).eps / 2, torch.finfo(DTYPES[dtype])
    shown = np.abs(g) + tol < info.max  # (fp16's largest is 65504)
    assert shown[:, 2:].all()
    tol = tol + eps * (np.abs(g) + tol) + info.smallest_normal * info.eps / 2
    off = np.abs(got - g) - tol
    assert (off[shown] <= 0).all(), (off[shown].max(),)
    near = (p / p.max(1, keepdims=True) > 2.0 ** -125.5) & shown
    near[:, :2] = False
    assert near.any() and (np.abs(got - g)[near] <= (tol - 1.01 * scale * experts / tokens * np.abs(s - along) * 2.0 ** -126 * (1 + eps))[near]).all()
    assert not got[:, 2:][below[:, 2:] > 87.4].any()  # as the header says
