"""The gradient of the balance loss where experts have as many slots, or nearly: what is left is small beside the shares themselves."""
import numpy as np
import pytest
import torch

import _int8_ref as R

pytestmark = pytest.mark.gpu
DTYPES = R.DTYPES
# tokens, slots, experts: every number of lanes a token, all experts chosen by each token among them
SIZES = [(6, 2, 2), (3, 7, 7), (9, 3, 3), (64, 8, 8), (60, 5, 12), (40, 4, 20), (4000, 8, 64), (1300, 2, 65), (640, 8, 128), (771, 2, 257), (1026, 3, 513), (2048, 4, 1024),
         (30000, 2, 4)]


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import decode_gemm_exl3_amd as ex
    ex.load()
    return ex


def even_ids(tokens, slots, experts):
    assert tokens * slots % experts == 0
    return (np.arange(tokens * slots) % experts).astype(np.int32).reshape(tokens, slots)


def backward(ex, logits, ids, dloss):
    x, i = logits.cuda(), torch.from_numpy(ids).cuda()
    _, counts = ex.moe_balance_loss(x, i, 0.5)
    return ex.moe_balance_loss_backward(torch.tensor(dloss, device="cuda"), x, i, counts, 0.5), counts


def random_logits(rng, tokens, experts, dtype):
    return torch.from_numpy(2 * rng.standard_normal((tokens, experts))).to(DTYPES[dtype])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens, slots, experts", SIZES)
def test_equal_counts_have_no_gradient(ex, tokens, slots, experts, dtype):
    """Whatever the logits: probabilities sum to one, so that equal shares cancel, all of them."""
    logits = random_logits(np.random.default_rng([61, tokens, experts]), tokens, experts, dtype)
    got, counts = backward(ex, logits, even_ids(tokens, slots, experts), 2.0 ** 16)
    assert len(set(counts[:-1].tolist())) == 1 and int(counts[-1]) == tokens
    assert not got.any(), got.abs().max()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens, slots, experts", SIZES)
def test_nearly_equal_counts(ex, tokens, slots, experts, dtype):
    """One slot goes to another expert.  With s less their mean, which changes nothing, s_e - sum_f p_f s_f is off by steps of
    the largest of them: a probability's error (its distance to the largest logit and the sum of all `experts`), the products' and sums', a few more."""
    rng = np.random.default_rng([62, tokens, experts])
    logits, ids = random_logits(rng, tokens, experts, dtype), even_ids(tokens, slots, experts)
    ids[tokens // 2, 0] = (ids[tokens // 2, 0] + 1) % experts
    wide = logits.double().numpy()
    dloss = 2.0 ** 16 if dtype != "fp16" else 2.0 ** 20
    got, counts = backward(ex, logits, ids, dloss)
    _, want, gradient, p, s = R.balance(wide, ids, 0.5)
    assert np.array_equal(counts.cpu().numpy(), want)
    g = gradient(dloss)
    centred, u = s - s.mean(), 2.0 ** -24
    below = float((wide.max(1, keepdims=True) - wide).max())
    of_p = (2 * (1.3 * below + 3) + experts + 4) * u
    tol = dloss * 0.5 * experts / tokens * p * (2 * of_p + (experts + 8) * u) * 2 * np.abs(centred).max() * 1.01
    info = torch.finfo(DTYPES[dtype])
    tol = tol + info.eps / 2 * (np.abs(g) + tol) + info.smallest_normal * info.eps / 2
    off = np.abs(got.cpu().double().numpy() - g) - tol
    assert (off <= 0).all(), (off.max(), np.abs(g).max())
