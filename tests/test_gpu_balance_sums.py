"""The balance loss's sums over tokens: no token lost or taken twice, and as near as the additions that are made allow."""
import numpy as np
import pytest
import torch

import _int8_ref as R

pytestmark = pytest.mark.gpu
DTYPES = R.DTYPES
# one workgroup, several and 256 of them; one lane a token to 64, with one to four pieces; a last round that is partly empty
SIZES = [(1, 2), (64, 3), (1025, 7), (333, 49), (70001, 2), (300000, 7), (9000, 64), (20011, 48), (4097, 128), (33000, 256), (5000, 384), (3001, 513),
         (1100, 1024), (70001, 65)]


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import decode_gemm_exl3_amd as ex
    ex.load()
    return ex


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens, experts", SIZES)
def test_every_token_once(ex, tokens, experts, dtype):
    """A token has all its probability on expert 1 or on expert 0, and all slots are expert 1's: the loss is experts times
    the share of the former tokens.  Their sums are of ones and exact, so that nothing but the result is rounded."""
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    slots = 2
    sets = {"last": [tokens - 1], "first": [0], "last round": range(max(0, tokens - 200), tokens, 3), "none": []}
    random = (torch.rand(tokens, generator=gen, device="cuda") < 0.3).nonzero().flatten()
    dropped = torch.rand(tokens, generator=gen, device="cuda") < 0.2
    for name, which in [*sets.items(), ("random", random)]:
        logits = torch.full((tokens, experts), -float("inf"), dtype=DTYPES[dtype], device="cuda")
        logits[:, 0] = 1.5
        which = torch.as_tensor(which, dtype=torch.int64, device="cuda")
        logits[which, 0], logits[which, 1] = -float("inf"), -2.25
        for drop in (None, dropped):
            ids = torch.ones((tokens, slots), dtype=torch.int32, device="cuda")
            if drop is not None:
                ids[drop] = -1
            live = tokens if drop is None else tokens - int(drop.sum())
            hits = which.numel() if drop is None else int((~drop[which]).sum())
            loss, counts = ex.moe_balance_loss(logits, ids, 0.25)
            want = [0] * experts + [live]
            want[1] = slots * live
            assert counts.tolist() == want, name
            ref = 0.25 * experts * hits / max(live, 1)
            assert abs(float(loss) - ref) <= 2.0 ** -24 * 1.0001 * ref, (name, float(loss), ref)


def additions(tokens, experts, size):
    """Of fp32 numbers one after the other: over a token's logits, over a lane's tokens and all joins behind them (sum_kernel, loss_kernel)."""
    pieces = -(-experts * size // 16)
    lanes = min(64, 1 << (pieces - 1).bit_length())
    held = -(-pieces // lanes) * (16 // size)
    held = 4 * (16 // size) if held > 2 * (16 // size) else held
    blocks = min(256, max(1, -(-tokens * experts // 16384)))
    each = 64 // lanes
    log = (lanes.bit_length() - 1, each.bit_length() - 1)
    return held + log[0], -(-tokens // (blocks * 16 * each)) + log[1] + 16 + (32 if blocks > 1 else 0)


def bound(below, tokens, experts, size):
    """Relative bound on the loss, in steps of u = 2^-24: an exponential is off by its distance to the largest logit (the
    difference, or its product with 1 / ln 2, which is off by 0.22 u itself, rounded: 1.3 u of it) and by the instruction's 2 u
    and the correction's u; a probability by its own exponential's error, the sum's (its terms' and its additions') and 2 u of the
    inverse; then the additions over tokens."""
    of_token, over_tokens = additions(tokens, experts, size)
    return (2 * (1.3 * below + 3) + of_token + 2 + over_tokens) * 2.0 ** -24 * 1.01


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens, experts", SIZES)
def test_loss_within_its_additions(ex, tokens, experts, dtype):
    rng = np.random.default_rng([41, tokens, experts])
    logits = torch.from_numpy(1.5 * rng.standard_normal((tokens, experts)) + rng.standard_normal(experts)).to(DTYPES[dtype])
    ids = rng.integers(-1, experts + 1, (tokens, 2)).astype(np.int32)
    wide = logits.double().numpy()
    ref, counts, _, _, _ = R.balance(wide, ids, 0.5)
    loss, got = ex.moe_balance_loss(logits.cuda(), torch.from_numpy(ids).cuda(), 0.5)
    assert np.array_equal(got.cpu().numpy(), counts)
    below = float((wide.max(1, keepdims=True) - wide).max())
    off = bound(below, tokens, experts, logits.element_size())
    assert abs(float(loss) - ref) <= (off + 2.0 ** -24) * ref, (float(loss), ref, (float(loss) - ref) / ref, off)


def test_a_lost_token_is_more_than_the_bound():
    """Else the test above would not see it: in up to 33000 tokens."""
    for tokens, experts in SIZES:
        for size in (2, 4):
            if tokens <= 33000:  # (beyond, test_every_token_once does)
                assert bound(20.0, tokens, experts, size) < 0.5 / tokens, (tokens, experts)


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_token_of_many_slots(ex, dtype):
    """More slots than lanes by far, in one token and in two; the last ones count too."""
    for tokens, experts in ((1, 1000), (1, 3), (2, 40)):
        slots = (1 << 16) + 37
        ids = torch.full((tokens, slots), -1, dtype=torch.int32, device="cuda")
        ids[:, -1] = experts - 1
        ids[0, 3::5] = 0
        loss, counts = ex.moe_balance_loss(torch.zeros((tokens, experts), dtype=DTYPES[dtype], device="cuda"), ids)
        want = torch.bincount(ids[ids >= 0].long(), minlength=experts).tolist() + [tokens]
        assert counts.tolist() == want
        # the probabilities are all 1 / experts: an error of the inverse and of the sums over experts and counts in fp32 and fp64
        ref = sum(want[:-1]) / (tokens * slots)
        assert abs(float(loss) - ref) <= 16 * 2.0 ** -24 * ref
