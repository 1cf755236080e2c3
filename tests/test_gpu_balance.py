"""The experts' balance loss, counts and gradient on the GPU against the definition in float64,
and a layer of experts on 8-bit weights as it is run and trained."""
import numpy as np
import pytest
import torch

import _int8_ref as R
import _mxfp4_ref as M

pytestmark = pytest.mark.gpu
DTYPES = R.DTYPES


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import decode_gemm_exl3_amd as ex
    ex.load()
    return ex


def dev(a):
    return (torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a).cuda()


def random_ids(rng, tokens, top_k, experts, dropped=0.1, dtype=np.int32):
    ids = rng.integers(0, experts, (tokens, top_k)).astype(dtype)
    ids[rng.random(ids.shape) < dropped] = -1
    ids[rng.random(ids.shape) < dropped / 2] = experts + 3
    ids[rng.random(tokens) < dropped] = -1
    return ids


def check(ex, logits, ids, coefficient=1.0, dloss=1.0):
    """logits: a CPU tensor, ids NumPy."""
    dt = logits.dtype
    x, i = logits.cuda(), dev(ids)
    loss, counts = ex.moe_balance_loss(x, i, coefficient)
    dlogits = ex.moe_balance_loss_backward(torch.tensor(dloss, device="cuda"), x, i, counts, coefficient)
    wide = logits.double().numpy()
    ref, ref_counts, gradient, p, s = R.balance(wide, ids, coefficient)
    assert loss.shape == () and loss.dtype == torch.float32 and np.array_equal(counts.cpu().numpy(), ref_counts)
    tol, _ = R.balance_tolerances(wide, ids, p, s, abs(coefficient), dt)
    assert abs(float(loss) - ref) <= tol + 2.0 ** -24 * abs(ref) + 2.0 ** -150, (float(loss), ref, tol)
    g = gradient(dloss)
    _, tol = R.balance_tolerances(wide, ids, p, s, abs(coefficient * dloss), dt)
    info = torch.finfo(dt)
    tol = tol + info.eps / 2 * (np.abs(g) + tol) + info.smallest_normal * info.eps / 2 + 2.0 ** -149
    assert dlogits.dtype == dt and dlogits.shape == logits.shape
    off = np.abs(dlogits.cpu().double().numpy() - g) - tol
    assert (off <= 0).all(), (off.max(), np.unravel_index(off.argmax(), off.shape))
    live = ((ids >= 0) & (ids < wide.shape[1])).any(1)
    assert (dlogits.cpu()[torch.from_numpy(~live)] == 0).all()
    return loss, counts, dlogits


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens, top_k, experts", [
    (1, 1, 1), (1, 8, 64), (5, 2, 8), (64, 1, 3), (67, 3, 20), (100, 3, 1024), (128, 8, 64), (129, 8, 65), (300, 70, 9), (513, 4, 16), (257, 2, 33),
    (1000, 6, 128), (40, 5, 129), (333, 8, 256), (77, 8, 257), (90, 8, 512), (61, 8, 513), (50, 8, 1000), (2000, 1, 2), (9000, 8, 64), (5000, 8, 384),
    (1100, 8, 1024), (70000, 2, 7)])
def test_sizes(ex, tokens, top_k, experts, dtype):
    rng = np.random.default_rng([1, tokens, experts])
    logits = torch.from_numpy(1.5 * rng.standard_normal((tokens, experts)) + rng.standard_normal(experts)).to(DTYPES[dtype])
    ids = random_ids(rng, tokens, top_k, experts, dtype=(np.int32, np.int64)[tokens % 2])
    check(ex, logits, ids, coefficient=0.01, dloss=65536.0 if dtype == "fp16" else 1.0)


@pytest.mark.parametrize("tokens", [3, 20000])
@pytest.mark.parametrize("experts", [6, 64, 300])
def test_an_even_router(ex, tokens, experts):
    """Equal logits and equal counts: the loss is the coefficient, the gradient zero."""
    tokens = tokens * experts // 3 if tokens == 3 else tokens // experts * experts
    ids = (np.arange(tokens * 3) % experts).astype(np.int32).reshape(tokens, 3)
    loss, counts, dlogits = check(ex, torch.full((tokens, experts), -3.25), ids, coefficient=0.5)
    assert abs(float(loss) - 0.5) < 1e-3 and len(set(counts[:-1].tolist())) == 1 and int(counts[-1]) == tokens


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens, experts", [(50, 20), (6000, 64)])
def test_padding_masks_and_rows_of_nothing(ex, tokens, experts, dtype):
    rng = np.random.default_rng([2, tokens])
    dt = DTYPES[dtype]
    logits = torch.from_numpy(rng.standard_normal((tokens, experts))).to(dt)
    ids = rng.integers(0, experts, (tokens, 2)).astype(np.int32)
    ids[3::7] = -1
    logits[3] = float("nan")                       # padding holds anything
    logits[10] = float("inf")
    logits[17] = -float("inf")
    logits[:, 5] = -float("inf")                   # an expert that is masked out
    logits[1, 6:] = torch.finfo(dt).min            # experts masked by the lowest value
    logits[2] = torch.finfo(dt).min
    logits[4] = -float("inf")                      # a token without any expert
    logits[5, 0] = torch.finfo(dt).max
    loss, counts, dlogits = check(ex, logits, ids)
    masked = torch.arange(tokens) != 2             # that token's logits are all the lowest value, the masked expert's too
    assert torch.isfinite(loss) and torch.isfinite(dlogits).all() and (dlogits[4] == 0).all() and (dlogits.cpu()[masked, 5] == 0).all()


def test_no_token_counts(ex):
    for tokens in (1, 70, 30000):
        logits, ids = torch.full((tokens, 12), float("nan")), np.full((tokens, 2), -1, np.int32)
        ids[:, 1] = 12
        loss, counts, dlogits = check(ex, logits, ids)
        assert float(loss) == 0 and not counts.any() and not dlogits.any()
    x, i = torch.empty((0, 12), device="cuda"), torch.empty((0, 2), dtype=torch.int64, device="cuda")
    loss, counts = ex.moe_balance_loss(x, i)
    assert float(loss) == 0 and counts.shape == (13,) and not counts.any()
    assert ex.moe_balance_loss_backward(loss, x, i, counts).shape == (0, 12)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_logit_shows(ex, bad):
    logits = torch.zeros((100, 10))
    logits[40, 3] = bad
    logits[40, 4:] = -float("inf")
    ids = dev(np.zeros((100, 1), np.int32))
    loss, counts = ex.moe_balance_loss(logits.cuda(), ids)
    d = ex.moe_balance_loss_backward(torch.ones((), device="cuda"), logits.cuda(), ids, counts)
    assert torch.isnan(loss) and torch.isnan(d[40]).all() and torch.isfinite(d[:40]).all() and torch.isfinite(d[41:]).all()


def test_ids_of_64_bits_are_not_cut(ex):
    ids = np.full((40, 2), 1 << 32, np.int64)  # not expert 0 of its low half
    ids[:, 1] = -(1 << 40)
    assert not ex.moe_balance_loss(torch.zeros((40, 8), device="cuda"), dev(ids))[1].any()


@pytest.mark.parametrize("tokens, experts", [(30, 12), (3000, 64)])
def test_the_same_every_time(ex, tokens, experts):
    rng = np.random.default_rng([3, tokens])
    x, ids = dev(rng.standard_normal((tokens, experts)).astype(np.float32)), dev(random_ids(rng, tokens, 4, experts))
    first = ex.moe_balance_loss(x, ids)
    for _ in range(20):
        again = ex.moe_balance_loss(x, ids)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_gradient_against_differences(ex):
    """The loss along random directions: differences of losses in fp32 are off by the losses' own
    rounding over the step, and by the third derivative (a softmax's derivatives are at most 1, and
    the loss is at most `experts` times its largest share)."""
    rng = np.random.default_rng(4)
    tokens, experts, step = 8, 6, 2.0 ** -4
    logits, ids = rng.standard_normal((tokens, experts)).astype(np.float32), rng.integers(0, experts, (tokens, 2)).astype(np.int32)
    x, i = dev(logits), dev(ids)
    loss, counts = ex.moe_balance_loss(x, i)
    d = ex.moe_balance_loss_backward(torch.ones((), device="cuda"), x, i, counts).cpu().double().numpy()
    _, _, _, p, s = R.balance(logits.astype(np.float64), ids)
    rounding = R.balance_tolerances(logits.astype(np.float64) + step, ids, p, s, 1.0, torch.float32)[0] * 1.5 + 2.0 ** -23
    for t in range(tokens):
        for e in range(experts):
            moved = []
            for sign in (1, -1):
                y = logits.copy()
                y[t, e] += sign * step
                moved.append((float(ex.moe_balance_loss(dev(y), i)[0]), y[t, e]))
            width = moved[0][1] - moved[1][1]
            slope = (moved[0][0] - moved[1][0]) / width
            # |third derivative| of sum_j s_j p_j in one logit: at most 6 times the largest share, over tokens
            third = 6 * experts * s.max() / tokens * step ** 2 / 6
            assert abs(slope - d[t, e]) <= 2 * rounding / width + third + 1e-6, (t, e, slope, d[t, e])


# ---- streams, graphs, workspaces ----

@pytest.mark.parametrize("tokens", [20, 5000])
def test_streams_and_captured_graphs(ex, tokens):
    rng = np.random.default_rng([5, tokens])
    cases = [(dev(rng.standard_normal((tokens, 48)).astype(np.float32)), dev(random_ids(rng, tokens, 3, 48))) for _ in range(4)]
    one = torch.ones((), device="cuda")

    def step(x, ids, stream=None):
        loss, counts = ex.moe_balance_loss(x, ids, 0.1, stream=stream)
        return loss, counts, ex.moe_balance_loss_backward(one, x, ids, counts, 0.1, stream=stream)
    refs = [step(*c) for c in cases]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    given = step(*cases[1], stream=side)
    with torch.cuda.stream(side):
        current = step(*cases[2])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(given, refs[1])) and all(torch.equal(a, b) for a, b in zip(current, refs[2]))
    held, graphs = [t.clone() for t in cases[0]], []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(*held)
        graphs.append((g, out))
    for i in (1, 2, 3, 0, 2):
        for t, s in zip(held, cases[i]):
            t.copy_(s)
        for g, _ in graphs:
            g.replay()
        eager = step(*cases[(i + 1) % 4])
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, refs[i]))
        assert all(torch.equal(a, b) for a, b in zip(eager, refs[(i + 1) % 4]))


def test_given_tensors_and_workspace(ex):
    rng = np.random.default_rng(6)
    tokens, experts = 4000, 40
    x, ids = dev(rng.standard_normal((tokens, experts)).astype(np.float32)), dev(random_ids(rng, tokens, 3, experts))
    loss, counts = ex.moe_balance_loss(x, ids)
    from decode_gemm_exl3_amd import moe
    need = moe._balance_workspace_bytes(tokens, experts)
    assert need > 0
    ws = torch.full((need + 64,), 0xCD, dtype=torch.uint8, device="cuda")
    losses, all_counts = torch.full((5,), 7.0, device="cuda"), torch.full((64,), 9, dtype=torch.int32, device="cuda")
    ex.moe_balance_loss(x, ids, loss=losses[3], counts=all_counts[4:45], workspace=ws[:need])
    assert torch.equal(losses[3], loss) and (losses[[0, 1, 2, 4]] == 7).all() and (ws[need:] == 0xCD).all()
    assert torch.equal(all_counts[4:45], counts) and (all_counts[:4] == 9).all() and (all_counts[45:] == 9).all()
    with pytest.raises(ex.Exl3Error, match="workspace"):
        ex.moe_balance_loss(x, ids, workspace=ws[:need - 16])


def test_many_tokens(ex):
    """2^23 tokens of 1024 experts, 2^33 logits: tokens repeat, so the loss is that of one set."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    base, tokens = 1024, 1 << 23
    x = torch.randn((base, 1024), generator=gen, device="cuda").bfloat16()
    ids = torch.randint(-100, 1024, (base, 2), generator=gen, device="cuda", dtype=torch.int32)
    loss, counts = ex.moe_balance_loss(x, ids)
    many_loss, many = ex.moe_balance_loss(x.repeat(tokens // base, 1), ids.repeat(tokens // base, 1))
    assert torch.equal(many, counts * (tokens // base))
    # chains of at most 2^23 / 256 additions (64 workgroups of four waves at least), and the joins
    assert abs(float(many_loss) - float(loss)) <= 2.0 ** -24 * (tokens // 256 + 400) * float(loss)


# ---- together ----

def silu(x):
    return x * torch.sigmoid(x)


@pytest.mark.parametrize("tokens, top_k, experts, n, hidden", [(1, 2, 8, 128, 64), (9, 2, 8, 256, 144), (300, 3, 12, 208, 176)])
def test_a_layer_of_experts_on_8_bit_weights(ex, tokens, top_k, experts, n, hidden):
    """Norm with the residual's addition, router, experts, their sum, and the balance loss with its gradient,
    each step against its definition on what the steps before it made."""
    rng = np.random.default_rng([7, tokens])
    dt = torch.bfloat16
    y, x = (R.rows(rng, tokens, n, dt).cuda() for _ in range(2))
    gain = dev(1 + 0.2 * rng.standard_normal(n)).to(dt)
    router = R.weight(rng, experts, n)
    up, down = R.weight(rng, experts, 2 * hidden, n), R.weight(rng, experts, n, hidden)
    codes, scales, x2 = ex.int8_rms_norm(y, gain, x, eps=1e-5)
    logits = ex.int8_matmul(codes, scales, dev(router[0]), dev(0.02 * router[1]), torch.float32)
    weights, ids = torch.softmax(logits, -1).topk(top_k)
    ids[tokens // 2, 0] = -1
    order, position, offsets = ex.moe_sort(ids, experts)
    normed = ex.int8_dequantize(codes, scales, dt)
    rows = ex.moe_gather(normed, position, offsets)
    h = ex.int8_linear(rows, dev(up[0]), dev(up[1]), offsets=offsets)
    act = silu(h[:, :hidden].float()).to(dt) * h[:, hidden:]
    out = ex.int8_linear(act, dev(down[0]), dev(down[1]), offsets=offsets)
    y2 = ex.moe_combine(out, position, offsets, weights)
    loss, counts = ex.moe_balance_loss(logits, ids, 0.01)
    dlogits = ex.moe_balance_loss_backward(torch.ones((), device="cuda"), logits, ids, counts, 0.01)

    rc, rs, rx = R.norm(y, gain, x, 1e-5)
    assert np.array_equal(codes.cpu().numpy(), rc) and R.equal(x2, rx)
    s = scales.cpu().numpy()
    assert np.allclose(s, rs, rtol=2.0 ** -23, atol=0)
    assert R.equal(logits, R.product(rc, s, router[0], (0.02 * router[1]).astype(np.float32), torch.float32))
    flat, _, at = M.sort(ids.cpu().numpy(), experts)
    assert np.array_equal(offsets.cpu().numpy(), at) and np.array_equal(order.cpu().numpy(), flat)
    kept = at[-1]
    for inp, got, (wc, ws) in ((rows, h, up), (act, out, down)):
        qc, qs = R.quantize(inp)
        for e in range(experts):
            a, b = at[e], at[e + 1]
            assert R.equal(got[a:b], R.product(qc[a:b], qs[a:b], wc[e], ws[e], dt))
        assert (got[kept:] == 0).all()
    pos, w = position.cpu().numpy(), weights.cpu().double().numpy()
    terms = np.where(pos < kept, w, 0)[..., None] * out.cpu().double().numpy()[pos]
    size = np.abs(terms).sum(1)
    tol = 2 * top_k * 2.0 ** -24 * size
    assert (np.abs(y2.cpu().double().numpy() - terms.sum(1)) <= tol + 2.0 ** -8 * (np.abs(terms.sum(1)) + tol)).all()
    check(ex, logits.cpu(), ids.cpu().numpy(), 0.01)
    assert torch.isfinite(dlogits).all() and int(counts[:-1].sum()) == kept


def test_training_a_router(ex):
    """The calls inside an autograd.Function, where grad mode is off; two gradients that meet in one leaf."""
    rng = np.random.default_rng(8)
    ids = dev(random_ids(rng, 50, 2, 10))

    class Balance(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits):
            loss, counts = ex.moe_balance_loss(logits, ids, 0.1)
            ctx.save_for_backward(logits, counts)
            return loss

        @staticmethod
        def backward(ctx, dloss):
            logits, counts = ctx.saved_tensors
            return ex.moe_balance_loss_backward(dloss, logits, ids, counts, 0.1)
    x = dev(rng.standard_normal((50, 10)).astype(np.float32)).requires_grad_()
    with pytest.raises(ex.Exl3Error, match="requires grad"):
        ex.moe_balance_loss(x, ids)
    (3 * Balance.apply(x) + 0.5 * Balance.apply(x)).backward()
    wide = x.detach().cpu().double().numpy()
    _, _, gradient, p, s = R.balance(wide, ids.cpu().numpy(), 0.1)
    _, tol = R.balance_tolerances(wide, ids.cpu().numpy(), p, s, 0.35, torch.float32)
    g = gradient(3.5)
    assert (np.abs(x.grad.cpu().double().numpy() - g) <= tol + 4 * 2.0 ** -24 * (np.abs(g) + tol)).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens, experts", [(70, 8), (67, 20), (4000, 64), (300, 257)])
def test_a_token_without_slots_leaves_the_others_results_as_they_are(ex, tokens, experts, dtype):
    """Bit for bit, whatever its logits: tokens that share a wave with it too."""
    dt = DTYPES[dtype]
    rng = np.random.default_rng([7, tokens, experts])
    x = torch.from_numpy(rng.standard_normal((tokens, experts))).to(dt)
    ids = rng.integers(0, experts, (tokens, 2)).astype(np.int32)
    dropped = rng.random(tokens) < 0.3
    ids[dropped] = -1
    one = torch.ones((), device="cuda")
    results = []
    for value in (0.0, float("nan"), float("inf"), -float("inf"), torch.finfo(dt).max, torch.finfo(dt).min, 2.0 ** 15):
        y = x.clone()
        y[torch.from_numpy(dropped)] = value
        y, i = y.cuda(), dev(ids)
        loss, counts = ex.moe_balance_loss(y, i)
        g = ex.moe_balance_loss_backward(one, y, i, counts)
        assert not g[torch.from_numpy(dropped).cuda()].any()
        results.append((loss.view(torch.int32), counts, g.view(torch.int32 if dt == torch.float32 else torch.int16)))
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, results[0]))
