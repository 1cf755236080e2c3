"""Expert routing on the GPU against its definition in float64, and the operators
together as a mixture-of-experts layer runs them."""
import numpy as np
import pytest
import torch

import _mxfp4_ref as R

pytestmark = pytest.mark.gpu
DTYPES = R.DTYPES
HALF32 = 2.0 ** -24  # half a step of fp32


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
    return ids


def route(rng, tokens, top_k, experts, dropped=0.1):
    order, position, offsets = R.sort(random_ids(rng, tokens, top_k, experts, dropped), experts)
    return position, offsets, dev(position.astype(np.int32)), dev(offsets.astype(np.int32))


def f64(t):
    return t.detach().cpu().double().numpy()


def slack(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 0.0  # half of fp16's smallest subnormal


# ---- sort ----

@pytest.mark.parametrize("id_type", [np.int32, np.int64])
@pytest.mark.parametrize("tokens, top_k, experts", [(1, 1, 1), (1, 8, 64), (5, 2, 8), (64, 1, 3), (100, 3, 1024), (128, 8, 64), (129, 8, 64), (512, 8, 64), (513, 8, 64),
                                                    (1365, 3, 200), (1366, 3, 200), (9000, 8, 128), (131072, 2, 7), (40000, 4, 1024)])
def test_sort(ex, tokens, top_k, experts, id_type):
    ids = random_ids(np.random.default_rng([1, tokens, top_k, experts]), tokens, top_k, experts, dtype=id_type)
    for got, ref in zip(ex.moe_sort(dev(ids), experts), R.sort(ids, experts)):
        assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("tokens", [3, 5000])
def test_sort_of_one_expert_and_of_dropped_slots(ex, tokens):
    for fill in (2, -1, 4, 1 << 30, -(1 << 31)):
        ids = np.full((tokens, 2), fill, np.int32)
        for got, ref in zip(ex.moe_sort(dev(ids), 4), R.sort(ids, 4)):
            assert np.array_equal(got.cpu().numpy(), ref)
    ids = np.full((tokens, 2), 1 << 32, np.int64)  # not expert 0 of its low half
    assert not ex.moe_sort(dev(ids), 4)[2].any()


def test_sort_of_no_tokens(ex):
    order, position, offsets = ex.moe_sort(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 5)
    assert order.numel() == 0 and position.shape == (0, 2) and not offsets.any()


# ---- gather, combine and their gradients ----

SHAPES = [(1, 1, 1, 8), (1, 8, 64, 4096), (5, 2, 8, 100), (67, 3, 20, 1000), (33, 4, 5, 2056), (3, 70, 9, 40), (200, 2, 8, 33), (4, 2, 4, 5000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens, top_k, experts, n", SHAPES)
def test_gather_and_its_gradient(ex, tokens, top_k, experts, n, dtype):
    rng = np.random.default_rng([2, tokens, n])
    position, offsets, pos, at = route(rng, tokens, top_k, experts)
    x = torch.from_numpy(rng.standard_normal((tokens, n))).to(DTYPES[dtype])
    slots, kept = tokens * top_k, int(offsets[-1])
    buf = torch.full((slots * n + 64,), 7.0, dtype=x.dtype, device="cuda")
    rows = ex.moe_gather(x.cuda(), pos, at, rows=buf[32:32 + slots * n].view(slots, n))
    assert (buf[:32] == 7).all() and (buf[32 + slots * n:] == 7).all()
    ref = torch.zeros((slots, n), dtype=x.dtype)
    ref[position.reshape(-1)] = x.repeat_interleave(top_k, 0)
    ref[kept:] = 0
    assert torch.equal(rows.cpu(), ref)

    dy = torch.from_numpy(rng.standard_normal((slots, n))).to(DTYPES[dtype])
    dy[kept:] = float("nan")  # a dropped slot's row is not read
    dx = f64(ex.moe_gather_backward(dy.cuda(), pos, at))
    g = f64(dy)
    g[kept:] = 0
    ref, size = g[position].sum(1), np.abs(g[position]).sum(1)
    tol = top_k * HALF32 * size
    assert (np.abs(dx - ref) <= tol + R.half_step(x.dtype) * (np.abs(ref) + tol) + slack(x.dtype)).all()


@pytest.mark.parametrize("weight_type", DTYPES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens, top_k, experts, n", SHAPES)
def test_combine_and_its_gradients(ex, tokens, top_k, experts, n, dtype, weight_type):
    rng = np.random.default_rng([3, tokens, n])
    position, offsets, pos, at = route(rng, tokens, top_k, experts)
    slots, kept, dt, wt = tokens * top_k, int(offsets[-1]), DTYPES[dtype], DTYPES[weight_type]
    rows = torch.from_numpy(rng.standard_normal((slots, n))).to(dt)
    dy = torch.from_numpy(rng.standard_normal((tokens, n))).to(dt)
    weights = torch.from_numpy(rng.random((tokens, top_k))).to(wt)
    live = position < kept
    rows[kept:] = float("nan")  # a dropped slot's row and weight are not used
    weights[torch.from_numpy(~live)] = float("inf")
    r, w, g = f64(rows), np.where(live, f64(weights), 0.0), f64(dy)
    r[kept:] = 0

    y = f64(ex.moe_combine(rows.cuda(), pos, at, weights.cuda()))
    terms = w[..., None] * r[position]
    ref, size = terms.sum(1), np.abs(terms).sum(1)
    tol = (top_k + 1) * HALF32 * size  # each product and each sum rounds once in fp32
    assert (np.abs(y - ref) <= tol + R.half_step(dt) * (np.abs(ref) + tol) + slack(dt)).all()

    buf = torch.full((slots * n + 64,), 7.0, dtype=dt, device="cuda")
    drows, dweights = ex.moe_combine_backward(dy.cuda(), rows.cuda(), pos, at, weights.cuda(), drows=buf[32:32 + slots * n].view(slots, n))
    assert (buf[:32] == 7).all() and (buf[32 + slots * n:] == 7).all()
    ref = np.zeros((slots, n))
    ref[position.reshape(-1)] = (w[..., None] * g[:, None]).reshape(slots, n)
    tol = HALF32 * np.abs(ref)
    assert (np.abs(f64(drows) - ref) <= tol + R.half_step(dt) * (np.abs(ref) + tol) + slack(dt)).all()
    terms = r[position] * g[:, None]
    ref, size = terms.sum(-1), np.abs(terms).sum(-1)
    tol = (n / 64 + 16) * 2 * HALF32 * size  # a lane's chain of products and sums, then the lanes' tree
    assert dweights.dtype == wt
    assert (np.abs(f64(dweights) - ref) <= tol + R.half_step(wt) * (np.abs(ref) + tol) + slack(wt)).all()


def test_combine_gradients_against_differences(ex):
    """y is linear in rows and in weights, so a difference quotient of any step is
    exact up to rounding: fp32, steps of 1, values of order 1 (sums of at most
    3 products of 40 columns, 2^-24 each, over a step of 2: far below 1e-4)."""
    rng = np.random.default_rng(4)
    tokens, top_k, experts, n = 6, 3, 4, 40
    position, offsets, pos, at = route(rng, tokens, top_k, experts, 0.2)
    rows, weights, dy = (torch.from_numpy(rng.standard_normal(s)).float().cuda() for s in ((18, n), (tokens, top_k), (tokens, n)))
    drows, dweights = ex.moe_combine_backward(dy, rows, pos, at, weights)

    def loss(r, w):
        return float((ex.moe_combine(r, pos, at, w).double() * dy.double()).sum())
    for s in range(18):
        for c in (0, 17, n - 1):
            step = torch.zeros_like(rows)
            step[s, c] = 1
            assert abs((loss(rows + step, weights) - loss(rows - step, weights)) / 2 - float(drows[s, c])) < 1e-4
    for t in range(tokens):
        for j in range(top_k):
            step = torch.zeros_like(weights)
            step[t, j] = 1
            assert abs((loss(rows, weights + step) - loss(rows, weights - step)) / 2 - float(dweights[t, j])) < 1e-4
    x, g = (torch.from_numpy(rng.standard_normal(s)).float().cuda() for s in ((tokens, n), (18, n)))
    dx = ex.moe_gather_backward(g, pos, at)
    for t in range(tokens):
        step = torch.zeros_like(x)
        step[t, 5] = 1
        diff = ((ex.moe_gather(x + step, pos, at) - ex.moe_gather(x - step, pos, at)).double() * g.double()).sum() / 2
        assert abs(float(diff) - float(dx[t, 5])) < 1e-4


@pytest.mark.parametrize("dtype", DTYPES)
def test_results_of_32_mib_and_more(ex, dtype):
    """Large results are stored another way: checked whole, on the GPU, in float64."""
    rng = np.random.default_rng(8)
    tokens, top_k, experts, n = 4100, 2, 9, 4096 if dtype == "fp32" else 8192
    position, offsets, pos, at = route(rng, tokens, top_k, experts)
    kept, dt = int(offsets[-1]), DTYPES[dtype]
    gen = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn((tokens, n), generator=gen, device="cuda").to(dt)
    weights = torch.rand((tokens, top_k), generator=gen, device="cuda")
    flat = pos.long().reshape(-1)
    rows = ex.moe_gather(x, pos, at)
    ref = torch.zeros_like(rows)
    ref[flat] = x.repeat_interleave(top_k, 0)
    ref[kept:] = 0
    assert torch.equal(rows, ref)
    w = torch.where(pos < kept, weights, 0.0).double()
    y = ex.moe_combine(rows, pos, at, weights).double()
    ref = (w[..., None] * rows.double()[pos.long()]).sum(1)
    size = (w[..., None] * rows.double()[pos.long()].abs()).sum(1)
    tol = (top_k + 1) * HALF32 * size
    assert bool(((y - ref).abs() <= tol + R.half_step(dt) * (ref.abs() + tol) + slack(dt)).all())
    drows, _ = ex.moe_combine_backward(x, rows, pos, at, weights)
    ref = torch.zeros(rows.shape, dtype=torch.float64, device="cuda")
    ref[flat] = (w[..., None] * x.double()[:, None]).flatten(0, 1)
    tol = HALF32 * ref.abs()
    assert bool(((drows.double() - ref).abs() <= tol + R.half_step(dt) * (ref.abs() + tol) + slack(dt)).all())


def test_positions_outside_the_slots_are_dropped(ex):
    x = torch.arange(24, dtype=torch.float32).reshape(3, 8).cuda()
    pos = torch.tensor([[0, -1], [2, 6], [1 << 30, 4]], dtype=torch.int32).cuda()
    at = torch.tensor([0, 100], dtype=torch.int32).cuda()  # more kept slots than there are
    rows = ex.moe_gather(x, pos, at, rows=torch.full((6, 8), 7.0).cuda())
    assert torch.equal(rows[[0, 2, 4]], x) and (rows[[1, 3, 5]] == 7).all()
    assert torch.equal(ex.moe_combine(rows, pos, at), x)
    w = torch.full((3, 2), 2.0).cuda()
    drows, dw = ex.moe_combine_backward(x, rows, pos, at, w, drows=torch.full((6, 8), 7.0).cuda())
    assert torch.equal(drows[[0, 2, 4]], 2 * x) and (drows[[1, 3, 5]] == 7).all()
    assert (dw.reshape(-1)[[1, 3, 4]] == 0).all()


# ---- together ----



@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens, top_k, experts", [(1, 2, 8), (7, 2, 4), (150, 3, 5)])
def test_mxfp4_expert_layer(ex, tokens, top_k, experts, dtype):
    rng = np.random.default_rng([5, tokens])
    n_in, n_out, dt = 288, 100, DTYPES[dtype]
    ids = random_ids(rng, tokens, top_k, experts)
    x, weights = R.rows(rng, tokens, n_in, dt), torch.from_numpy(rng.random((tokens, top_k))).float()
    codes, scales = R.weight(rng, experts, n_out, n_in)
    order, position, offsets = ex.moe_sort(dev(ids), experts)
    rows = ex.moe_gather(x.cuda(), position, offsets)
    out = ex.mxfp4_linear(rows, dev(codes), dev(scales), offsets=offsets)
    y = f64(ex.moe_combine(out, position, offsets, weights.cuda()))
    values, weight = R.dequantize(*R.quantize(x)), R.dequantize(codes, scales)
    live = (ids >= 0) & (ids < experts)
    w = np.where(live, f64(weights), 0.0)
    each = np.einsum("ti,tjoi->tjo", values, weight[np.where(live, ids, 0)])
    size = np.einsum("ti,tjoi->tjo", np.abs(values), np.abs(weight[np.where(live, ids, 0)]))
    ref = (w[..., None] * each).sum(1)
    # the product's bound, its rounding to dt, and the combine's, each times the weight
    inner = (2 * 3 + 16) * HALF32 * size
    inner = inner + R.half_step(dt) * (np.abs(each) + inner) + slack(dt)
    tol = (w[..., None] * (inner + (top_k + 1) * HALF32 * (np.abs(each) + inner))).sum(1)
    assert (np.abs(y - ref) <= tol + R.half_step(dt) * (np.abs(ref) + tol) + slack(dt)).all()


def test_trellis_expert_layer(ex):
    """The same routing around the library's own trellis weights: exl3_linear on each expert's rows."""
    import synth
    from oracle import exl3_oracle as O
    experts, tokens, top_k, K, n_in, n_out = 3, 21, 2, 3, 256, 64
    rng = np.random.default_rng(6)
    made = [synth.random_case(n_in, n_out, K, 1, [60, e]) for e in range(experts)]
    ids = random_ids(rng, tokens, top_k, experts)
    x = torch.from_numpy(rng.standard_normal((tokens, n_in))).half()
    weights = torch.from_numpy(rng.random((tokens, top_k))).float()
    order, position, offsets = ex.moe_sort(dev(ids), experts)
    rows = ex.moe_gather(x.cuda(), position, offsets)
    out = torch.zeros((tokens * top_k, n_out), dtype=torch.float16, device="cuda")
    at = offsets.tolist()
    for e, (words, _, sign, scale) in enumerate(made):
        if at[e + 1] > at[e]:
            part = rows[at[e]:at[e + 1]]
            ex.linear(part, dev(words.view(np.int16)), dev(sign), dev(scale), K, y=out[at[e]:at[e + 1]])
    y = f64(ex.moe_combine(out, position, offsets, weights.cuda()))
    ref, w = np.zeros((tokens, n_out)), f64(weights)
    for e, (words, _, sign, scale) in enumerate(made):
        full = O.linear(x.numpy(), words, sign, scale, K)
        for j in range(top_k):
            ref += np.where((ids[:, j] == e)[:, None], w[:, j:j + 1] * full, 0.0)
    # the product's own bar (relative 1e-3 of the norm), and half a step of fp16 for the combine
    assert np.linalg.norm(y - ref) <= (1e-3 + 2.0 ** -11) * np.linalg.norm(ref)


def test_captured_layer_with_changing_routes(ex):
    rng = np.random.default_rng(7)
    tokens, top_k, experts, n_in, n_out = 12, 2, 6, 128, 64
    codes, scales = (dev(a) for a in R.weight(rng, experts, n_out, n_in))
    cases = [(dev(random_ids(rng, tokens, top_k, experts)), R.rows(rng, tokens, n_in, torch.bfloat16).cuda(),
              torch.from_numpy(rng.random((tokens, top_k))).float().cuda()) for _ in range(4)]

    def layer(ids, x, w):
        _, position, offsets = ex.moe_sort(ids, experts)
        rows = ex.moe_gather(x, position, offsets)
        out = ex.mxfp4_linear(rows, codes, scales, offsets=offsets)
        y = ex.moe_combine(out, position, offsets, w)
        drows, dw = ex.moe_combine_backward(y, out, position, offsets, w)
        return y, drows, dw
    refs = [[t.clone() for t in layer(*c)] for c in cases]
    held = [t.clone() for t in cases[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(*held)
    for i in (1, 2, 3, 0, 2):
        for h, c in zip(held, cases[i]):
            h.copy_(c)
        graph.replay()
        eager = layer(*cases[(i + 1) % 4])
        torch.cuda.synchronize()
        for a, b in zip(got, refs[i]):
            assert torch.equal(a, b)
        for a, b in zip(eager, refs[(i + 1) % 4]):
            assert torch.equal(a, b)


def test_more_than_32_bits_of_values(ex):
    tokens, top_k, n, dropped = 1 << 19, 2, 4160, 6
    slots = tokens * top_k
    x = torch.randn((1024, n), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").half().repeat(tokens // 1024, 1)
    pos = torch.arange(slots - 1, -1, -1, dtype=torch.int32, device="cuda").reshape(tokens, top_k)  # the first slots come last
    at = torch.tensor([0, slots - dropped], dtype=torch.int32, device="cuda")
    rows = ex.moe_gather(x, pos, at)
    assert rows.numel() > 1 << 32
    none = dropped // top_k  # tokens without a place
    for t in (none, 1, 1000, tokens // 2 - 1, tokens // 2, tokens - 1):
        for j in range(top_k):
            assert torch.equal(rows[slots - 1 - t * top_k - j], x[t] if t >= none else torch.zeros_like(x[t])), (t, j)
    # two equal rows add up without a rounding
    y = ex.moe_combine(rows, pos, at)
    assert torch.equal(y[none:], x[none:] * 2) and not y[:none].any()
    del y
    weights = torch.full((tokens, top_k), 0.5, device="cuda")
    drows, dweights = ex.moe_combine_backward(x, rows, pos, at, weights)
    for a in range(0, slots, 1 << 17):
        assert torch.equal(drows[a:a + (1 << 17)], rows[a:a + (1 << 17)] * 0.5), a
    assert not dweights[:none].any() and bool((dweights[none:] > 0).all())


def test_sort_of_many_slots(ex):
    slots, experts = (1 << 26) + 5, 100
    ids = torch.randint(-3, experts + 3, (slots, 1), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda", dtype=torch.int32)
    order, position, offsets = ex.moe_sort(ids, experts)
    bins = torch.where((ids < 0) | (ids >= experts), experts, ids).reshape(-1)
    counts = torch.bincount(bins, minlength=experts + 1)
    assert torch.equal(offsets[1:].long(), counts.cumsum(0)[:experts]) and int(offsets[0]) == 0
    sorted_bins = bins[order.long()]
    assert bool((sorted_bins[1:] >= sorted_bins[:-1]).all())
    assert bool(((order[1:] > order[:-1]) | (sorted_bins[1:] > sorted_bins[:-1])).all())  # stable, and each slot once
    assert torch.equal(position.reshape(-1)[order.long()], torch.arange(slots, device="cuda", dtype=torch.int32))
