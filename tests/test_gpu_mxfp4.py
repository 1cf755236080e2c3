"""MXFP4 quantisation and products on the GPU against their definition in float64."""
import numpy as np
import pytest
import torch

import _mxfp4_ref as R

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
    return (torch.from_numpy(a) if isinstance(a, np.ndarray) else a).cuda()


def assert_quantized(ex, x):
    codes, scales = ex.mxfp4_quantize(x)
    ref_codes, ref_scales = R.quantize(x)
    assert np.array_equal(scales.cpu().numpy(), ref_scales)
    assert np.array_equal(codes.cpu().numpy(), ref_codes)


# ---- quantise and dequantise: bit for bit ----

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows, n, pad", [(1, 32, 0), (1, 4096, 0), (3, 64, 8), (7, 2080, 24), (257, 96, 0), (33, 1056, 64), (2, 14336, 0)])
def test_quantize_sizes(ex, dtype, rows, n, pad):
    rng = np.random.default_rng([1, rows, n, pad])
    x = R.rows(rng, rows, n + pad, DTYPES[dtype]).cuda()[:, :n]
    assert_quantized(ex, x)


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_every_exponent_and_tie(ex, dtype):
    info = torch.finfo(DTYPES[dtype])
    low = int(np.log2(info.smallest_normal)) - {"fp16": 10, "bf16": 7, "fp32": 23}[dtype]
    high = int(np.floor(np.log2(info.max)))
    eighths = np.concatenate([np.arange(0, 64) / 8, -np.arange(0, 64) / 8]).reshape(4, 32)  # every code, border and tie
    blocks = [eighths[i] * 2.0 ** (e - 2) for e in range(low, high + 1) for i in range(4)]
    # just under and over the borders
    for e in (0, 5):
        for f in (1 - info.eps, 1 + info.eps):
            blocks += [eighths[i] * f * 2.0 ** e for i in range(4)]
    x = torch.from_numpy(np.stack(blocks)).to(DTYPES[dtype]).cuda()
    assert torch.isfinite(x).all()
    assert_quantized(ex, x)


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_zeros_infinities_and_nan(ex, dtype):
    x = torch.ones((9, 96), dtype=DTYPES[dtype])
    x[0] = 0
    x[1] = -0.0
    x[2, 40] = float("inf")
    x[3, 0] = -float("inf")
    x[4, 95] = float("nan")
    x[5, 31], x[5, 32] = float("nan"), float("inf")
    x[6] = torch.finfo(x.dtype).max
    x[7] = -torch.finfo(x.dtype).smallest_normal
    x[8] = torch.finfo(x.dtype).smallest_normal / 4
    assert_quantized(ex, x.cuda())
    codes, scales = ex.mxfp4_quantize(x.cuda())
    v = ex.mxfp4_dequantize(codes, scales, x.dtype).cpu()
    assert torch.isnan(v).nonzero().tolist() == [[r, c] for r, lo, hi in ((2, 32, 64), (3, 0, 32), (4, 64, 96), (5, 0, 64)) for c in range(lo, hi)]


@pytest.mark.parametrize("dtype", DTYPES)
def test_dequantize_every_code_and_scale(ex, dtype):
    scales = np.arange(256, dtype=np.uint8)[:, None]
    codes = np.tile(np.arange(16, dtype=np.uint8) * 0x11 ^ 0x30, (256, 1))
    got = ex.mxfp4_dequantize(dev(codes), dev(scales), DTYPES[dtype]).cpu()
    with np.errstate(over="ignore"):
        ref = torch.from_numpy(R.dequantize(codes, scales)).to(DTYPES[dtype])
    assert torch.equal(got[:255], ref[:255])
    assert torch.isnan(got[255]).all()


def test_dequantize_of_quantized_rows_is_exact(ex):
    for dtype in DTYPES.values():
        x = R.rows(np.random.default_rng(2), 37, 352, dtype).cuda()
        codes, scales = ex.mxfp4_quantize(x)
        assert np.array_equal(ex.mxfp4_dequantize(codes, scales, dtype).cpu().double().numpy(), R.dequantize(codes, scales))


def test_quantize_into_given_tensors_leaves_what_surrounds_them(ex):
    x = R.rows(np.random.default_rng(3), 5, 64, torch.float16).cuda()
    codes, scales = torch.full((9, 32), 0xAB, dtype=torch.uint8).cuda(), torch.full((42,), 0xAB, dtype=torch.uint8).cuda()
    ex.mxfp4_quantize(x, codes=codes[2:7], scales=scales[16:26].view(5, 2))
    assert (codes[:2] == 0xAB).all() and (codes[7:] == 0xAB).all() and (scales[:16] == 0xAB).all() and (scales[26:] == 0xAB).all()
    assert np.array_equal(codes[2:7].cpu().numpy(), R.quantize(x)[0])


# ---- products ----

def check_linear(ex, m, n_in, n_out, dtype, pad=0, seed=0):
    rng = np.random.default_rng([seed, m, n_in, n_out])
    x = R.rows(rng, m, n_in + pad, DTYPES[dtype]).cuda()[:, :n_in]
    codes, scales = R.weight(rng, n_out, n_in)
    values = R.dequantize(*R.quantize(x))
    weight = R.dequantize(codes, scales)
    # y in the middle of a larger buffer: nothing around it may change
    buf = torch.full((m * n_out + 64,), 7.0, dtype=x.dtype, device="cuda")
    y = buf[32:32 + m * n_out].view(m, n_out)
    ex.mxfp4_linear(x, dev(codes), dev(scales), y=y)
    R.assert_product(y, values, weight, x.dtype, ("linear", m, n_in, n_out, dtype))
    assert (buf[:32] == 7).all() and (buf[32 + m * n_out:] == 7).all()
    xc, xs = ex.mxfp4_quantize(x)
    y = ex.mxfp4_matmul(xc, xs, dev(codes), dev(scales), x.dtype)
    R.assert_product(y, values, weight, x.dtype, ("matmul", m, n_in, n_out, dtype))


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 97, 127, 128, 129, 192, 255, 256, 257, 400, 513])
def test_linear_rows(ex, m):
    check_linear(ex, m, 544, 272, ("fp16", "bf16", "fp32")[m % 3])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m", [1, 5, 40, 100, 300])
@pytest.mark.parametrize("n_in", [32, 64, 96, 128, 480, 512, 1056, 4096 + 32])
def test_linear_inputs(ex, m, n_in, dtype):
    check_linear(ex, m, n_in, 48, dtype, pad=(n_in // 32) % 3 * 8)


@pytest.mark.parametrize("m", [1, 20, 70, 140])
@pytest.mark.parametrize("n_out", [1, 2, 3, 5, 15, 16, 17, 63, 64, 65, 255, 256, 257, 511, 1001])
def test_linear_outputs(ex, m, n_out):
    check_linear(ex, m, 288, n_out, ("fp16", "bf16", "fp32")[n_out % 3])


@pytest.mark.parametrize("m, n_in, n_out, dtype", [(1, 14336, 4096, "bf16"), (16, 28672, 512, "fp16"), (600, 4096, 1024, "bf16"),
                                                    (1100, 1024, 2100, "fp32")])
def test_linear_large(ex, m, n_in, n_out, dtype):
    check_linear(ex, m, n_in, n_out, dtype)


@pytest.mark.parametrize("m", [3, 30, 90, 300])
def test_nan_stays_in_its_row_and_column(ex, m):
    rng = np.random.default_rng([4, m])
    x = R.rows(rng, m, 672, torch.float32)
    x[m - 1, 671] = float("inf")  # the last row, also read for the padding rows of its tile
    codes, scales = R.weight(rng, 77, 672)
    scales[76, 20] = 255
    scales[3, 0] = 255
    y = ex.mxfp4_linear(x.cuda(), dev(codes), dev(scales))
    R.assert_product(y, R.dequantize(*R.quantize(x)), R.dequantize(codes, scales), torch.float32)
    bad = torch.isnan(y)
    assert bad[m - 1].all() and bad[:, 76].all() and bad[:, 3].all() and int(bad.sum()) == 77 + 2 * (m - 1)


def test_no_rows(ex):
    codes, scales = R.weight(np.random.default_rng(5), 8, 64)
    assert ex.mxfp4_linear(torch.empty((0, 64), device="cuda"), dev(codes), dev(scales)).shape == (0, 8)
    assert ex.mxfp4_quantize(torch.empty((0, 64), device="cuda"))[0].shape == (0, 32)


# ---- groups ----

def check_groups(ex, counts, behind, n_in, n_out, dtype, seed=0):
    rng = np.random.default_rng([6, seed, n_in, n_out, len(counts)])
    groups, m = len(counts), sum(counts) + behind
    x = R.rows(rng, m, n_in, DTYPES[dtype])
    if behind:
        x[sum(counts):] = float("nan")  # rows of no group are not read into a result
    codes, scales = R.weight(rng, groups, n_out, n_in)
    for g, c in enumerate(counts):
        if c == 0:
            scales[g] = 255  # nor are weights of empty groups
    at = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    values, weight = R.dequantize(*R.quantize(x)), R.dequantize(codes, scales)
    buf = torch.full((m * n_out + 64,), 7.0, dtype=x.dtype, device="cuda")
    y = buf[32:32 + m * n_out].view(m, n_out)
    ex.mxfp4_linear(x.cuda(), dev(codes), dev(scales), offsets=dev(at), y=y)
    xc, xs = ex.mxfp4_quantize(x.cuda())
    z = ex.mxfp4_matmul(xc, xs, dev(codes), dev(scales), x.dtype, offsets=dev(at))
    assert (buf[:32] == 7).all() and (buf[32 + m * n_out:] == 7).all()
    for out in (y, z):
        for g in range(groups):
            R.assert_product(out[at[g]:at[g + 1]], values[at[g]:at[g + 1]], weight[g], x.dtype, ("group", g, counts[g]))
        assert (out[at[-1]:] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts, behind", [([1], 0), ([0, 3], 0), ([0, 0, 0], 5), ([2, 0, 1, 0], 1), ([16, 17, 1, 0, 33], 3),
                                            ([40, 0, 65, 3], 0), ([200, 100, 0, 130], 70), ([300, 1, 600], 0)])
def test_groups(ex, counts, behind, dtype):
    check_groups(ex, counts, behind, 352, 80, dtype)


@pytest.mark.parametrize("n_in, n_out", [(160, 2500), (160, 10000), (256, 10001)])
def test_large_groups(ex, n_in, n_out):
    check_groups(ex, [700, 0, 900, 450], 30, n_in, n_out, "bf16")


def test_many_groups(ex):
    rng = np.random.default_rng(7)
    check_groups(ex, [int(c) for c in rng.integers(0, 4, 150)], 9, 64, 33, "bf16")
    check_groups(ex, [0] * 127 + [5], 0, 64, 33, "bf16")
    check_groups(ex, [int(c) for c in rng.integers(0, 90, 70)], 0, 128, 40, "fp16")
    check_groups(ex, [0] * 64 + [400] + [0] * 63, 1, 128, 40, "fp16")


@pytest.mark.parametrize("groups", [191, 192, 255, 256, 257, 511, 1030])
def test_more_groups_than_one_batch_of_offsets(ex, groups):
    # a tile is looked for 64 groups at a time, 256 of them loaded together
    rng = np.random.default_rng([8, groups])
    check_groups(ex, [int(c) for c in rng.integers(0, 3, groups)], 2, 64, 17, "fp16")
    check_groups(ex, [0] * (groups - 1) + [3], 0, 64, 17, "bf16")
    check_groups(ex, [0] * (groups - 70) + [150] + [0] * 69, 5, 64, 17, "fp32")


@pytest.mark.parametrize("n_in", [96, 512, 2048, 4096, 4128, 16384, 16416])
@pytest.mark.parametrize("m", [1, 2, 4, 5, 8])
def test_few_rows_of_every_length(ex, m, n_in):
    check_linear(ex, m, n_in, 40, ("fp16", "bf16", "fp32")[(m + n_in // 32) % 3], pad=16)


# the tile sizes: 128 x 128 and 256 x 256, every number of stages of 256 inputs from 1 to 5, and rows of scales that start at any byte
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_in", [96, 256, 288, 640, 1024, 1056])
@pytest.mark.parametrize("m, n_out", [(1100, 2100), (2050, 6001)])
def test_linear_large_tiles(ex, m, n_in, n_out, dtype):
    check_linear(ex, m, n_in, n_out, dtype)


@pytest.mark.parametrize("n_in, n_out, dtype", [(288, 10200, "bf16"), (544, 10203, "fp32"), (256, 10201, "fp16")])
def test_linear_of_both_large_tiles(ex, n_in, n_out, dtype):
    check_linear(ex, 2040, n_in, n_out, dtype)


@pytest.mark.parametrize("m, n_in, n_out", [(70, 4096, 700), (200, 2048, 3000), (200, 2080, 3000), (600, 1056, 2000), (1500, 512, 1500)])
def test_linear_of_many_tiles(ex, m, n_in, n_out):
    check_linear(ex, m, n_in, n_out, "bf16")


def test_offsets_outside_the_rows_are_taken_as_the_nearer_end(ex):
    rng = np.random.default_rng(8)
    x = R.rows(rng, 6, 64, torch.float32)
    codes, scales = R.weight(rng, 3, 16, 64)
    y = ex.mxfp4_linear(x.cuda(), dev(codes), dev(scales), offsets=dev(np.array([-5, 2, 4, 1 << 30], np.int32)))
    values, weight = R.dequantize(*R.quantize(x)), R.dequantize(codes, scales)
    for g in range(3):
        R.assert_product(y[2 * g:2 * g + 2], values[2 * g:2 * g + 2], weight[g], torch.float32)


# ---- streams and graphs ----

@pytest.mark.parametrize("m", [2, 300])
def test_on_another_stream(ex, m):
    rng = np.random.default_rng([9, m])
    x = R.rows(rng, m, 512, torch.bfloat16)
    codes, scales = (dev(a) for a in R.weight(rng, 64, 512))
    xd = x.cuda()
    ref = ex.mxfp4_linear(xd, codes, scales)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    given = ex.mxfp4_linear(xd, codes, scales, stream=side)
    with torch.cuda.stream(side):
        current = ex.mxfp4_linear(xd, codes, scales)
    torch.cuda.synchronize()
    assert torch.equal(given, ref) and torch.equal(current, ref)


def test_two_captured_graphs_and_eager_calls(ex):
    rng = np.random.default_rng(10)
    codes, scales = (dev(a) for a in R.weight(rng, 96, 512))
    batches = [[R.rows(rng, m, 512, torch.float16).cuda() for _ in range(4)] for m in (3, 200)]
    refs = [[ex.mxfp4_linear(x, codes, scales).clone() for x in xs] for xs in batches]
    graphs = []
    for xs in batches:
        x = xs[0].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            ex.mxfp4_linear(x, codes, scales)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = ex.mxfp4_linear(x, codes, scales)
        graphs.append((g, x, y))
    for i in (1, 2, 3, 0):
        for (g, x, y), xs, ref in zip(graphs, batches, refs):
            x.copy_(xs[i])
            g.replay()
            eager = ex.mxfp4_linear(xs[(i + 1) % 4], codes, scales)
            torch.cuda.synchronize()
            assert torch.equal(y, ref[i]) and torch.equal(eager, ref[(i + 1) % 4])


def test_given_workspace(ex):
    rng = np.random.default_rng(11)
    x = R.rows(rng, 100, 512, torch.float16).cuda()
    codes, scales = (dev(a) for a in R.weight(rng, 64, 512))
    need = ex.mxfp4_workspace_bytes(100, 512)
    ws = torch.full((need + 256,), 0xCD, dtype=torch.uint8, device="cuda")
    y = ex.mxfp4_linear(x, codes, scales, workspace=ws[:need])
    assert torch.equal(y, ex.mxfp4_linear(x, codes, scales)) and (ws[need:] == 0xCD).all()
    with pytest.raises(ex.Exl3Error, match="workspace"):
        ex.mxfp4_linear(x, codes, scales, workspace=ws[:need - 16])


# ---- more than 2^32 elements ----
#
# Large tensors repeat 1024 rows, so that every part of a result has to equal the
# first.  Codes under a scale of 1 have products that are multiples of 1/4, at most
# 36, and up to 16384 of them sum to less than 2^24 / 4: fp32 sums are exact.

def test_quantize_more_than_32_bits_of_values(ex):
    rows, n = 1 << 20, 4128
    base = torch.randn((1024, n), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    x = base.repeat(rows // 1024, 1)
    assert x.numel() > 1 << 32
    codes, scales = ex.mxfp4_quantize(x)
    ref = ex.mxfp4_quantize(base)
    del x
    out = ex.mxfp4_dequantize(codes, scales, torch.bfloat16)
    ref += (ex.mxfp4_dequantize(*ref, torch.bfloat16),)
    for i in (0, 1, 507, 508, 1016, 1022, 1023):
        for got, want in zip((codes, scales, out), ref):
            assert torch.equal(got[1024 * i:1024 * (i + 1)], want), i


def test_product_of_more_than_32_bits_of_outputs(ex):
    gen = torch.Generator(device="cuda").manual_seed(2)
    m, n_in, n_out = 1 << 20, 64, 4160
    base = torch.randint(0, 256, (1024, n_in // 2), generator=gen, device="cuda", dtype=torch.uint8)
    w = torch.randint(0, 256, (n_out, n_in // 2), generator=gen, device="cuda", dtype=torch.uint8)
    one = lambda rows: torch.full((rows, n_in // 32), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    y = ex.mxfp4_matmul(base.repeat(m // 1024, 1), one(m), w, one(n_out))
    assert y.numel() > 1 << 32
    ref = (ex.mxfp4_dequantize(base, one(1024), torch.float32).double().cpu()
           @ ex.mxfp4_dequantize(w, one(n_out), torch.float32).double().cpu().T).bfloat16().cuda()
    for i in (0, 1, 503, 504, 1007, 1022, 1023):
        assert torch.equal(y[1024 * i:1024 * (i + 1)], ref), i


@pytest.mark.parametrize("rows", [3, 20, 200, 1500])
def test_weights_of_more_than_32_bits(ex, rows):
    gen = torch.Generator(device="cuda").manual_seed(3)
    groups, n_out, n_in = 72, 8192, 16384
    w = torch.randint(0, 256, (n_out, n_in // 2), generator=gen, device="cuda", dtype=torch.uint8).repeat(groups, 1, 1)
    assert w.numel() > 1 << 32
    w[-1] ^= 0x5A
    scales = torch.full((groups, n_out, n_in // 32), 127, dtype=torch.uint8, device="cuda")
    xc = torch.randint(0, 256, (rows, n_in // 2), generator=gen, device="cuda", dtype=torch.uint8)
    xs = torch.full((rows, n_in // 32), 127, dtype=torch.uint8, device="cuda")
    at = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    at[-1], at[-2] = rows, 1  # one row of the last group but one, the others of the last
    y = ex.mxfp4_matmul(xc, xs, w, scales, torch.float32, offsets=at)
    for g, a, b in ((-2, 0, 1), (-1, 1, rows)):
        assert torch.equal(y[a:b], ex.mxfp4_matmul(xc[a:b].clone(), xs[a:b].clone(), w[g], scales[g], torch.float32)), g
    ref = ex.mxfp4_dequantize(xc[1:3], xs[1:3].contiguous(), torch.float32).double().cpu() \
        @ ex.mxfp4_dequantize(w[-1], scales[-1], torch.float32).double().cpu().T
    assert torch.equal(y[1:3].double().cpu(), ref)
