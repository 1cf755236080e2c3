"""8-bit quantisation, norm and products on the GPU against their definitions: codes and
products bit for bit, a norm's scales to the rounding of their last step."""
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


def dev(a):
    return (torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a).cuda()


def same(t, a):
    return np.array_equal(t.cpu().numpy(), a, equal_nan=t.is_floating_point())


# ---- quantise and dequantise ----

SIZES = [(1, 16, 0), (1, 4096, 0), (3, 64, 8), (7, 2064, 24), (257, 48, 0), (33, 1040, 64), (2, 14336, 0), (5, 512, 0), (6, 528, 0),
         (4, 2048, 0), (3, 8192, 0), (3, 8208, 8), (2, 32768, 0), (2, 32784, 0), (1, 131072, 8)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows, n, pad", SIZES)
def test_quantize_sizes(ex, dtype, rows, n, pad):
    x = R.rows(np.random.default_rng([1, rows, n]), rows, n + pad, DTYPES[dtype]).cuda()[:, :n]
    codes, scales = ex.int8_quantize(x)
    ref_codes, ref_scales = R.quantize(x)
    assert same(codes, ref_codes) and same(scales, ref_scales)
    for out in DTYPES.values():
        assert R.equal(ex.int8_dequantize(codes, scales, out), (torch.from_numpy(ref_codes).float() * torch.from_numpy(ref_scales)[:, None]).to(out))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [16, 32, 48, 64, 96, 128, 144, 256, 272, 512, 1024, 1040, 2048, 2064, 4096, 4112, 8192, 14336])
def test_many_rows(ex, dtype, n):
    """More than the few rows that other waves and pieces are chosen for."""
    rng = np.random.default_rng([21, n])
    x, r = (R.rows(rng, 700, n, DTYPES[dtype]).cuda() for _ in range(2))
    x[3, n // 2] = float("nan")
    codes, scales = ex.int8_quantize(x)
    ref = R.quantize(x)
    assert same(codes, ref[0]) and same(scales, ref[1])
    check_norm(ex, x, torch.from_numpy(1 + 0.3 * rng.standard_normal(n)).to(DTYPES[dtype]).cuda(), r, 1e-6)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("largest", [1.0, 127.0, 254.0, 1.9921875, 93.0, 2.0 ** -14, 2.0 ** -24])
def test_quantize_ties(ex, dtype, largest):
    """Half of the largest value is a tie for any of them, every odd multiple of 1 / 254 for 127."""
    dt = DTYPES[dtype]
    steps = np.arange(-254, 255) / 254 * largest
    x = torch.from_numpy(np.concatenate([steps, [largest / 2, -largest / 2, largest, -largest, 0.0, -0.0] + [0.0] * 13])).to(dt)
    x = x[:528 // 16 * 16][None].repeat(3, 1)
    x[1] *= 0.5
    x[2] = torch.nextafter(x[2].float(), torch.tensor(9e9)).to(dt).clamp(-largest, largest)
    codes, scales = ex.int8_quantize(x.cuda())
    ref_codes, ref_scales = R.quantize(x)
    assert same(codes, ref_codes) and same(scales, ref_scales)


def test_quantize_values_next_to_ties(ex):
    """fp32 values one step to either side of every tie: the quotient is exact."""
    rng = np.random.default_rng(2)
    a = np.exp2(rng.uniform(-120, 120, 64)).astype(np.float32)
    tie = ((np.arange(-127, 127) + 0.5)[None] * (a.astype(np.float64) / 127)[:, None]).astype(np.float32)
    x = np.concatenate([tie, np.nextafter(tie, np.float32(np.inf)), np.nextafter(tie, np.float32(-np.inf)), a[:, None], 0 * tie[:, :5]], 1)
    x = x[:, :x.shape[1] // 16 * 16]
    x[:, 0] = a
    codes, scales = ex.int8_quantize(dev(x))
    ref_codes, ref_scales = R.quantize(torch.from_numpy(x))
    assert same(codes, ref_codes) and same(scales, ref_scales)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [96, 1040, 5120, 40000])
def test_quantize_zeros_infinities_nan_and_the_ends_of_the_range(ex, dtype, n):
    dt = DTYPES[dtype]
    x = torch.ones((9, n), dtype=dt)
    x[0], x[1] = 0, -0.0
    x[2, 40], x[3, 0], x[4, n - 1] = float("inf"), -float("inf"), float("nan")
    x[5, 31], x[5, 32] = float("nan"), float("inf")
    x[6] = torch.finfo(dt).max
    x[7, ::3] = -torch.finfo(dt).smallest_normal
    x[7, 1::3] = torch.finfo(dt).smallest_normal / 4
    x[7, 2::3] = 0
    x[8] = 0
    x[8, 5] = 2.0 ** -24 if dtype == "fp16" else 2.0 ** -133
    codes, scales = ex.int8_quantize(x.cuda())
    ref_codes, ref_scales = R.quantize(x)
    assert same(codes, ref_codes) and same(scales, ref_scales)
    assert torch.isnan(scales).cpu().tolist() == [r in (2, 3, 4, 5) for r in range(9)] and not codes[2:6].any()
    assert torch.isnan(ex.int8_dequantize(codes, scales, dt)[2:6]).all()


def test_given_tensors_and_what_surrounds_them(ex):
    x = R.rows(np.random.default_rng(3), 5, 64, torch.float16).cuda()
    codes, scales = torch.full((9, 64), 99, dtype=torch.int8).cuda(), torch.full((9,), 7.0).cuda()
    ex.int8_quantize(x, codes=codes[2:7], scales=scales[3:8])  # scales at any fp32
    ref = R.quantize(x)
    assert same(codes[2:7], ref[0]) and same(scales[3:8], ref[1])
    assert (codes[:2] == 99).all() and (codes[7:] == 99).all() and (scales[:3] == 7).all() and (scales[8:] == 7).all()


def test_no_rows(ex):
    x = torch.empty((0, 64), device="cuda")
    c, s = ex.int8_quantize(x)
    assert c.shape == (0, 64) and s.shape == (0,) and ex.int8_dequantize(c, s).shape == (0, 64)
    assert [t.shape for t in ex.int8_rms_norm(x, torch.ones(64, device="cuda"), x.clone())] == [(0, 64), (0,), (0, 64)]
    wc, ws = R.weight(np.random.default_rng(4), 8, 64)
    assert ex.int8_linear(x, dev(wc), dev(ws)).shape == (0, 8) and ex.int8_matmul(c, s, dev(wc), dev(ws)).shape == (0, 8)


# ---- norm ----

def check_norm(ex, x, weight, residual, eps):
    got = ex.int8_rms_norm(x, weight, residual, eps=eps)
    codes, scales, h = R.norm(x, weight, residual, eps)
    assert len(got) == (2 if residual is None else 3)
    assert same(got[0], codes)
    if residual is not None:
        assert R.equal(got[2], h)
    s = got[1].cpu().double().numpy()
    assert (np.isnan(s) == np.isnan(scales)).all()
    # 64 bits up to the last rounding: half a step of fp32 (of its smallest subnormal), and n sums and a few steps of 2^-53
    tol = scales * (2.0 ** -24 + (x.shape[1] + 16) * 2.0 ** -53) * 1.0001 + 2.0 ** -150
    assert (np.abs(s - scales) <= tol)[~np.isnan(scales)].all()
    return got


@pytest.mark.parametrize("with_residual", [True, False])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows, n, pad", SIZES)
def test_norm_sizes(ex, dtype, rows, n, pad, with_residual):
    rng = np.random.default_rng([5, rows, n])
    dt = DTYPES[dtype]
    x = R.rows(rng, rows, n + pad, dt).cuda()[:, :n]
    residual = R.rows(rng, rows, n + 16, dt).cuda()[:, 16:] if with_residual else None
    weight_type = list(DTYPES.values())[(rows + n // 16) % 3]
    check_norm(ex, x, torch.from_numpy(1 + 0.3 * rng.standard_normal(n)).to(weight_type).cuda(), residual, 1e-6)


@pytest.mark.parametrize("weight_type", DTYPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_types_and_eps(ex, dtype, weight_type):
    rng = np.random.default_rng(6)
    x, r = (R.rows(rng, 4, 400, DTYPES[dtype]).cuda() for _ in range(2))
    w = torch.from_numpy(rng.standard_normal(400)).to(DTYPES[weight_type]).cuda()
    for eps in (0.0, 1e-6, 1e-5, 1.0, 1e30):
        check_norm(ex, x, w, r, eps)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [64, 1040, 5120, 40000])
def test_norm_of_rows_at_the_edge(ex, dtype, n):
    dt = DTYPES[dtype]
    info = torch.finfo(dt)
    x, r = torch.ones((10, n), dtype=dt), torch.zeros((10, n), dtype=dt)
    x[0] = 0                                             # nothing at all: eps alone under the root
    x[1], r[1] = 3, -3                                   # a sum of zeros
    x[2, 7] = float("inf")
    r[3, n - 1] = float("nan")
    x[4], r[4] = info.max, info.max                      # the sum is infinite
    x[5] = info.max                                      # its squares are beyond fp32 (bf16, fp32)
    x[6] = info.smallest_normal                          # its squares are below
    x[7, :] = 0
    x[7, 3] = info.smallest_normal
    x[8, 1], r[8, 1] = float("inf"), -float("inf")       # NaN
    w = torch.ones(n, dtype=dt)
    for eps in (0.0, 1e-6):
        codes, scales, h = check_norm(ex, x.cuda(), w.cuda(), r.cuda(), eps)
        assert torch.isnan(scales).cpu().tolist() == [i in (2, 3, 4, 8) for i in range(10)]
        assert not codes[[0, 1, 2, 3, 4, 8]].any() and (scales[:2] == 0).all()
    w[5] = float("nan")
    assert torch.isnan(ex.int8_rms_norm(x.cuda(), w.cuda())[1]).all()
    w = torch.zeros(n, dtype=dt)
    codes, scales = ex.int8_rms_norm(x[5:8].cuda(), w.cuda())
    assert not codes.any() and not scales.any()
    # a product with the weight that leaves fp32
    codes, scales = check_norm(ex, x[5:6].cuda(), torch.full((n,), 1e38, device="cuda"), None, 1e-6)
    assert torch.isnan(scales).all() and not codes.any()


def test_norm_into_given_tensors(ex):
    rng = np.random.default_rng(7)
    x, r = (R.rows(rng, 5, 48, torch.bfloat16).cuda() for _ in range(2))
    w = torch.ones(48, device="cuda")
    codes, scales, added = torch.full((7, 48), 99, dtype=torch.int8).cuda(), torch.full((9,), 7.0).cuda(), torch.full((7, 48), 7.0).bfloat16().cuda()
    ex.int8_rms_norm(x, w, r, codes=codes[1:6], scales=scales[2:7], added=added[1:6])
    ref = ex.int8_rms_norm(x, w, r)
    for got, want, fill in ((codes, ref[0], 99), (added, ref[2], 7)):
        assert torch.equal(got[1:6], want) and (got[[0, 6]] == fill).all()
    assert torch.equal(scales[2:7], ref[1]) and (scales[[0, 1, 7, 8]] == 7).all()


def test_more_rows_than_workgroups(ex):
    """More rows than a launch has workgroups: they take row after row."""
    n, rows = 16, (1 << 22) + 5
    base = R.rows(np.random.default_rng(8), 64, n, torch.bfloat16)
    x = base.repeat(rows // 64 + 1, 1)[:rows].cuda()
    codes, scales = ex.int8_quantize(x)
    ref = R.quantize(base)
    at = torch.arange(rows, device="cuda") % 64
    assert torch.equal(codes, dev(ref[0])[at]) and torch.equal(scales, dev(ref[1])[at])


# ---- products ----

def check_product(ex, m, n_in, n_out, dtype, pad=0, seed=0):
    rng = np.random.default_rng([9, seed, m, n_in, n_out])
    dt = DTYPES[dtype]
    x = R.rows(rng, m, n_in + pad, dt).cuda()[:, :n_in]
    wc, ws = R.weight(rng, n_out, n_in)
    ref = R.product(*R.quantize(x), wc, ws, dt)
    # y in the middle of a larger buffer: nothing around it may change
    buf = torch.full((m * n_out + 64,), 7.0, dtype=dt, device="cuda")
    y = ex.int8_linear(x, dev(wc), dev(ws), y=buf[32:32 + m * n_out].view(m, n_out))
    assert R.equal(y, ref), ("linear", m, n_in, n_out, dtype)
    assert (buf[:32] == 7).all() and (buf[32 + m * n_out:] == 7).all()
    y = ex.int8_matmul(*ex.int8_quantize(x), dev(wc), dev(ws), dt)
    assert R.equal(y, ref), ("matmul", m, n_in, n_out, dtype)


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 97, 127, 128, 129, 192, 255, 256, 257, 400, 513])
def test_linear_rows(ex, m):
    check_product(ex, m, 528, 272, ("fp16", "bf16", "fp32")[m % 3])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m", [1, 5, 40, 100, 300])
@pytest.mark.parametrize("n_in", [16, 32, 48, 96, 112, 128, 144, 256, 496, 512, 1040, 4112])
def test_linear_inputs(ex, m, n_in, dtype):
    check_product(ex, m, n_in, 48, dtype, pad=(n_in // 16) % 3 * 8)


@pytest.mark.parametrize("m", [1, 20, 70, 140])
@pytest.mark.parametrize("n_out", [1, 2, 3, 5, 15, 16, 17, 63, 64, 65, 255, 256, 257, 511, 1001])
def test_linear_outputs(ex, m, n_out):
    check_product(ex, m, 272, n_out, ("fp16", "bf16", "fp32")[n_out % 3])


@pytest.mark.parametrize("m, n_in, n_out, dtype", [(1, 14336, 4096, "bf16"), (16, 28672, 512, "fp16"), (600, 4096, 1024, "bf16"), (3, 65552, 40, "fp16"),
                                                    (1100, 1024, 2100, "fp32"), (70, 4096, 700, "fp16"), (200, 2064, 3000, "bf16"),
                                                    (8, 4096, 5000, "bf16"), (13, 14336, 1000, "bf16"), (24, 14336, 300, "bf16")])
def test_linear_large(ex, m, n_in, n_out, dtype):
    check_product(ex, m, n_in, n_out, dtype)


# large tiles at every number of stages, odd ends
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_in", [16, 128, 144, 272, 640, 1040])
@pytest.mark.parametrize("m, n_out", [(1100, 2100), (2050, 6001)])
def test_linear_large_tiles(ex, m, n_in, n_out, dtype):
    check_product(ex, m, n_in, n_out, dtype)


@pytest.mark.parametrize("n_in, n_out, dtype", [(272, 10200, "bf16"), (528, 10203, "fp32"), (256, 10201, "fp16")])
def test_linear_of_many_tiles(ex, n_in, n_out, dtype):
    check_product(ex, 2040, n_in, n_out, dtype)


@pytest.mark.parametrize("m", [2, 40, 300, 1100])
def test_largest_sums(ex, m):
    """All codes -128 over the longest row: 2^14 * 131056, 2^18 below 2^31."""
    n_in, n_out = (1 << 17) - 16, 70
    xc, wc = torch.full((m, n_in), -128, dtype=torch.int8, device="cuda"), torch.full((n_out, n_in), -128, dtype=torch.int8, device="cuda")
    wc[3] = 127
    y = ex.int8_matmul(xc, torch.ones(m, device="cuda"), wc, torch.ones(n_out, device="cuda"), torch.float32)
    ref = torch.full((m, n_out), float(2 ** 14 * n_in), device="cuda")
    ref[:, 3] = -float(128 * 127 * n_in)
    assert torch.equal(y, ref)


@pytest.mark.parametrize("m", [3, 30, 90, 300])
def test_nan_stays_in_its_row_and_column(ex, m):
    rng = np.random.default_rng([10, m])
    x = R.rows(rng, m, 656, torch.float32)
    x[m - 1, 655] = float("inf")  # the last row, also read for the padding rows of its tile
    wc, ws = R.weight(rng, 77, 656)
    ws[76] = ws[3] = np.nan
    y = ex.int8_linear(x.cuda(), dev(wc), dev(ws))
    assert R.equal(y, R.product(*R.quantize(x), wc, ws, torch.float32))
    bad = torch.isnan(y)
    assert bad[m - 1].all() and bad[:, 76].all() and bad[:, 3].all() and int(bad.sum()) == 77 + 2 * (m - 1)


@pytest.mark.parametrize("m", [3, 100])
def test_scales_of_any_size(ex, m):
    rng = np.random.default_rng([11, m])
    xc, wc = (rng.integers(-128, 128, s, dtype=np.int8) for s in ((m, 64), (40, 64)))
    xs, ws = (np.exp2(rng.uniform(-140, 120, n)).astype(np.float32) for n in (m, 40))
    for dt in DTYPES.values():
        y = ex.int8_matmul(dev(xc), dev(xs), dev(wc), dev(ws), dt)
        assert R.equal(y, R.product(xc, xs, wc, ws, dt))


def test_rows_of_a_weight_and_of_an_input(ex):
    """Slices from any row on: codes start at 16 bytes, scales at 4."""
    rng = np.random.default_rng(12)
    wc, ws = R.weight(rng, 90, 48)
    x = R.rows(rng, 50, 48, torch.bfloat16)
    codes, scales = ex.int8_quantize(x.cuda())
    y = ex.int8_matmul(codes[7:40], scales[7:40], dev(wc)[5:82], dev(ws)[5:82])
    assert R.equal(y, R.product(*R.quantize(x[7:40]), wc[5:82], ws[5:82], torch.bfloat16))


# ---- groups ----

def check_groups(ex, counts, behind, n_in, n_out, dtype, seed=0):
    rng = np.random.default_rng([13, seed, n_in, n_out, len(counts)])
    groups, m, dt = len(counts), sum(counts) + behind, DTYPES[dtype]
    x = R.rows(rng, m, n_in, dt)
    if behind:
        x[sum(counts):] = float("nan")  # rows of no group are not read into a result
    wc, ws = R.weight(rng, groups, n_out, n_in)
    for g, c in enumerate(counts):
        if c == 0:
            ws[g] = np.nan  # nor are weights of empty groups
    at = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    xc, xs = R.quantize(x)
    buf = torch.full((m * n_out + 64,), 7.0, dtype=dt, device="cuda")
    y = ex.int8_linear(x.cuda(), dev(wc), dev(ws), offsets=dev(at), y=buf[32:32 + m * n_out].view(m, n_out))
    z = ex.int8_matmul(dev(xc), dev(xs), dev(wc), dev(ws), dt, offsets=dev(at))
    assert (buf[:32] == 7).all() and (buf[32 + m * n_out:] == 7).all()
    for out in (y, z):
        for g in range(groups):
            lo, hi = at[g], at[g + 1]
            assert R.equal(out[lo:hi], R.product(xc[lo:hi], xs[lo:hi], wc[g], ws[g], dt)), ("group", g, counts[g])
        assert (out[at[-1]:] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts, behind", [([1], 0), ([0, 3], 0), ([0, 0, 0], 5), ([2, 0, 1, 0], 1), ([16, 17, 1, 0, 33], 3),
                                            ([40, 0, 65, 3], 0), ([200, 100, 0, 130], 70), ([300, 1, 600], 0)])
def test_groups(ex, counts, behind, dtype):
    check_groups(ex, counts, behind, 336, 80, dtype)


@pytest.mark.parametrize("n_in, n_out", [(144, 2500), (144, 10000), (256, 10001)])
def test_large_groups(ex, n_in, n_out):
    check_groups(ex, [700, 0, 900, 450], 30, n_in, n_out, "bf16")


def test_many_groups(ex):
    rng = np.random.default_rng(14)
    check_groups(ex, [int(c) for c in rng.integers(0, 4, 150)], 9, 64, 33, "bf16")
    check_groups(ex, [0] * 127 + [5], 0, 64, 33, "bf16")
    check_groups(ex, [int(c) for c in rng.integers(0, 90, 70)], 0, 128, 40, "fp16")
    check_groups(ex, [0] * 64 + [400] + [0] * 63, 1, 128, 40, "fp16")


@pytest.mark.parametrize("groups", [191, 192, 255, 256, 257, 1030])
def test_more_groups_than_one_batch_of_offsets(ex, groups):
    rng = np.random.default_rng([15, groups])
    check_groups(ex, [int(c) for c in rng.integers(0, 3, groups)], 2, 64, 17, "fp16")
    check_groups(ex, [0] * (groups - 1) + [3], 0, 64, 17, "bf16")
    check_groups(ex, [0] * (groups - 70) + [150] + [0] * 69, 5, 64, 17, "fp32")


def test_offsets_outside_the_rows_are_taken_as_the_nearer_end(ex):
    rng = np.random.default_rng(16)
    x = R.rows(rng, 6, 64, torch.float32)
    wc, ws = R.weight(rng, 3, 16, 64)
    y = ex.int8_linear(x.cuda(), dev(wc), dev(ws), offsets=dev(np.array([-5, 2, 4, 1 << 30], np.int32)))
    xc, xs = R.quantize(x)
    for g in range(3):
        assert R.equal(y[2 * g:2 * g + 2], R.product(xc[2 * g:2 * g + 2], xs[2 * g:2 * g + 2], wc[g], ws[g], torch.float32))


# ---- streams, graphs, workspaces ----

@pytest.mark.parametrize("m", [2, 300])
def test_on_another_stream(ex, m):
    rng = np.random.default_rng([17, m])
    x, r = (R.rows(rng, m, 512, torch.bfloat16).cuda() for _ in range(2))
    w = torch.ones(512, device="cuda")
    codes, scales = (dev(a) for a in R.weight(rng, 64, 512))
    calls = [lambda s: ex.int8_linear(x, codes, scales, stream=s), lambda s: ex.int8_quantize(x, stream=s)[0],
             lambda s: ex.int8_rms_norm(x, w, r, stream=s)[2], lambda s: ex.int8_matmul(*ex.int8_quantize(x, stream=s), codes, scales, stream=s),
             lambda s: ex.int8_dequantize(*ex.int8_quantize(x, stream=s), stream=s)]
    refs = [c(None) for c in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    given = [c(side) for c in calls]
    with torch.cuda.stream(side):
        current = [c(None) for c in calls]
    torch.cuda.synchronize()
    for a, b, ref in zip(given, current, refs):
        assert torch.equal(a, ref) and torch.equal(b, ref)


def test_two_captured_graphs_and_eager_calls(ex):
    rng = np.random.default_rng(18)
    codes, scales = (dev(a) for a in R.weight(rng, 96, 512))
    w = dev(rng.standard_normal(512).astype(np.float32))

    def step(x, r):
        c, s, h = ex.int8_rms_norm(x, w, r)
        return ex.int8_matmul(c, s, codes, scales, x.dtype), h, ex.int8_linear(h, codes, scales)
    batches = [[tuple(R.rows(rng, m, 512, torch.float16).cuda() for _ in range(2)) for _ in range(4)] for m in (3, 200)]
    refs = [[tuple(t.clone() for t in step(*xs)) for xs in batch] for batch in batches]
    graphs = []
    for batch in batches:
        held = tuple(t.clone() for t in batch[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(*held)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(*held)
        graphs.append((g, held, out))
    for i in (1, 2, 3, 0):
        for (g, held, out), batch, ref in zip(graphs, batches, refs):
            for t, s in zip(held, batch[i]):
                t.copy_(s)
            g.replay()
            eager = step(*batch[(i + 1) % 4])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, ref[i])) and all(torch.equal(a, b) for a, b in zip(eager, ref[(i + 1) % 4]))


def test_calls_on_two_streams_at_once(ex):
    rng = np.random.default_rng(19)
    codes, scales = (dev(a) for a in R.weight(rng, 512, 1040))
    xs = [R.rows(rng, m, 1040, torch.bfloat16).cuda() for m in (300, 13)]
    refs = [ex.int8_linear(x, codes, scales) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(8):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k].append(ex.int8_linear(xs[k], codes, scales))
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(torch.equal(y, refs[k]) for y in got[k])


def test_given_workspace(ex):
    rng = np.random.default_rng(20)
    x = R.rows(rng, 100, 512, torch.float16).cuda()
    codes, scales = (dev(a) for a in R.weight(rng, 64, 512))
    need = ex.int8_workspace_bytes(100, 512)
    ws = torch.full((need + 256,), 0xCD, dtype=torch.uint8, device="cuda")
    y = ex.int8_linear(x, codes, scales, workspace=ws[:need])
    assert torch.equal(y, ex.int8_linear(x, codes, scales)) and (ws[need:] == 0xCD).all()
    with pytest.raises(ex.Exl3Error, match="workspace"):
        ex.int8_linear(x, codes, scales, workspace=ws[:need - 16])


# ---- more than 2^32 elements: large tensors repeat 1024 rows ----

def test_more_than_32_bits_of_values(ex):
    rows, n = 1 << 20, 4112
    base = torch.randn((1024, n), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    x = base.repeat(rows // 1024, 1)
    assert x.numel() > 1 << 32
    w = torch.ones(n, device="cuda")
    codes, scales, added = ex.int8_rms_norm(x, w, x.clone())
    ref = ex.int8_rms_norm(base, w, base.clone())
    del x
    out, ref_out = ex.int8_dequantize(codes, scales), ex.int8_dequantize(*ref[:2])
    for i in (0, 1, 507, 508, 1016, 1022, 1023):
        for got, want in zip((codes, scales, added, out), (*ref, ref_out)):
            assert torch.equal(got[1024 * i:1024 * (i + 1)], want), i


def test_product_of_more_than_32_bits_of_outputs(ex):
    gen = torch.Generator(device="cuda").manual_seed(2)
    m, n_in, n_out = 1 << 20, 64, 4160
    base = torch.randint(-128, 128, (1024, n_in), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (n_out, n_in), generator=gen, device="cuda", dtype=torch.int8)
    y = ex.int8_matmul(base.repeat(m // 1024, 1), torch.ones(m, device="cuda"), w, torch.ones(n_out, device="cuda"))
    assert y.numel() > 1 << 32
    ref = (base.double().cpu() @ w.double().cpu().T).bfloat16().cuda()
    for i in (0, 1, 503, 504, 1007, 1022, 1023):
        assert torch.equal(y[1024 * i:1024 * (i + 1)], ref), i


@pytest.mark.parametrize("rows", [3, 20, 200, 1500])
def test_weights_of_more_than_32_bits(ex, rows):
    gen = torch.Generator(device="cuda").manual_seed(3)
    groups, n_out, n_in = 36, 8192, 16384
    w = torch.randint(-128, 128, (n_out, n_in), generator=gen, device="cuda", dtype=torch.int8).repeat(groups, 1, 1)
    assert w.numel() > 1 << 32
    w[-1] ^= 0x5A
    scales = torch.ones((groups, n_out), device="cuda")
    xc = torch.randint(-128, 128, (rows, n_in), generator=gen, device="cuda", dtype=torch.int8)
    xs = torch.ones(rows, device="cuda")
    at = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    at[-1], at[-2] = rows, 1  # one row of the last group but one, the others of the last
    y = ex.int8_matmul(xc, xs, w, scales, torch.float32, offsets=at)
    for g, a, b in ((-2, 0, 1), (-1, 1, rows)):
        assert torch.equal(y[a:b], ex.int8_matmul(xc[a:b].clone(), xs[a:b].clone(), w[g], scales[g], torch.float32)), g
    ref = (xc[1:3].double().cpu() @ w[-1].double().cpu().T).float()
    assert torch.equal(y[1:3].cpu(), ref)


# 256 x 256 and 128 x 256 tiles, several a workgroup, whole rounds of the former with the latter behind them, and groups in either
@pytest.mark.parametrize("m, n_in, n_out, dtype", [(2050, 272, 20003, "bf16"), (2050, 16, 20003, "fp32"), (1030, 144, 40001, "fp16"), (4100, 256, 5001, "fp32"),
                                                    (2048, 400, 28672, "bf16"), (2048, 272, 28669, "fp16"), (770, 1040, 28671, "fp32"), (1500, 528, 4100, "bf16")])
def test_linear_of_several_tiles_a_workgroup(ex, m, n_in, n_out, dtype):
    check_product(ex, m, n_in, n_out, dtype)


@pytest.mark.parametrize("counts, behind, n_in, n_out, dtype", [([700, 0, 900, 450, 1, 256, 257], 300, 144, 9001, "fp16"), ([3000, 20, 1500], 0, 272, 12003, "bf16"),
                                                                 ([260] * 12, 5, 400, 2816, "fp32"), ([0, 0, 5000], 0, 16, 7000, "bf16"), ([0, 0], 3000, 48, 9000, "fp32")])
def test_groups_of_several_tiles_a_workgroup(ex, counts, behind, n_in, n_out, dtype):
    check_groups(ex, counts, behind, n_in, n_out, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m, n_in, n_out", [
    (17, 528, 4090), (33, 16, 2040), (128, 1168, 1022),       # strips of 16 outputs
    (40, 528, 4001), (65, 144, 2047), (250, 1040, 1000),      # of 32
    (100, 272, 4040), (33, 48, 8190), (255, 656, 2001),       # of 64
    (250, 272, 4090), (130, 1040, 5001),                      # 64 x 64 tiles, one a CU
    (450, 144, 4090), (130, 656, 10001)])                     # and two
def test_strips_and_tiles_of_some_rows(ex, m, n_in, n_out, dtype):
    check_product(ex, m, n_in, n_out, dtype, pad=m % 2 * 8)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts, n_in, n_out", [
    ([9, 0, 17, 1, 40, 0, 3, 30], 272, 130), ([20, 11, 0, 33], 528, 1000), ([64, 0, 0, 5], 144, 2050), ([12] * 30 + [0, 100], 400, 1100),
    ([31, 0, 70, 2] * 6, 1040, 700)])
def test_groups_of_some_rows(ex, counts, n_in, n_out, dtype):
    check_groups(ex, counts, 3, n_in, n_out, dtype)
