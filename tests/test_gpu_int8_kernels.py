"""8-bit products in each kernel that makes them: groups of every number that the tiles' search treats in its own
way, and the longest inputs."""
import numpy as np
import pytest
import torch

import _int8_cases as C
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


@pytest.mark.parametrize("kernel, groups, rows, behind, n_in, n_out, dtype", [(k, *c) for cases in (C.GROUPED, C.FEW_GROUPED) for k, cs in cases.items() for c in cs])
def test_groups(ex, kernel, groups, rows, behind, n_in, n_out, dtype):
    """Uneven groups, empty ones whose weights' scales are NaN, rows of no group that hold NaN, results inside a larger buffer."""
    dt, counts = DTYPES[dtype], C.uneven(groups, rows - behind, 0)
    rng = np.random.default_rng([32, groups, rows, n_in, n_out])
    x = R.rows(rng, rows, n_in, dt)
    x[rows - behind:] = float("nan")
    wc, ws = R.weight(rng, groups, n_out, n_in)
    ws[[g for g, c in enumerate(counts) if c == 0]] = np.nan
    at = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    xc, xs = R.quantize(x)
    buf = torch.full((rows * n_out + 64,), 7.0, dtype=dt, device="cuda")
    weight = dev(wc), dev(ws)
    y = ex.int8_linear(x.cuda(), *weight, offsets=dev(at), y=buf[32:32 + rows * n_out].view(rows, n_out))
    xc, xs = dev(xc), dev(xs)
    z = ex.int8_matmul(xc, xs, *weight, dt, offsets=dev(at))
    assert (buf[:32] == 7).all() and (buf[32 + rows * n_out:] == 7).all()
    for g, c in enumerate(counts):
        if c:
            lo, hi = at[g], at[g + 1]
            acc = xc[lo:hi].double() @ weight[0][g].double().T  # whole numbers below 2^53: exact
            ref = (acc.float() * xs[lo:hi, None] * weight[1][g]).to(dt)
            assert torch.equal(y[lo:hi], ref) and torch.equal(z[lo:hi], ref), ("group", g, c)
    assert not y[at[-1]:].any() and not z[at[-1]:].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_in, n_out", [(64, 40), (4096, 72), (16384, 20), (28672, 33)])
@pytest.mark.parametrize("rows, ends", [(1, (0, 0)), (1, (0, 1)), (3, (0, 2)), (4, (0, 0)), (4, (0, 4)), (4, (-3, 9)), (9, (0, 5)), (70, (0, 1))])
def test_one_group_and_rows_behind_it(ex, rows, ends, n_in, n_out, dtype):
    """Few rows are quantised inside the product, with offsets too."""
    dt, kept = DTYPES[dtype], max(0, min(ends[1], rows))
    rng = np.random.default_rng([34, rows, n_in])
    x = R.rows(rng, rows, n_in, dt)
    x[kept:] = float("inf")
    wc, ws = R.weight(rng, 1, n_out, n_in)
    y = ex.int8_linear(x.cuda(), dev(wc), dev(ws), offsets=torch.tensor(ends, dtype=torch.int32, device="cuda"))
    xc, xs = R.quantize(x[:kept])
    assert R.equal(y[:kept], R.product(xc, xs, wc[0], ws[0], dt)) and not y[kept:].any()


@pytest.mark.parametrize("kernel, m, n_in, n_out, dtype", [(k, *c) for k, cs in C.FEW.items() for c in cs])
def test_few_rows_of_many_outputs(ex, kernel, m, n_in, n_out, dtype):
    dt = DTYPES[dtype]
    rng = np.random.default_rng([33, m, n_in, n_out])
    x = R.rows(rng, m, n_in + 8, dt).cuda()[:, :n_in]
    wc, ws = (dev(a) for a in R.weight(rng, n_out, n_in))
    xc, xs = (dev(a) for a in R.quantize(x))
    acc = xc.double() @ wc.double().T  # whole numbers below 2^53: exact
    ref = (acc.float() * xs[:, None] * ws).to(dt)
    buf = torch.full((m * n_out + 64,), 7.0, dtype=dt, device="cuda")
    y = ex.int8_linear(x, wc, ws, y=buf[32:32 + m * n_out].view(m, n_out))
    assert torch.equal(y, ref) and (buf[:32] == 7).all() and (buf[32 + m * n_out:] == 7).all()
    assert torch.equal(ex.int8_matmul(xc, xs, wc, ws, dt), ref)


@pytest.mark.parametrize("kernel", C.LONG)
def test_the_longest_inputs(ex, kernel):
    """Sums next to 2^31, and random codes against whole sums in 64 bits."""
    (m, n_out), n_in = C.LONG[kernel], C.LONGEST
    one_m, one_n = torch.ones(m, device="cuda"), torch.ones(n_out, device="cuda")
    xc, wc = (torch.full((k, n_in), -128, dtype=torch.int8, device="cuda") for k in (m, n_out))
    wc[3] = wc[-1] = 127
    y = ex.int8_matmul(xc, one_m, wc, one_n, torch.float32)
    ref = torch.full((n_out,), float(2 ** 14 * n_in), device="cuda")
    ref[3] = ref[-1] = -float(128 * 127 * n_in)
    assert bool((y == ref).all())
    del y
    gen = torch.Generator(device="cuda").manual_seed(7)
    for t in (xc, wc):
        for a in range(0, t.shape[0], 1024):  # in parts, for the generator's 32-bit offsets
            t[a:a + 1024].random_(-128, 128, generator=gen)
    y = ex.int8_matmul(xc, one_m, wc, one_n, torch.float32)
    rows = [i for i in dict.fromkeys((0, 1, 17, m // 2, m - 2, m - 1))]
    outs = [i for i in dict.fromkeys((0, 1, 15, 16, 31, 63, 100, 127, n_out // 2, n_out // 2 + 1, n_out - 17, n_out - 2, n_out - 1)) if i < n_out]
    ref = (xc[rows].cpu().double() @ wc[outs].cpu().double().T).float()  # whole numbers below 2^53
    assert torch.equal(y[rows][:, outs].cpu(), ref)
