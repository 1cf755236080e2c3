"""MXFP4 and expert operators on the GPU: calls at the edge of what they allow."""
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


@pytest.mark.parametrize("dtype", DTYPES)
def test_results_between_the_rows_of_an_input(ex, dtype):
    """Rows of a wider buffer whose rest holds the results: no byte is shared."""
    rng = np.random.default_rng(1)
    m, n_in, n_out, dt = 3, 64, 48, DTYPES[dtype]
    x = R.rows(rng, m, n_in, dt)
    codes, scales = R.weight(rng, n_out, n_in)
    buf = torch.full((m, n_in + 160), 7.0, dtype=dt, device="cuda")
    buf[:, :n_in] = x.cuda()
    y = buf.view(-1)[n_in:n_in + m * n_out].view(m, n_out)
    ex.mxfp4_linear(buf[:, :n_in], dev(codes), dev(scales), y=y)
    R.assert_product(y, R.dequantize(*R.quantize(x)), R.dequantize(codes, scales), dt)
    assert torch.equal(buf[:, :n_in].cpu(), x) and (buf[1:, n_in:] == 7).all() and (buf[0, n_in + m * n_out:] == 7).all()


def test_routing_inside_an_autograd_function(ex):
    """The way to train through the routing: grad mode is off inside, the gradients are the calls."""
    rng = np.random.default_rng(2)
    tokens, top_k, experts, n = 7, 2, 4, 24
    _, position, offsets = ex.moe_sort(dev(rng.integers(-1, experts, (tokens, top_k)).astype(np.int32)), experts)

    class Gather(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return ex.moe_gather(x, position, offsets)

        @staticmethod
        def backward(ctx, drows):
            return ex.moe_gather_backward(drows.contiguous(), position, offsets)

    class Combine(torch.autograd.Function):
        @staticmethod
        def forward(ctx, rows, weights):
            ctx.save_for_backward(rows, weights)
            return ex.moe_combine(rows, position, offsets, weights)

        @staticmethod
        def backward(ctx, dy):
            return ex.moe_combine_backward(dy.contiguous(), ctx.saved_tensors[0], position, offsets, ctx.saved_tensors[1])

    x, w, dy = (torch.from_numpy(rng.standard_normal(s)).float().cuda() for s in ((tokens, n), (tokens, top_k), (tokens, n)))
    x.requires_grad_(), w.requires_grad_()
    with pytest.raises(ex.Exl3Error, match="requires grad"):
        ex.moe_gather(x, position, offsets)
    (Combine.apply(Gather.apply(x).tanh(), w) * dy).sum().backward()
    live = (position < offsets[-1]).double().cpu()
    xd, wd = (t.detach().cpu().double().requires_grad_() for t in (x, w))
    (((live * wd)[..., None] * xd.tanh()[:, None]).sum(1) * dy.cpu().double()).sum().backward()
    # tanh, its derivative and its argument's product a few steps of fp32 each (16 allowed), then top_k products and sums; dw: n of them
    size = ((live * wd.detach()).abs().sum(1, keepdim=True) * dy.cpu().double().abs())
    assert ((x.grad.cpu().double() - xd.grad).abs() <= (16 + 2 * top_k) * 2.0 ** -24 * size + 1e-30).all()
    size = (xd.detach().tanh().abs() * dy.cpu().double().abs()).sum(1, keepdim=True).expand(tokens, top_k)
    assert ((w.grad.cpu().double() - wd.grad).abs() <= (16 + n) * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_gradients_of_weights_keep_small_terms(ex, dtype):
    """A product of 1 and 65535 of 1.875 * 2^-25, each less than half a step next to 1.  A lane
    sums every 16-byte piece's N values apart: n / (64 N) products a chain, each rounded once, then
    log2(N) sums of its own and 6 over the lanes (one step more for terms of second order)."""
    n, dt = 65536, DTYPES[dtype]
    per_piece = 128 // torch.finfo(dt).bits
    rows, dy = torch.full((1, n), 1.875 * 2.0 ** -12, dtype=dt, device="cuda"), torch.full((1, n), 2.0 ** -13, dtype=dt, device="cuda")
    rows[0, 0] = 2.0 ** 13
    pos, at = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    _, dweights = ex.moe_combine_backward(dy, rows, pos, at, torch.ones((1, 1), device="cuda"))
    ref = float((rows.double() * dy.double()).sum())
    steps = n // (64 * per_piece) + {4: 2, 8: 3}[per_piece] + 6 + 1
    assert abs(float(dweights) - ref) <= steps * 2.0 ** -24 * ref


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows, n, pad", [(2051, 1056, 0), (2051, 1056, 24), (1024, 4128, 0), (257, 8192, 8)])
def test_quantize_of_many_values(ex, dtype, rows, n, pad):
    """From 2^18 units of 8 values on a thread takes four: bit for bit, contiguous rows and slices."""
    assert rows * (n // 8) >= 1 << 18
    x = R.rows(np.random.default_rng([3, rows, pad]), rows, n + pad, DTYPES[dtype]).cuda()[:, :n]
    codes, scales = ex.mxfp4_quantize(x)
    ref_codes, ref_scales = R.quantize(x)
    assert np.array_equal(scales.cpu().numpy(), ref_scales) and np.array_equal(codes.cpu().numpy(), ref_codes)
    got = ex.mxfp4_dequantize(codes, scales, DTYPES[dtype])
    assert np.array_equal(got.cpu().double().numpy(), R.dequantize(ref_codes, ref_scales))


@pytest.mark.parametrize("m, n_out, n_in", [(1, 256, 96), (4, 256, 512), (16, 256, 672), (40, 256, 96), (256, 256, 96), (600, 256, 288),
                                            (2048, 2048, 256)])
@pytest.mark.parametrize("x_code, w_code", [(2, 2), (7, 15), (1, 3), (0, 7)])
def test_product_of_every_pair_of_scales(ex, m, n_out, n_in, x_code, w_code):
    """One product a result, of any scales: exact down to fp32's subnormals, infinite from 2^128 on, NaN for 255."""
    rng = np.random.default_rng([4, m])
    at = 17 if n_in < 200 else 130  # an odd column
    xs, ws = (rng.permutation(256)[:m] if m < 256 else np.arange(m) % 256), np.arange(n_out) % 256
    xc, wc = np.zeros((m, n_in // 2), np.uint8), np.zeros((n_out, n_in // 2), np.uint8)
    xc[:, at // 2], wc[:, at // 2] = x_code << 4 * (at & 1), w_code << 4 * (at & 1)
    x_scales, w_scales = np.full((m, n_in // 32), 127, np.uint8), np.full((n_out, n_in // 32), 127, np.uint8)
    x_scales[:, at // 32], w_scales[:, at // 32] = xs, ws
    y = ex.mxfp4_matmul(dev(xc), dev(x_scales), dev(wc), dev(w_scales), torch.float32).cpu().numpy()
    value = R.VALUES[x_code] * R.VALUES[w_code & 7] * (-1 if w_code & 8 else 1)
    with np.errstate(over="ignore", under="ignore"):
        ref = np.ldexp(value, xs[:, None] + ws[None, :] - 254).astype(np.float32)
    ref[xs == 255], ref[:, ws == 255] = np.nan, np.nan
    assert np.array_equal(y, ref, equal_nan=True)


def test_calls_on_two_streams_at_once(ex):
    rng = np.random.default_rng(5)
    codes, scales = (dev(a) for a in R.weight(rng, 512, 1056))
    xs = [R.rows(rng, m, 1056, torch.bfloat16).cuda() for m in (300, 200)]
    ids = [dev(rng.integers(-1, 40, (3000, 2)).astype(np.int32)) for _ in range(2)]
    refs = [(ex.mxfp4_linear(x, codes, scales), *ex.moe_sort(i, 40)) for x, i in zip(xs, ids)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k].append((ex.mxfp4_linear(xs[k], codes, scales), *ex.moe_sort(ids[k], 40)))
    torch.cuda.synchronize()
    for k in (0, 1):
        for outs in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(outs, refs[k]))


def test_captured_sort_of_many_slots(ex):
    rng = np.random.default_rng(6)
    cases = [rng.integers(-2, 70, (2500, 2)).astype(np.int32) for _ in range(4)]
    refs = [R.sort(ids, 64) for ids in cases]
    held = dev(cases[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ex.moe_sort(held, 64)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ex.moe_sort(held, 64)
    for i in (1, 2, 3, 0, 2):
        held.copy_(dev(cases[i]))
        graph.replay()
        eager = ex.moe_sort(dev(cases[(i + 1) % 4]), 64)
        torch.cuda.synchronize()
        for out, ref in ((got, refs[i]), (eager, refs[(i + 1) % 4])):
            assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(out, ref))


def test_temporaries_of_a_call_on_a_given_stream(ex):
    """A tensor dropped right after a call with stream= is not handed out again before that stream has read it."""
    rng = np.random.default_rng(7)
    tokens, top_k, n = 600, 2, 512
    codes, scales = (dev(a) for a in R.weight(rng, 256, n))
    _, position, offsets = ex.moe_sort(dev(rng.integers(0, 9, (tokens, top_k)).astype(np.int32)), 9)
    x, w = R.rows(rng, tokens, n, torch.bfloat16).cuda(), torch.rand((tokens, top_k), device="cuda")
    rows = ex.moe_gather(x, position, offsets)
    calls = [(lambda x, s: ex.mxfp4_linear(x, codes, scales, stream=s), (x,)), (lambda x, s: ex.mxfp4_quantize(x, stream=s)[0], (x,)),
             (lambda x, p, s: ex.moe_gather(x, p, offsets, stream=s), (x, position)),
             (lambda r, w, s: ex.moe_combine(r, position, offsets, w, stream=s), (rows, w))]
    refs = [call(*args, None) for call, args in calls]
    busy, side = torch.ones((4096, 4096), device="cuda"), torch.cuda.Stream()
    for (call, args), ref in zip(calls, refs):
        temporaries = [t.clone() for t in args]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):  # in front of the call
                busy @ busy
        got = call(*temporaries, side)
        del temporaries
        others = [torch.ones_like(t) for t in args for _ in range(4)]  # on the current stream, at once
        torch.cuda.synchronize()
        assert torch.equal(got, ref) and all(bool((t == 1).all()) for t in others)


def test_captured_calls_on_a_given_stream(ex):
    rng = np.random.default_rng(8)
    codes, scales = (dev(a) for a in R.weight(rng, 64, 512))
    xs = [R.rows(rng, 200, 512, torch.float16).cuda() for _ in range(3)]
    refs = [ex.mxfp4_linear(x, codes, scales) for x in xs]
    held, graph = xs[0].clone(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = ex.mxfp4_linear(held, codes, scales, stream=torch.cuda.current_stream())
    for i in (1, 2, 0, 1):
        held.copy_(xs[i])
        graph.replay()
        eager = ex.mxfp4_linear(xs[(i + 1) % 3].clone(), codes, scales, stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert torch.equal(y, refs[i]) and torch.equal(eager, refs[(i + 1) % 3])
