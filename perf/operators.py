"""The MXFP4 and mixture-of-experts operators at the sizes they are used at.

Five operators: `quantize` (a tensor to microscaled 4-bit codes and back to the
values they stand for), `linear` (16- or 32-bit rows times an MXFP4 weight, the
rows quantised on the way in), `experts` (the same product with one weight per
group of rows), `dispatch` (tokens sorted by expert, their rows gathered, and
the gather's gradient) and `combine` (the experts' rows back to the tokens with
the router's weights, and its gradients).

MXFP4: 32 consecutive values share a power-of-two scale 2^(b - 127), b =
max(floor(log2(amax)) - 2 + 127, 0); each is held as sign, two exponent bits and one
mantissa bit (0, .5, 1, 1.5, 2, 3, 4, 6), rounded to nearest, ties to even, and
saturated at 6.  The code of an even position sits in the low half of its byte.
"""
import math

import torch

own = False

BLOCK = 32
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token's activations of a 4096-wide layer: latency alone
        {"name": "quantize-token", "op": "quantize", "dtype": "bf16", "rows": 1, "n": 4096, "pad": 0},
        # the gate and up weight of a 70B-shaped layer, once when a model is loaded
        {"name": "quantize-weight", "op": "quantize", "dtype": "fp16", "rows": 28672, "n": 8192, "pad": 0},
        # one token through a square attention projection
        {"name": "linear-token", "op": "linear", "dtype": "fp16", "m": 1, "n_in": 4096, "n_out": 4096, "pad": 0},
        # a decode batch of 13 sequences through an 8B-shaped down projection
        {"name": "linear-batch", "op": "linear", "dtype": "bf16", "m": 13, "n_in": 14336, "n_out": 4096, "pad": 0},
        # a short prompt of odd length, an odd number of blocks and of outputs, rows that are a slice of a wider buffer
        {"name": "linear-ragged", "op": "linear", "dtype": "fp32", "m": 333, "n_in": 2080, "n_out": 1001, "pad": 96},
        # a prompt of 2048 tokens through a 70B-shaped gate and up
        {"name": "linear-prompt", "op": "linear", "dtype": "bf16", "m": 2048, "n_in": 8192, "n_out": 28672, "pad": 0},
        # three tokens, two of eight experts each: decode, bound by the weights of the experts that are hit
        {"name": "experts-decode", "op": "experts", "dtype": "bf16", "tokens": 3, "top_k": 2, "experts": 8,
         "n_in": 4096, "n_out": 14336, "dropped": 0.0},
        # a prompt over many small experts, uneven loads, some slots dropped
        {"name": "experts-prompt", "op": "experts", "dtype": "fp16", "tokens": 2048, "top_k": 8, "experts": 64,
         "n_in": 2048, "n_out": 2816, "dropped": 0.02},
        # routing of one decode step
        {"name": "dispatch-decode", "op": "dispatch", "dtype": "bf16", "tokens": 5, "top_k": 2, "experts": 8, "n": 4096,
         "dropped": 0.0},
        # routing of a packed batch of prompts whose padding tokens have no expert
        {"name": "dispatch-prompt", "op": "dispatch", "dtype": "fp16", "tokens": 8192, "top_k": 8, "experts": 64, "n": 2048,
         "dropped": 0.05},
        # a short ragged batch in full precision
        {"name": "combine-short", "op": "combine", "dtype": "fp32", "tokens": 67, "top_k": 3, "experts": 20, "n": 1000,
         "dropped": 0.1},
        # a training step's batch of tokens
        {"name": "combine-train", "op": "combine", "dtype": "bf16", "tokens": 4096, "top_k": 2, "experts": 8, "n": 4096,
         "dropped": 0.02},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "experts", "experts", "dispatch", "combine"])
    dtype = rng.choice(["fp16", "bf16", "bf16", "fp32"])
    if op == "quantize":
        n = BLOCK * _log(rng, 1, 896)
        rows = _log(rng, 1, min(28672, 28672 * 8192 // (n * SIZE[dtype])))
        return {"op": op, "dtype": dtype, "rows": rows, "n": n, "pad": rng.choice([0, 0, 8, 64])}
    if op == "linear":
        n_in, n_out = BLOCK * _log(rng, 2, 448), _log(rng, 7, 28672)
        m = _log(rng, 1, min(2048, 2048 * 8192 * 28672 // (n_in * n_out)))
        return {"op": op, "dtype": dtype, "m": m, "n_in": n_in, "n_out": n_out, "pad": rng.choice([0, 0, 8, 64])}
    experts = _log(rng, 2, 128)
    top_k = rng.randint(1, min(8, experts))
    tokens = _log(rng, 1, 8192 if op == "dispatch" else 2048)
    dropped = rng.choice([0.0, 0.0, 0.03, 0.2])
    if op == "experts":
        n_in = BLOCK * _log(rng, 4, 128)
        n_out = _log(rng, 16, min(14336, 64 * 2048 * 2816 // (experts * n_in)))
        return {"op": op, "dtype": dtype, "tokens": tokens, "top_k": top_k, "experts": experts, "n_in": n_in, "n_out": n_out,
                "dropped": dropped}
    return {"op": op, "dtype": dtype, "tokens": tokens, "top_k": top_k, "experts": experts, "n": 8 * _log(rng, 8, 512),
            "dropped": dropped}


# ---- inputs ----

def _rows(gen, rows, n, dtype, pad=0):
    """Activations: normal, a few channels an order of magnitude larger, rows of different size."""
    x = torch.randn((rows, n + pad), generator=gen, device="cuda", dtype=torch.float32)
    channel = torch.rand((n + pad,), generator=gen, device="cuda")
    x *= torch.where(channel < 0.01, 12.0, 1.0)
    x *= torch.exp2(torch.randn((rows, 1), generator=gen, device="cuda"))
    x = x.to(dtype)
    return x[:, :n] if pad else x


def _weights(gen, rows, n):
    """An MXFP4 weight whose values have a standard deviation of about n^-1/2."""
    w = torch.randn((rows, n), generator=gen, device="cuda", dtype=torch.float32) * n ** -0.5
    return _quantize(w)


def _route(gen, case):
    """Distinct experts per token, some of them popular; a dropped slot has expert -1."""
    tokens, top_k, experts = case["tokens"], case["top_k"], case["experts"]
    score = torch.rand((tokens, experts), generator=gen, device="cuda") + 0.5 * torch.rand((experts,), generator=gen, device="cuda")
    ids = score.argsort(dim=1, descending=True)[:, :top_k].to(torch.int32)
    return torch.where(torch.rand((tokens, 1), generator=gen, device="cuda") < case["dropped"], -1, ids).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = {"op": op, "dtype": dtype}
    if op == "quantize":
        s["x"] = _rows(gen, case["rows"], case["n"], dtype, case["pad"])
    elif op == "linear":
        s["x"] = _rows(gen, case["m"], case["n_in"], dtype, case["pad"])
        s["codes"], s["scales"] = _weights(gen, case["n_out"], case["n_in"])
    elif op == "experts":
        ids = _route(gen, case).reshape(-1)
        s["x"] = _rows(gen, ids.numel(), case["n_in"], dtype)
        codes, scales = [], []
        for _ in range(case["experts"]):
            c, b = _weights(gen, case["n_out"], case["n_in"])
            codes.append(c)
            scales.append(b)
        s["codes"], s["scales"] = torch.stack(codes), torch.stack(scales)
        count = (ids[:, None] == torch.arange(case["experts"], device="cuda")).sum(0)
        s["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)
    else:
        s["ids"], s["top_k"], s["experts"] = _route(gen, case), case["top_k"], case["experts"]
        slots, n = case["tokens"] * case["top_k"], case["n"]
        if op == "dispatch":
            s["x"] = _rows(gen, case["tokens"], n, dtype)
            s["dy"] = _rows(gen, slots, n, dtype)
        else:
            _, s["position"], s["offsets"] = _sort(s["ids"], case["experts"])
            s["x"] = _rows(gen, slots, n, dtype)
            s["dy"] = _rows(gen, case["tokens"], n, dtype)
            s["weights"] = torch.softmax(torch.randn(s["ids"].shape, generator=gen, device="cuda"), dim=1)
    return s


# ---- plain forms ----

def _quantize(x):
    """Codes uint8 [rows, n / 2] and scales uint8 [rows, n / 32]."""
    v = x.float().unflatten(-1, (-1, BLOCK))
    amax = v.abs().amax(-1, keepdim=True)
    b = ((amax.view(torch.int32) >> 23) - 2).clamp(min=0)  # the amax's own exponent, less that of the largest code
    inverse = ((254 - b) << 23).view(torch.float32)
    a = v.abs() * inverse
    a = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2))).clamp(max=6)
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + 8 * torch.signbit(v).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), b.squeeze(-1).to(torch.uint8)


def _dequantize(codes, scales):
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), device=codes.device)
    code = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).int()
    power = torch.where(scales == 0, 1 << 22, scales.int() << 23).view(torch.float32)  # 2^(b - 127), subnormal at b = 0
    return (table[code].unflatten(-1, (-1, BLOCK)) * power.unsqueeze(-1)).flatten(-2)


def _sort(ids, experts):
    """Slots in the order of their experts, each expert's in the order of the tokens, dropped ones last:
    order[s] is the slot at place s, position its inverse, offsets the experts' first places."""
    flat = ids.reshape(-1).long()
    group = torch.where((flat < 0) | (flat >= experts), experts, flat)
    hit = (group == torch.arange(experts + 1, device=ids.device)[:, None]).to(torch.int32)
    before = hit.cumsum(1)
    start = torch.cat([before.new_zeros(1), before[:, -1].cumsum(0)])
    place = start[group] + before.gather(0, group[None]).squeeze(0) - 1
    order = torch.empty_like(place)
    order[place] = torch.arange(flat.numel(), device=ids.device)
    return order.to(torch.int32), place.to(torch.int32).reshape(ids.shape), start[:-1].to(torch.int32)


def _plain(s):
    op, dtype = s["op"], s["dtype"]
    if op == "quantize":
        codes, scales = _quantize(s["x"])
        return _dequantize(codes, scales).to(dtype)
    if op == "linear":
        x = _dequantize(*_quantize(s["x"]))
        return (x @ _dequantize(s["codes"], s["scales"]).t()).to(dtype)
    if op == "experts":
        x, at = _dequantize(*_quantize(s["x"])), s["offsets"].tolist()
        y = x.new_zeros((x.shape[0], s["codes"].shape[1]))
        for e in range(len(at) - 1):
            if at[e + 1] > at[e]:
                y[at[e]:at[e + 1]] = x[at[e]:at[e + 1]] @ _dequantize(s["codes"][e], s["scales"][e]).t()
        return y.to(dtype)
    if op == "dispatch":
        order, position, offsets = _sort(s["ids"], s["experts"])
        used = (torch.arange(order.numel(), device=order.device) < offsets[-1])[:, None]
        rows = torch.where(used, s["x"][(order // s["top_k"]).long()], 0)
        dx = torch.where(used, s["dy"].float(), 0.0)[position.long()].sum(1).to(dtype)
        return order, position, offsets, rows, dx
    position, weights, dy = s["position"].long(), s["weights"], s["dy"].float()
    used = position < s["offsets"][-1]
    rows = torch.where(used[..., None], s["x"].float()[position], 0.0)
    weights = torch.where(used, weights, 0.0)
    y = (weights[..., None] * rows).sum(1)
    drows = torch.empty(s["x"].shape, device=dy.device)
    drows[position.reshape(-1)] = (weights[..., None] * dy[:, None]).flatten(0, 1)
    return y.to(dtype), drows.to(dtype), (rows * dy[:, None]).sum(-1)


# ---- the framework's operators ----

def _own(s):
    import decode_gemm_exl3_amd as ex
    op = s["op"]
    if op == "quantize":
        codes, scales = ex.mxfp4_quantize(s["x"])
        return ex.mxfp4_dequantize(codes, scales, s["dtype"])
    if op == "linear":
        return ex.mxfp4_linear(s["x"], s["codes"], s["scales"])
    if op == "experts":
        return ex.mxfp4_linear(s["x"], s["codes"], s["scales"], offsets=s["offsets"])
    if op == "dispatch":
        order, position, offsets = ex.moe_sort(s["ids"], s["experts"])
        rows = ex.moe_gather(s["x"], position, offsets)
        return order, position, offsets, rows, ex.moe_gather_backward(s["dy"], position, offsets)
    y = ex.moe_combine(s["x"], s["position"], s["offsets"], s["weights"])
    return (y, *ex.moe_combine_backward(s["dy"], s["x"], s["position"], s["offsets"], s["weights"]))


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ----

def work(case):
    op, size = case["op"], SIZE[case["dtype"]]
    if op == "quantize":
        elems = case["rows"] * case["n"]
        return {"bytes": 2 * elems * size, "flops": 4 * elems}
    if op == "linear":
        m, k, n = case["m"], case["n_in"], case["n_out"]
        return {"bytes": m * k * size + n * k // 2 + n * k // BLOCK + m * n * size, "flops": 2 * m * n * k}
    slots, experts = case["tokens"] * case["top_k"], case["experts"]
    used = slots * (1 - case["dropped"])
    if op == "experts":
        k, n = case["n_in"], case["n_out"]
        hit = experts * (1 - (1 - case["top_k"] / experts) ** (case["tokens"] * (1 - case["dropped"])))
        return {"bytes": used * k * size + hit * (n * k // 2 + n * k // BLOCK) + slots * n * size, "flops": 2 * used * n * k}
    n = case["n"]
    if op == "dispatch":
        return {"bytes": 4 * slots * 3 + 4 * experts + (case["tokens"] * n + slots * n + used * n + case["tokens"] * n) * size,
                "flops": used * n}
    return {"bytes": 4 * slots * 3 + (2 * case["tokens"] * n + used * n + slots * n) * size, "flops": 5 * used * n}


# ---- the definition in 64 bits ----

def _power(e):
    """2^e in 64 bits for whole e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(x):
    """The values of the MXFP4 quantisation of x, in 64 bits: nearest code by the midpoints, a tie to the even code."""
    v = x.double().reshape(-1, BLOCK)
    exponent = torch.frexp(v.abs().amax(1, keepdim=True))[1] - 1
    shared = _power(torch.where(v.abs().amax(1, keepdim=True) == 0, -127, (exponent - 2).clamp(min=-127)))
    a = v.abs() / shared
    q = torch.zeros_like(a)
    for k in range(7):
        middle = (VALUES[k] + VALUES[k + 1]) / 2
        q = torch.where(a >= middle if k % 2 else a > middle, VALUES[k + 1], q)
    return (torch.sign(v) * q * shared).reshape(x.shape)


def _exact_weight(codes, scales):
    out = torch.empty((codes.shape[0], codes.shape[1] * 2), device=codes.device, dtype=torch.float64)
    value = torch.tensor(VALUES, device=codes.device, dtype=torch.float64)
    for half, code in enumerate((codes % 16, codes // 16)):
        out[:, half::2] = value[(code % 8).long()] * (1.0 - 2.0 * (code // 8).double())
    return out * _power(scales.int() - 127).repeat_interleave(BLOCK, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_values(s["x"])
    if op == "linear":
        return torch.matmul(_exact_values(s["x"]), _exact_weight(s["codes"], s["scales"]).transpose(0, 1).contiguous())
    if op == "experts":
        x, at = _exact_values(s["x"]), s["offsets"].tolist()
        y = [torch.matmul(x[lo:hi], _exact_weight(s["codes"][e], s["scales"][e]).transpose(0, 1).contiguous())
             for e, (lo, hi) in enumerate(zip(at[:-1], at[1:]))]
        return torch.cat(y + [x.new_zeros((x.shape[0] - at[-1], s["codes"].shape[1]))])
    ids = s["ids"].reshape(-1).long()
    group = torch.where(ids < 0, case["experts"], ids)
    order = torch.sort(group, stable=True)[1]
    position = torch.argsort(order).reshape(s["ids"].shape)
    offsets = torch.searchsorted(group[order].contiguous(), torch.arange(case["experts"] + 1, device="cuda"))
    last = int(offsets[-1])
    token = order // case["top_k"]
    if op == "dispatch":
        rows = s["x"].double()[token]
        rows[last:] = 0
        dx = torch.zeros(s["x"].shape, device="cuda", dtype=torch.float64)
        for j in range(case["top_k"]):
            at = position[:, j]
            dx += torch.where((at < last)[:, None], s["dy"].double()[at], 0.0)
        return order.int(), position.int(), offsets.int(), rows, dx
    x, dy, weight = s["x"].double(), s["dy"].double(), s["weights"].double().reshape(-1)
    y, drows, dweights = torch.zeros_like(dy), torch.zeros_like(x), torch.zeros_like(weight)
    for j in range(case["top_k"]):
        at, slot = position[:, j], torch.arange(case["tokens"], device="cuda") * case["top_k"] + j
        keep = (at < last)[:, None]
        y += torch.where(keep, weight[slot][:, None] * x[at], 0.0)
        drows[at] = torch.where(keep, weight[slot][:, None] * dy, 0.0)
        dweights[slot] = torch.where(keep, x[at] * dy, 0.0).sum(1)
    return y, drows, dweights.reshape(s["ids"].shape)
