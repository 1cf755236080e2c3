"""The 8-bit integer operators and the experts' balance loss at the sizes they are used at.

Five operators: `norm` (a root-mean-square norm with the residual's addition, its
result in 8 bits with a scale for each row), `project` (that norm and the product
that takes its 8-bit rows), `linear` (16- or 32-bit rows times an 8-bit weight, the
rows quantised on the way in), `experts` (the same product with one weight per group
of rows) and `balance` (the loss that evens out a router's experts, their counts and
the loss's gradient to the router's logits).

Eight bits: a row of values v with the largest magnitude A is held as the codes
round(127 v / A), ties to the even one, and the scale A / 127; a weight's rows are its
outputs.  A product sums codes as whole numbers and takes both scales at the end.
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}


def listed():
    return [
        # one token between two sublayers of a 4096-wide model: latency alone
        {"name": "norm-token", "op": "norm", "dtype": "bf16", "rows": 1, "n": 4096, "pad": 0, "residual": True},
        # a packed batch of prompts between two sublayers of a 70B-shaped model
        {"name": "norm-prompt", "op": "norm", "dtype": "fp16", "rows": 8192, "n": 8192, "pad": 0, "residual": True},
        # a decode batch of 13 sequences: norm, then an 8B-shaped query, key and value projection
        {"name": "project-batch", "op": "project", "dtype": "bf16", "m": 13, "n_in": 4096, "n_out": 6144, "pad": 0, "residual": True},
        # a prompt of 1000 tokens: norm, then an 8B-shaped gate and up projection
        {"name": "project-prompt", "op": "project", "dtype": "bf16", "m": 1000, "n_in": 4096, "n_out": 28672, "pad": 0, "residual": True},
        # one token through a square attention projection
        {"name": "linear-token", "op": "linear", "dtype": "fp16", "m": 1, "n_in": 4096, "n_out": 4096, "pad": 0},
        # the same 13 sequences through an 8B-shaped down projection
        {"name": "linear-batch", "op": "linear", "dtype": "bf16", "m": 13, "n_in": 14336, "n_out": 4096, "pad": 0},
        # a short prompt of odd length, an odd number of 16-byte pieces and of outputs, rows that are a slice of a wider buffer
        {"name": "linear-ragged", "op": "linear", "dtype": "fp32", "m": 333, "n_in": 2064, "n_out": 1001, "pad": 96},
        # a prompt of 2048 tokens through a 70B-shaped gate and up
        {"name": "linear-prompt", "op": "linear", "dtype": "bf16", "m": 2048, "n_in": 8192, "n_out": 28672, "pad": 0},
        # three tokens, two of eight experts each: decode, bound by the weights of the experts that are hit
        {"name": "experts-decode", "op": "experts", "dtype": "bf16", "tokens": 3, "top_k": 2, "experts": 8,
         "n_in": 4096, "n_out": 14336, "dropped": 0.0},
        # a prompt over many small experts, uneven loads, some slots dropped
        {"name": "experts-prompt", "op": "experts", "dtype": "fp16", "tokens": 2048, "top_k": 8, "experts": 64,
         "n_in": 2048, "n_out": 2816, "dropped": 0.02},
        # a short ragged batch in full precision, some of it padding
        {"name": "balance-short", "op": "balance", "dtype": "fp32", "tokens": 67, "top_k": 3, "experts": 20, "dropped": 0.1},
        # a training step's batch of tokens over many experts
        {"name": "balance-train", "op": "balance", "dtype": "bf16", "tokens": 32768, "top_k": 8, "experts": 256, "dropped": 0.02},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "project", "linear", "linear", "experts", "experts", "balance"])
    dtype = rng.choice(["fp16", "bf16", "bf16", "fp32"])
    if op == "norm":
        n = 16 * _log(rng, 2, 1024)
        rows = _log(rng, 1, min(65536, 8192 * 8192 * 2 // (n * SIZE[dtype])))
        return {"op": op, "dtype": dtype, "rows": rows, "n": n, "pad": rng.choice([0, 0, 8, 64]), "residual": rng.random() < 0.8}
    if op in ("project", "linear"):
        n_in, n_out = 16 * _log(rng, 4, 896), _log(rng, 7, 28672)
        m = _log(rng, 1, min(4096, 2048 * 8192 * 28672 // (n_in * n_out)))
        case = {"op": op, "dtype": dtype, "m": m, "n_in": n_in, "n_out": n_out, "pad": rng.choice([0, 0, 8, 64])}
        return {**case, "residual": rng.random() < 0.8} if op == "project" else case
    experts = _log(rng, 2, 128 if op == "experts" else 512)
    top_k = rng.randint(1, min(8, experts))
    tokens = _log(rng, 1, 2048 if op == "experts" else 32768)
    dropped = rng.choice([0.0, 0.0, 0.03, 0.2])
    if op == "experts":
        n_in = 16 * _log(rng, 8, 256)
        n_out = _log(rng, 16, min(14336, 64 * 2048 * 2816 // (experts * n_in)))
        return {"op": op, "dtype": dtype, "tokens": tokens, "top_k": top_k, "experts": experts, "n_in": n_in, "n_out": n_out,
                "dropped": dropped}
    tokens = min(tokens, 32768 * 256 * 2 // (experts * SIZE[dtype]))
    return {"op": op, "dtype": dtype, "tokens": tokens, "top_k": top_k, "experts": experts, "dropped": dropped}


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
    """An 8-bit weight whose values have a standard deviation of about n^-1/2."""
    return _quantize(torch.randn((rows, n), generator=gen, device="cuda", dtype=torch.float32) * n ** -0.5)


def _route(gen, case, score):
    """The experts with the largest scores, distinct for a token; a dropped slot has expert -1: all of a
    padding token's, and now and then one that its expert has no room for."""
    ids = score.argsort(dim=1, descending=True)[:, :case["top_k"]].to(torch.int32)
    ids = torch.where(torch.rand((case["tokens"], 1), generator=gen, device="cuda") < case["dropped"], -1, ids)
    return torch.where(torch.rand(ids.shape, generator=gen, device="cuda") < case["dropped"] / 4, -1, ids).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = {"op": op, "dtype": dtype}
    if op in ("norm", "project"):
        rows, n = (case["rows"], case["n"]) if op == "norm" else (case["m"], case["n_in"])
        s["x"] = _rows(gen, rows, n, dtype, case["pad"])
        s["residual"] = 2 * _rows(gen, rows, n, dtype) if case["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn((n,), generator=gen, device="cuda")).to(dtype)
        if op == "project":
            s["codes"], s["scales"] = _weights(gen, case["n_out"], n)
    elif op == "linear":
        s["x"] = _rows(gen, case["m"], case["n_in"], dtype, case["pad"])
        s["codes"], s["scales"] = _weights(gen, case["n_out"], case["n_in"])
    else:
        popular = torch.randn((case["experts"],), generator=gen, device="cuda")
        score = 1.5 * torch.randn((case["tokens"], case["experts"]), generator=gen, device="cuda") + 0.5 * popular
        if op == "balance":
            s["logits"] = score.to(dtype)
            s["ids"] = _route(gen, case, s["logits"].float())
            # a loss's own gradient: one, or the scale that training in 16 bits of float16 needs
            s["dloss"] = torch.full((), 65536.0 if case["dtype"] == "fp16" else 1.0, device="cuda")
            return s
        ids = _route(gen, case, score).reshape(-1)
        s["x"] = _rows(gen, ids.numel(), case["n_in"], dtype)
        codes, scales = [], []
        for _ in range(case["experts"]):
            c, b = _weights(gen, case["n_out"], case["n_in"])
            codes.append(c)
            scales.append(b)
        s["codes"], s["scales"] = torch.stack(codes), torch.stack(scales)
        count = (ids[:, None] == torch.arange(case["experts"], device="cuda")).sum(0)
        s["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)
    return s


# ---- plain forms ----

def _codes(v, largest):
    """127 v / largest to the nearest whole number; in 64 bits, as ties are common (half of the largest, say)."""
    return torch.where(largest > 0, torch.round(127 * v.double() / largest.double()), 0.0).to(torch.int8)


def _quantize(x):
    """Codes int8 [rows, n] and scales fp32 [rows]."""
    v = x.float()
    largest = v.abs().amax(-1, keepdim=True)
    return _codes(v, largest), (largest.double() / 127).float().squeeze(-1)


def _norm(s):
    """Codes and scales of the norm, and the sum of x and the residual."""
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["dtype"])
    u = h.float() * s["weight"].float()
    largest = u.abs().amax(-1, keepdim=True)
    mean = h.double().square().mean(-1, keepdim=True)
    scale = largest.double() / (127 * torch.sqrt(mean + EPS))
    return _codes(u, largest), scale.float().squeeze(-1), None if s["residual"] is None else h


def _product(xc, xs, wc, ws):
    return (xc.float() @ wc.float().t()) * xs[:, None] * ws


def _plain(s):
    op, dtype = s["op"], s["dtype"]
    if op in ("norm", "project"):
        codes, scales, added = _norm(s)
        y = codes.float() * scales[:, None] if op == "norm" else _product(codes, scales, s["codes"], s["scales"])
        return (y.to(dtype),) if added is None else (y.to(dtype), added)
    if op == "linear":
        return _product(*_quantize(s["x"]), s["codes"], s["scales"]).to(dtype)
    if op == "experts":
        codes, scales = _quantize(s["x"])
        at = s["offsets"].tolist()
        y = torch.zeros((codes.shape[0], s["codes"].shape[1]), device=codes.device)
        for e in range(len(at) - 1):
            if at[e + 1] > at[e]:
                y[at[e]:at[e + 1]] = _product(codes[at[e]:at[e + 1]], scales[at[e]:at[e + 1]], s["codes"][e], s["scales"][e])
        return y.to(dtype)
    logits, ids = s["logits"].float(), s["ids"]
    experts, top_k = logits.shape[1], ids.shape[1]
    kept = (ids >= 0) & (ids < experts)
    counts = torch.zeros(experts + 1, device=ids.device, dtype=torch.int32)
    counts.scatter_add_(0, torch.where(kept, ids, experts).reshape(-1).long(), torch.ones_like(ids).reshape(-1))
    valid = kept.any(1)
    tokens = valid.sum()
    counts[experts] = tokens
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    p = torch.where(valid[:, None], e / e.sum(1, keepdim=True), 0.0)
    of = tokens.clamp(min=1).float()
    share = counts[:experts].float() / (of * top_k)
    loss = experts * (share * (p.sum(0) / of)).sum()
    dlogits = s["dloss"] * (experts / of) * p * (share - (p * share).sum(1, keepdim=True))
    return loss, counts, dlogits.to(dtype)


# ---- the framework's operators ----

def _own(s):
    import decode_gemm_exl3_amd as ex
    op = s["op"]
    if op in ("norm", "project"):
        codes, scales, *added = ex.int8_rms_norm(s["x"], s["weight"], s["residual"], eps=EPS)
        if op == "norm":
            return (ex.int8_dequantize(codes, scales, s["dtype"]), *added)
        return (ex.int8_matmul(codes, scales, s["codes"], s["scales"], s["dtype"]), *added)
    if op == "linear":
        return ex.int8_linear(s["x"], s["codes"], s["scales"])
    if op == "experts":
        return ex.int8_linear(s["x"], s["codes"], s["scales"], offsets=s["offsets"])
    loss, counts = ex.moe_balance_loss(s["logits"], s["ids"])
    return loss, counts, ex.moe_balance_loss_backward(s["dloss"], s["logits"], s["ids"], counts)


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ----

def work(case):
    op, size = case["op"], SIZE[case["dtype"]]
    if op == "norm":
        elems = case["rows"] * case["n"]
        return {"bytes": (4 if case["residual"] else 2) * elems * size + case["n"] * size, "flops": 8 * elems}
    if op in ("project", "linear"):
        m, k, n = case["m"], case["n_in"], case["n_out"]
        rows = 3 if op == "project" and case["residual"] else 1
        return {"bytes": rows * m * k * size + n * k + 4 * n + m * n * size, "flops": 2 * m * n * k}
    slots, experts = case["tokens"] * case["top_k"], case["experts"]
    if op == "experts":
        k, n, used = case["n_in"], case["n_out"], slots * (1 - case["dropped"])
        hit = experts * (1 - (1 - case["top_k"] / experts) ** (case["tokens"] * (1 - case["dropped"])))
        return {"bytes": used * k * size + hit * (n * k + 4 * n) + slots * n * size, "flops": 2 * used * n * k}
    elems = case["tokens"] * experts
    return {"bytes": 2 * elems * size + 4 * slots + 4 * experts, "flops": 12 * elems}


# ---- the definition in 64 bits ----

def _nearest(a):
    """The whole number nearest to each of a, a tie's even one."""
    low = torch.floor(a)
    odd = torch.remainder(low, 2) == 1
    up = (a - low > 0.5) | ((a - low == 0.5) & odd)
    return low + up.double()


def _eight_bits(v, factor=1.0):
    """What v's codes and scales stand for, the scales times `factor`."""
    largest = torch.max(v.abs(), dim=1, keepdim=True)[0]
    codes = _nearest(127 * v / torch.where(largest == 0, 1.0, largest))
    return codes * (largest * factor / 127)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "project"):
        x, total = s["x"].double(), None
        if s["residual"] is not None:
            total = x + s["residual"].double()
            x = total.to(s["dtype"]).double()
        power = (x * x).sum(1, keepdim=True) / x.shape[1]
        y = _eight_bits(x * s["weight"].double(), torch.pow(power + EPS, -0.5))
        if op == "project":
            y = torch.matmul(y, (s["codes"].double() * s["scales"].double().unsqueeze(1)).transpose(0, 1).contiguous())
        return (y,) if total is None else (y, total)
    if op == "linear":
        w = s["codes"].double() * s["scales"].double().unsqueeze(1)
        return torch.matmul(_eight_bits(s["x"].double()), w.transpose(0, 1).contiguous())
    if op == "experts":
        x, at = _eight_bits(s["x"].double()), s["offsets"].tolist()
        y = []
        for e, (lo, hi) in enumerate(zip(at[:-1], at[1:])):
            w = s["codes"][e].double() * s["scales"][e].double().unsqueeze(1)
            y.append(torch.matmul(x[lo:hi], w.transpose(0, 1).contiguous()))
        return torch.cat(y + [x.new_zeros((x.shape[0] - at[-1], s["codes"].shape[1]))])
    experts, top_k = case["experts"], case["top_k"]
    ids = s["ids"].long()
    live = (ids >= 0).sum(1) > 0
    counts = torch.bincount(ids[ids >= 0], minlength=experts)
    tokens = int(live.sum())
    of = max(tokens, 1)
    p = torch.softmax(s["logits"].double(), dim=1) * live.double().unsqueeze(1)
    share = counts.double() / (of * top_k)
    loss = experts * torch.dot(share, p.mean(0) * (case["tokens"] / of))
    along = torch.mv(p, share).unsqueeze(1)
    dlogits = s["dloss"].double() * experts / of * (p * share - p * along)
    return loss, torch.cat([counts, counts.new_tensor([tokens])]).int(), dlogits
