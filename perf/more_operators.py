"""Routing to experts and FP8 products with a scale for each block of 128, at the sizes they are
used at: the router, quantisation to FP8 and back, the linear layer with an FP8 weight, and
a mixture-of-experts layer from its router's logits to its combined output.

FP8: E4M3 codes; rows of activations have one fp32 scale for 128 consecutive k, weights one for
128 rows x 128 k. A value is code * scale.

`run` computes a case either with elementary torch operations (`own` false) or with the
library's calls (`own` true); `exact` is the same result in 64 bits, written apart.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
TOP = 448.0  # E4M3's largest value
F8 = torch.float8_e4m3fn
MOST_FLOPS = 2.0 * 8192 * 14336 * 4096  # the largest listed product


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # the activations of a decode step of 16 requests, on their way into an 8-bit layer
        {"name": "quantize decode", "op": "quantize", "M": 16, "K": 4096, "x": "bf16", "pitch": 4096, "rows": 1, "pow2": False},
        # a prompt's activations before the down projection, rows inside a wider buffer
        {"name": "quantize prompt", "op": "quantize", "M": 2048, "K": 14336, "x": "bf16", "pitch": 28672, "rows": 1, "pow2": False},
        # the smallest product: one token through a square projection, activations kept in BF16
        {"name": "linear one token", "op": "linear", "act": "bf16", "M": 1, "N": 2048, "K": 2048, "y": "f32"},
        # sixteen requests through a fused QKV projection: the weight is read once for all
        {"name": "linear decode", "op": "linear", "act": "fp8", "M": 16, "N": 12288, "K": 4096, "y": "bf16"},
        # a short batch through a projection of odd width; neither side ends with a block
        {"name": "linear ragged", "op": "linear", "act": "bf16", "M": 333, "N": 1001, "K": 1104, "y": "f32"},
        # a prompt through an MLP up projection
        {"name": "linear prompt", "op": "linear", "act": "fp8", "M": 2048, "N": 14336, "K": 4096, "y": "bf16"},
        # a batch of prompts
        {"name": "linear prompts", "op": "linear", "act": "fp8", "M": 8192, "N": 14336, "K": 4096, "y": "bf16"},
        # one token's experts: softmax scores, renormalised
        {"name": "route one token", "op": "route", "T": 1, "E": 128, "top_k": 8, "scoring": "softmax", "bias": False, "groups": 1,
         "top_groups": 1, "group_score": "max", "renormalize": True, "logits": "bf16", "skew": 0.0, "pad": 0},
        # a prompt batch, the last rows of it padding: sigmoid scores, a bias for balance, 4 of 8 groups
        {"name": "route prompts groups", "op": "route", "T": 16384, "E": 256, "top_k": 8, "scoring": "sigmoid", "bias": True, "groups": 8,
         "top_groups": 4, "group_score": "top2", "renormalize": True, "logits": "f32", "skew": 0.5, "pad": 100},
        # a mixture-of-experts layer for one token: latency
        {"name": "moe one token", "op": "moe", "act": "bf16", "T": 1, "E": 128, "top_k": 8, "H": 2048, "I": 768, "skew": 0.0},
        # the same layer for a decode step of 16 requests
        {"name": "moe decode", "op": "moe", "act": "bf16", "T": 16, "E": 128, "top_k": 8, "H": 2048, "I": 768, "skew": 0.0},
        # the same layer for a prompt, activations quantised, experts unevenly loaded
        {"name": "moe prompt", "op": "moe", "act": "fp8", "T": 4096, "E": 128, "top_k": 8, "H": 2048, "I": 768, "skew": 0.5},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _steps(rng, low, high, step):
    return step * _log(rng, low // step, high // step)


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "route", "moe"])
    if op == "quantize":
        M, K = _log(rng, 1, 8192), _steps(rng, 16, 14336, 16)
        return {"op": op, "M": M, "K": K, "x": rng.choice(["bf16", "f32"]), "pitch": K * rng.choice([1, 1, 2]),
                "rows": rng.choice([1, 1, 128]), "pow2": rng.random() < 0.3}
    act = rng.choice(["bf16", "fp8"])
    if op == "linear":
        M, N, K = _log(rng, 1, 8192), _log(rng, 16, 14336), _steps(rng, 64, 14336, 16)
        M = max(1, min(M, int(MOST_FLOPS / (2.0 * N * K))))
        return {"op": op, "act": act, "M": M, "N": N, "K": K, "y": rng.choice(["f32", "bf16"])}
    if op == "route":
        G = rng.choice([1, 1, 2, 4, 8])
        E = G * _log(rng, max(2, 8 // G), 512 // G)
        most = rng.randint(1, G)
        T = _log(rng, 1, 16384)
        return {"op": op, "T": T, "E": E, "top_k": rng.randint(1, min(16, E // G * most)), "scoring": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "groups": G, "top_groups": most, "group_score": rng.choice(["max", "top2"]),
                "renormalize": rng.random() < 0.7, "logits": rng.choice(["f32", "bf16"]), "skew": rng.choice([0.0, 0.5, 2.0]),
                "pad": rng.choice([0, T // 10])}
    E, T, H, I = _log(rng, 4, 128), _log(rng, 1, 4096), _steps(rng, 128, 4096, 16), _steps(rng, 128, 1536, BLOCK)
    k = rng.randint(1, min(8, E))
    return {"op": op, "act": act, "T": max(1, min(T, int(MOST_FLOPS / (6.0 * k * H * I)))), "E": E, "top_k": k, "H": H, "I": I,
            "skew": rng.choice([0.0, 0.5, 2.0])}


def work(case):
    weight = 1 + 4.0 / BLOCK ** 2  # bytes of a stored weight
    if case["op"] == "quantize":
        n = case["M"] * case["K"]
        return {"bytes": n * ((2 if case["x"] == "bf16" else 4) + 2 + 4.0 / (BLOCK * case["rows"])), "flops": 0}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + weight * N * K + (4 if case["y"] == "f32" else 2) * M * N, "flops": 2.0 * M * N * K}
    T, E, k = case["T"], case["E"], case["top_k"]
    if case["op"] == "route":
        # an exponential and a comparison with each of the picks so far, for each score
        return {"bytes": T * E * (4 if case["logits"] == "f32" else 2) + (4 * E if case["bias"] else 0) + 8 * T * k,
                "flops": float(T * E * (1 + k))}
    used = E * (1 - (1 - k / E) ** T)  # experts that a token picks, when all are as popular
    H, I = case["H"], case["I"]
    return {"bytes": 2 * T * E + 2 * T * H + used * weight * 3 * H * I + 8 * T * k + 2 * T * H, "flops": 6.0 * T * k * H * I}


# ------------------------------------------------------------------------------ the inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _acts(g, M, K, dtype, pitch=None):
    """Activation rows: unit normal, a few channels twenty times as large as the others."""
    x = torch.randn((M, K), generator=g, device=DEV)
    loud = torch.rand((K,), generator=g, device=DEV) < 0.004
    x = (x * (1 + 19 * loud)).to(dtype)
    if pitch is None or pitch == K:
        return x
    wide = torch.zeros((M, pitch), dtype=dtype, device=DEV)
    wide[:, :K] = x
    return wide[:, :K]


def _weight(g, *shape):
    """A normal weight of deviation 0.02, its rows of different loudness, in FP8."""
    w = torch.randn(shape, generator=g, device=DEV)
    w = 0.02 * w * torch.exp(0.3 * torch.randn((*shape[:-1], 1), generator=g, device=DEV))
    if len(shape) == 2:
        return _plain_quantize(w, BLOCK)
    c, s = zip(*(_plain_quantize(one, BLOCK) for one in w))
    return torch.stack([one.view(torch.uint8) for one in c]).view(F8), torch.stack(s)


def _logits(g, T, E, skew, dtype):
    """Each expert's popularity and the tokens' own taste."""
    liking = skew * torch.randn((E,), generator=g, device=DEV)
    return (liking - torch.log(-torch.log(torch.rand((T, E), generator=g, device=DEV).clamp(1e-7, 1 - 1e-6)))).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": dict(case)}
    if case["op"] == "quantize":
        s["x"] = _acts(g, case["M"], case["K"], torch.bfloat16 if case["x"] == "bf16" else torch.float32, case["pitch"])
        return s
    if case["op"] == "linear":
        s["x"] = _acts(g, case["M"], case["K"], torch.bfloat16)
        s["w"] = _weight(g, case["N"], case["K"])
        return s
    T, E = case["T"], case["E"]
    if case["op"] == "route":
        s["logits"] = _logits(g, T, E, case["skew"], torch.float32 if case["logits"] == "f32" else torch.bfloat16)
        if case["pad"]:
            s["logits"][T - case["pad"]:] = -math.inf
        s["bias"] = 0.05 * torch.randn((E,), generator=g, device=DEV) if case["bias"] else None
        return s
    s["logits"] = _logits(g, T, E, case["skew"], torch.bfloat16)
    s["x"] = _acts(g, T, case["H"], torch.bfloat16)
    s["gate_up"] = _weight(g, E, 2 * case["I"], case["H"])
    s["down"] = _weight(g, E, case["H"], case["I"])
    return s


# ------------------------------------------------------------------- the plain form (32 bits)

def _plain_blocks(x, rows):
    """x [M][K], padded with zeros, as [blocks down][rows][blocks along][128]."""
    M, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % BLOCK, 0, -M % rows))
    return x.reshape(x.shape[0] // rows, rows, x.shape[1] // BLOCK, BLOCK)


def _plain_quantize(x, rows=1, pow2=False):
    """(codes, scales): a block's scale is its largest magnitude over 448, or the next power of
    two; its codes are the nearest E4M3 values of x over the scale, ties to the even code."""
    b = _plain_blocks(x.float(), rows)
    s = b.abs().amax((1, 3))
    s = s / torch.full_like(s, TOP)  # (a number would be multiplied by as its inverse)
    if pow2:
        m, e = torch.frexp(s)
        s = torch.where(s > 0, torch.ldexp(torch.ones_like(s), e - (m == 0.5).int()), s)
    d = s[:, None, :, None]
    q = torch.where(d > 0, b / d, torch.zeros_like(b)).clamp(-TOP, TOP)
    return q.reshape(q.shape[0] * rows, -1)[:x.shape[0], :x.shape[1]].to(F8).contiguous(), s


def _plain_dequantize(codes, scales, rows=1):
    b = _plain_blocks(codes.float(), rows) * scales[:, None, :, None]
    return b.reshape(b.shape[0] * rows, -1)[:codes.shape[0], :codes.shape[1]]


def _plain_acts(x, act):
    return x.float() if act == "bf16" else _plain_dequantize(*_plain_quantize(x))


def _plain_grouped(rows, codes, scales, ids):
    """rows [R][K] of the routes, a weight [E][N][K] -> [R][N]: the weights of the experts that
    are picked, the rows of each side by side, padded to the largest group, and one batched
    product."""
    used, e, counts = torch.unique(ids, return_inverse=True, return_counts=True)
    N, K = codes.shape[1:]
    spread = scales[used].repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :K]
    w = codes.view(torch.uint8)[used].view(F8).float() * spread
    e, order = torch.sort(e.reshape(-1), stable=True)
    at = torch.arange(e.numel(), device=e.device) - (torch.cumsum(counts, 0) - counts)[e]
    buf = rows.new_zeros((used.numel(), int(counts.max()), rows.shape[1]))
    buf[e, at] = rows[order]
    out = rows.new_empty((e.numel(), w.shape[1]))
    out[order] = torch.bmm(buf, w.transpose(1, 2).contiguous())[e, at]
    return out


def _plain_route(logits, k, scoring, bias, G, top_groups, group_score, renormalize):
    """(ids, weights) by descending score, the lower id first where two are equal. Scores are
    held in 64 bits: many experts lie close together, and the picks have to be the right ones."""
    z = logits.double()
    open_ = z > -math.inf
    if scoring == "softmax":
        p = torch.exp(z - z.amax(1, keepdim=True))
        p = torch.where(open_, p / p.sum(1, keepdim=True), torch.zeros_like(p))
    else:
        p = 1 / (1 + torch.exp(-z))
    # without a bias the order of the scores is that of the logits
    c = p + bias.double() if bias is not None else p if group_score == "top2" and G > 1 else z
    c = torch.where(open_, c, torch.full_like(c, -math.inf))
    if G > 1:
        best = torch.sort(c.unflatten(1, (G, -1)), dim=2, descending=True)[0]
        score = best[:, :, 0]
        if group_score == "top2":
            score = score + torch.where(best[:, :, 1] > -math.inf, best[:, :, 1], torch.zeros_like(score))
        rank = torch.sort(torch.sort(score, dim=1, descending=True, stable=True)[1], dim=1)[1]
        c = torch.where((rank < top_groups).repeat_interleave(c.shape[1] // G, 1), c, torch.full_like(c, -math.inf))
    top, ids = torch.sort(c, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    got = top > -math.inf
    w = torch.where(got, torch.gather(p, 1, ids), torch.zeros_like(top))
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return torch.where(got, ids, torch.full_like(ids, -1)).to(torch.int32), w.float()


def _plain(s):
    case = s["case"]
    if case["op"] == "quantize":
        codes, scales = _plain_quantize(s["x"], case["rows"], case["pow2"])
        return _plain_dequantize(codes, scales, case["rows"]).to(torch.bfloat16), scales
    if case["op"] == "route":
        return _plain_route(s["logits"], case["top_k"], case["scoring"], s["bias"], case["groups"], case["top_groups"],
                            case["group_score"], case["renormalize"])
    x = _plain_acts(s["x"], case["act"])
    if case["op"] == "linear":
        y = x @ _plain_dequantize(*s["w"], BLOCK).t()
        return y if case["y"] == "f32" else y.to(torch.bfloat16)
    k = case["top_k"]
    ids, weights = _plain_route(s["logits"], k, "softmax", None, 1, 1, "max", True)
    h = _plain_grouped(x.repeat_interleave(k, 0), *s["gate_up"], ids)
    gate, up = h.chunk(2, 1)
    a = (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16)
    r = _plain_grouped(_plain_acts(a, case["act"]), *s["down"], ids)
    y = (r.unflatten(0, (-1, k)) * weights.unsqueeze(-1)).sum(1)
    return y.to(torch.bfloat16), ids, weights


# -------------------------------------------------------------------- the library's operators

def _own(s):
    import nvfp4_block_scaled_linear_amd as nv

    case = s["case"]
    if case["op"] == "quantize":
        codes, scales = nv.fp8_quantize(s["x"], block_rows=case["rows"], pow2_scales=case["pow2"])
        return nv.fp8_dequantize(codes, scales, block_rows=case["rows"]), scales
    if case["op"] == "route":
        return nv.moe_route(s["logits"], case["top_k"], scoring=case["scoring"], bias=s["bias"], groups=case["groups"],
                            top_groups=case["top_groups"], group_score=case["group_score"], renormalize=case["renormalize"])
    if case["op"] == "linear":
        x, xs = (s["x"], None) if case["act"] == "bf16" else nv.fp8_quantize(s["x"])
        return nv.fp8_linear(x, *s["w"], x_scales=xs, out_dtype=torch.float32 if case["y"] == "f32" else torch.bfloat16)
    T, E, k, H, I = (case[n] for n in ("T", "E", "top_k", "H", "I"))
    if "workspace" not in s:  # a program keeps it, as it keeps its weights
        mid = nv.OUT_SWIGLU_BF16 if case["act"] == "bf16" else nv.OUT_SWIGLU_FP8
        size = max(nv.fp8_grouped_workspace_size(T, k, 2 * I, H, E, mid), nv.fp8_grouped_workspace_size(T, k, H, I, E, nv.OUT_COMBINE))
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["x"].device)
    ws = s["workspace"]
    ids, weights = nv.moe_route(s["logits"], k)
    if case["act"] == "bf16":
        a, a_s = nv.fp8_grouped_linear(s["x"], *s["gate_up"], ids, out_mode=nv.OUT_SWIGLU_BF16, workspace=ws), None
    else:
        x, xs = nv.fp8_quantize(s["x"])
        a, a_s = nv.fp8_grouped_linear(x, *s["gate_up"], ids, x_scales=xs, out_mode=nv.OUT_SWIGLU_FP8, workspace=ws)
    y = nv.fp8_grouped_linear(a, *s["down"], ids, x_scales=a_s, topk_w=weights, out_mode=nv.OUT_COMBINE, rows_per_route=True,
                              out_dtype=torch.bfloat16, workspace=ws, reuse_grouping=True)
    return y, ids, weights


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------- the definition, in 64 bits

def _e4m3_values():
    """The magnitudes of codes 0 to 0x7E."""
    return torch.tensor([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127],
                        dtype=torch.float64, device=DEV)


def _values(codes, scales, rows):
    """What codes [..., N, K] under scales [..., blocks, blocks] stand for."""
    table = torch.cat([_e4m3_values(), torch.full((1,), math.nan, dtype=torch.float64, device=DEV)])
    raw = codes.view(torch.uint8).long()
    v = table[raw & 127] * (1 - 2 * (raw >> 7)).double()
    N, K = v.shape[-2:]
    i, j = torch.arange(N, device=DEV) // rows, torch.arange(K, device=DEV) // BLOCK
    return v * scales.double()[..., i, :][..., j]


def _round_trip(x, rows=1, pow2=False):
    """(values, scales): nearest E4M3 multiples of each block's scale. The scale, and a value over
    its scale, are fp32 numbers by definition."""
    mags = _e4m3_values()
    between = (mags[1:] + mags[:-1]) / 2
    out, scales = [], []
    step = rows * max(1, (1 << 24) // (x.shape[1] * rows))
    for part in x.double().split(step):
        M, K = part.shape
        i, j = torch.arange(M, device=DEV) // rows, torch.arange(K, device=DEV) // BLOCK
        top = torch.stack([one.abs().amax(1) for one in part.split(BLOCK, 1)], 1)
        top = torch.stack([one.amax(0) for one in top.split(rows)]) if rows > 1 else top
        s = (top / TOP).float().double()
        if pow2:
            s = torch.where(s > 0, torch.pow(2.0, torch.ceil(torch.log2(torch.where(s > 0, s, 1.0)))), s)
        d = s[i][:, j]
        q = (part.abs() / torch.where(d > 0, d, 1.0)).float().double() * (d > 0)
        at = torch.searchsorted(between, q)  # the lower of the two at a tie
        tie = (at < 126) & (q == between[at.clamp(max=125)]) & (at % 2 == 1)
        out.append(torch.copysign(mags[at + tie.long()], part) * d)
        scales.append(s)
    return torch.cat(out), torch.cat(scales)


def _exact_route(case, logits, bias):
    E, k, G = case["E"], case["top_k"], case.get("groups", 1)
    z = logits.double()
    closed = torch.isinf(z)
    if case.get("scoring", "softmax") == "softmax":
        p = torch.softmax(torch.where(closed.all(1, keepdim=True), torch.zeros_like(z), z), 1)
    else:
        p = torch.sigmoid(z)
    top2 = case.get("group_score") == "top2"
    c = z.clone() if bias is None and not (top2 and G > 1) else p + (0 if bias is None else bias.double())
    c[closed] = -math.inf
    lowest_first = torch.arange(E, 0, -1, device=DEV).expand(c.shape)

    def best(c):  # the largest, the lowest index of equals
        return torch.where(c == c.amax(1, keepdim=True), lowest_first[:, :c.shape[1]], 0).argmax(1, keepdim=True)

    if G > 1:
        scores = []
        for part in c.split(E // G, 1):
            first = part.amax(1, keepdim=True)
            second = part.scatter(1, best(part), -math.inf).amax(1, keepdim=True)
            scores.append(first + torch.where(torch.isinf(second), torch.zeros_like(second), second) if top2 else first)
        scores, kept = torch.cat(scores, 1), torch.zeros((c.shape[0], G), dtype=torch.bool, device=DEV)
        for _ in range(case["top_groups"]):
            one = best(scores)
            kept.scatter_(1, one, True)
            scores = scores.scatter(1, one, -math.inf)
        c[~kept[:, torch.arange(E, device=DEV) // (E // G)]] = -math.inf
    ids, weights = [], []
    for _ in range(k):
        one = best(c)
        none = torch.isinf(torch.gather(c, 1, one))
        weights.append(torch.where(none, 0.0, torch.gather(p, 1, one)))
        ids.append(torch.where(none, -1, one))
        c = c.scatter(1, one, -math.inf)
    ids, weights = torch.cat(ids, 1), torch.cat(weights, 1)
    if case.get("renormalize", True):
        weights = weights / torch.where(weights.sum(1, keepdim=True) > 0, weights.sum(1, keepdim=True), 1.0)
    return ids.to(torch.int32), weights


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _round_trip(s["x"], case["rows"], case["pow2"])
    if case["op"] == "route":
        return _exact_route(case, s["logits"], s["bias"])
    x = s["x"].double() if case["act"] == "bf16" else _round_trip(s["x"])[0]
    if case["op"] == "linear":
        return x @ _values(*s["w"], BLOCK).t()
    picked, weights = _exact_route(case, s["logits"], None)
    ids, k = picked.long(), case["top_k"]
    routes = torch.arange(ids.numel(), device=DEV)
    flat = ids.reshape(-1)
    a = torch.zeros((ids.numel(), case["I"]), dtype=torch.float64, device=DEV)
    for e in range(case["E"]):
        mine = routes[flat == e]
        h = x[mine // k] @ _values(s["gate_up"][0][e], s["gate_up"][1][e], BLOCK).t()
        g, u = h[:, :case["I"]], h[:, case["I"]:]
        a[mine] = g * torch.sigmoid(g) * u
    a = a.to(torch.bfloat16)
    a = a.double() if case["act"] == "bf16" else _round_trip(a)[0]
    y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device=DEV)
    share = weights.reshape(-1, 1)
    for e in range(case["E"]):
        mine = routes[flat == e]
        r = a[mine] @ _values(s["down"][0][e], s["down"][1][e], BLOCK).t()
        y.index_add_(0, mine // k, r * share[mine])
    return y, picked, weights
