"""The MXFP4 operators at the sizes they are used at: quantisation to MXFP4 and back, the
linear layer with an MXFP4 weight, and its expert-grouped form.

MXFP4: E2M1 codes, two per byte (even k in the low nibble), and one E8M0 scale byte s per 32
consecutive k; a value is e2m1(code) * 2^(s - 127).

`run` computes a case either with elementary torch operations (`own` false) or with the
library's calls (`own` true); `exact` is the same result in 64 bits, written apart.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32
MOST_FLOPS = 2.0 * 8192 * 14336 * 4096  # the largest listed product


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # the activations of a decode step of 16 requests, on their way into a W4A4 layer
        {"name": "quantize decode", "op": "quantize", "M": 16, "K": 4096, "x": "bf16", "pitch": 4096},
        # a prompt's activations before the down projection, rows inside a wider buffer
        {"name": "quantize prompt", "op": "quantize", "M": 2048, "K": 14336, "x": "bf16", "pitch": 28672},
        # the smallest call: one token through a square projection
        {"name": "linear one token", "op": "linear", "act": "bf16", "M": 1, "N": 2048, "K": 2048, "y": "f32"},
        # sixteen requests through a fused QKV projection: the weight is read once for all
        {"name": "linear decode", "op": "linear", "act": "bf16", "M": 16, "N": 12288, "K": 4096, "y": "f32"},
        # a prompt through an MLP up projection, activations kept in BF16
        {"name": "linear prompt", "op": "linear", "act": "bf16", "M": 2048, "N": 14336, "K": 4096, "y": "bf16"},
        # a four-row verify step with the activations quantised too
        {"name": "linear w4a4 verify", "op": "linear", "act": "mxfp4", "M": 4, "N": 4096, "K": 4096, "y": "f32"},
        # a short prompt, activations quantised
        {"name": "linear w4a4 short prompt", "op": "linear", "act": "mxfp4", "M": 512, "N": 4096, "K": 4096, "y": "f32"},
        # a batch of prompts, activations quantised: the largest product
        {"name": "linear w4a4 prompts", "op": "linear", "act": "mxfp4", "M": 8192, "N": 14336, "K": 4096, "y": "bf16"},
        # ragged groups of odd sizes: few popular experts, K no multiple of 128, N odd
        {"name": "grouped ragged", "op": "grouped", "act": "bf16", "T": 333, "E": 24, "top_k": 3, "N": 1001, "K": 1056, "skew": 2.0, "y": "f32"},
        # a mixture-of-experts layer for one token: latency
        {"name": "moe one token", "op": "moe", "act": "bf16", "T": 1, "E": 128, "top_k": 8, "H": 2048, "I": 768, "skew": 0.0},
        # the same layer for a decode step of 16 requests
        {"name": "moe decode", "op": "moe", "act": "bf16", "T": 16, "E": 128, "top_k": 8, "H": 2048, "I": 768, "skew": 0.0},
        # the same layer for a prompt, activations quantised, experts unevenly loaded
        {"name": "moe w4a4 prompt", "op": "moe", "act": "mxfp4", "T": 4096, "E": 128, "top_k": 8, "H": 2048, "I": 768, "skew": 0.5},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _blocks(rng, low, high, step=BLOCK):
    return step * _log(rng, low // step, high // step)


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "grouped", "moe"])
    act = rng.choice(["bf16", "mxfp4"])
    if op == "quantize":
        M, K = _log(rng, 1, 8192), _blocks(rng, 32, 14336)
        return {"op": op, "M": M, "K": K, "x": rng.choice(["bf16", "f32"]), "pitch": K * rng.choice([1, 1, 2])}
    if op == "linear":
        M, N, K = _log(rng, 1, 8192), _log(rng, 16, 14336), _blocks(rng, 32, 14336)
        M = max(1, min(M, int(MOST_FLOPS / (2.0 * N * K))))
        return {"op": op, "act": act, "M": M, "N": N, "K": K, "y": rng.choice(["f32", "bf16"])}
    E = _log(rng, 4, 128)
    T, k = _log(rng, 1, 4096), rng.randint(1, min(8, E))
    skew = rng.choice([0.0, 0.5, 2.0])
    if op == "grouped":
        return {"op": op, "act": act, "T": T, "E": E, "top_k": k, "N": _log(rng, 16, 4096),
                "K": _blocks(rng, 64, 4096), "skew": skew, "y": rng.choice(["f32", "bf16"])}
    return {"op": op, "act": act, "T": T, "E": E, "top_k": k, "H": _blocks(rng, 128, 4096),
            "I": _blocks(rng, 64, 1536), "skew": skew}


def _y_bytes(case):
    return 4 if case.get("y") == "f32" else 2


def work(case):
    weight = 0.5 + 1.0 / BLOCK  # bytes of a stored element
    if case["op"] == "quantize":
        n = case["M"] * case["K"]
        return {"bytes": n * ((2 if case["x"] == "bf16" else 4) + 2), "flops": 0}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + weight * N * K + _y_bytes(case) * M * N, "flops": 2.0 * M * N * K}
    T, E, k = case["T"], case["E"], case["top_k"]
    used = E * (1 - (1 - k / E) ** T)  # experts that a token picks, when all are as popular
    if case["op"] == "grouped":
        N, K = case["N"], case["K"]
        return {"bytes": 2 * T * K + used * weight * N * K + 4 * T * k + _y_bytes(case) * T * k * N,
                "flops": 2.0 * T * k * N * K}
    H, I = case["H"], case["I"]
    return {"bytes": 2 * T * H + used * weight * 3 * H * I + 8 * T * k + 2 * T * H,
            "flops": 6.0 * T * k * H * I}


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
    """A normal weight of deviation 0.02 in MXFP4."""
    return _plain_quantize(0.02 * torch.randn(shape, generator=g, device=DEV))


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
    T, E, k = case["T"], case["E"], case["top_k"]
    liking = case["skew"] * torch.randn((E,), generator=g, device=DEV)
    logits = liking - torch.log(-torch.log(torch.rand((T, E), generator=g, device=DEV).clamp(1e-7, 1 - 1e-7)))
    top, ids = torch.topk(logits, k, dim=1)
    s["ids"] = ids.to(torch.int32).contiguous()
    s["router"] = torch.softmax(top, dim=1).contiguous()
    if case["op"] == "grouped":
        s["x"] = _acts(g, T, case["K"], torch.bfloat16)
        s["w"] = _weight(g, E, case["N"], case["K"])
    else:
        s["x"] = _acts(g, T, case["H"], torch.bfloat16)
        s["gate_up"] = _weight(g, E, 2 * case["I"], case["H"])
        s["down"] = _weight(g, E, case["H"], case["I"])
    return s


# ------------------------------------------------------------------- the plain form (32 bits)

def _plain_quantize(x):
    """(codes, scales): the scale's exponent is that of the block's largest value less two
    (6 = 1.5 * 2^2 is the largest E2M1 value), elements round to nearest, ties to the even
    code, and saturate."""
    xb = x.float().unflatten(-1, (-1, BLOCK))
    amax = xb.abs().amax(-1)
    s = (torch.frexp(amax)[1] + (126 - 2)).clamp(0, 254)
    s = torch.where(amax == 0, torch.zeros_like(s), s)
    q = torch.ldexp(xb, (127 - s).unsqueeze(-1))
    a = q.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    code = (code + 8 * torch.signbit(q)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.to(torch.uint8)


def _plain_dequantize(codes, scales):
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = table[code.int()].unflatten(-1, (-1, BLOCK))
    return torch.ldexp(v, (scales.int() - 127).unsqueeze(-1)).flatten(-2)


def _plain_acts(x, act):
    return x.float() if act == "bf16" else _plain_dequantize(*_plain_quantize(x))


def _plain_grouped(rows, codes, scales, ids):
    """rows [R][K] of the routes, a weight [E][N][K] -> [R][N]: the weights of the experts that
    are picked, the rows of each side by side, padded to the largest group, and one batched
    product."""
    used, e, counts = torch.unique(ids, return_inverse=True, return_counts=True)
    w = _plain_dequantize(codes[used], scales[used])
    e, order = torch.sort(e.reshape(-1), stable=True)
    at = torch.arange(e.numel(), device=e.device) - (torch.cumsum(counts, 0) - counts)[e]
    buf = rows.new_zeros((used.numel(), int(counts.max()), rows.shape[1]))
    buf[e, at] = rows[order]
    out = rows.new_empty((e.numel(), w.shape[1]))
    out[order] = torch.bmm(buf, w.transpose(1, 2).contiguous())[e, at]
    return out


def _plain(s):
    case = s["case"]
    if case["op"] == "quantize":
        return _plain_dequantize(*_plain_quantize(s["x"])).to(torch.bfloat16)
    x = _plain_acts(s["x"], case["act"])
    if case["op"] == "linear":
        y = x @ _plain_dequantize(*s["w"]).t()
        return y if case["y"] == "f32" else y.to(torch.bfloat16)
    k = case["top_k"]
    rows = x.repeat_interleave(k, 0)
    if case["op"] == "grouped":
        y = _plain_grouped(rows, *s["w"], s["ids"])
        return y if case["y"] == "f32" else y.to(torch.bfloat16)
    h = _plain_grouped(rows, *s["gate_up"], s["ids"])
    gate, up = h.chunk(2, 1)
    a = (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16)
    r = _plain_grouped(_plain_acts(a, case["act"]), *s["down"], s["ids"])
    y = (r.unflatten(0, (-1, k)) * s["router"].unsqueeze(-1)).sum(1)
    return y.to(torch.bfloat16)


# -------------------------------------------------------------------- the library's operators

def _own(s):
    import nvfp4_block_scaled_linear_amd as nv

    case = s["case"]
    if case["op"] == "quantize":
        return nv.mxfp4_dequantize(*nv.mxfp4_quantize(s["x"]))
    x, xs = (s["x"], None) if case["act"] == "bf16" else nv.mxfp4_quantize(s["x"])
    y_type = torch.float32 if case.get("y") == "f32" else torch.bfloat16
    if case["op"] == "linear":
        return nv.mxfp4_linear(x, *s["w"], x_scales=xs, out_dtype=y_type)
    if case["op"] == "grouped":
        return nv.mxfp4_grouped_linear(x, *s["w"], s["ids"], x_scales=xs, out_dtype=y_type)
    T, k = s["ids"].shape
    E, N, _ = s["gate_up"][0].shape
    if "workspace" not in s:  # a program keeps it, as it keeps its weights
        size = max(nv.mxfp4_grouped_workspace_size(T, k, N, case["H"], E, nv.OUT_SWIGLU_BF16),
                   nv.mxfp4_grouped_workspace_size(T, k, case["H"], case["I"], E, nv.OUT_COMBINE))
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["x"].device)
    ws = s["workspace"]
    if case["act"] == "bf16":
        a, a_s = nv.mxfp4_grouped_linear(x, *s["gate_up"], s["ids"], out_mode=nv.OUT_SWIGLU_BF16, workspace=ws), None
    else:
        a, a_s = nv.mxfp4_grouped_linear(x, *s["gate_up"], s["ids"], x_scales=xs, out_mode=nv.OUT_SWIGLU_MXFP4, workspace=ws)
    return nv.mxfp4_grouped_linear(a, *s["down"], s["ids"], x_scales=a_s, topk_w=s["router"], out_mode=nv.OUT_COMBINE,
                                   rows_per_route=True, out_dtype=torch.bfloat16, workspace=ws, reuse_grouping=True)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------- the definition, in 64 bits

def _bytes_to_values(codes, scales):
    half = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    nibble = half + [-v for v in half]
    pairs = torch.tensor([[nibble[b % 16], nibble[b // 16]] for b in range(256)], dtype=torch.float64, device=DEV)
    v = pairs[codes.long()].reshape(*codes.shape[:-1], -1, BLOCK)
    return (v * torch.pow(2.0, scales.double() - 127).unsqueeze(-1)).reshape(*codes.shape[:-1], -1)


def _round_trip(x):
    """Nearest MXFP4 values of the rows x (finite): the distance to every magnitude decides, a
    hair against the odd codes settles the ties."""
    out = []
    for rows in x.double().split(max(1, (1 << 24) // x.shape[1])):
        b = rows.reshape(rows.shape[0], -1, BLOCK)
        top = b.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
        e = e + (torch.pow(2.0, e + 1) <= top).double() - ((torch.pow(2.0, e) > top) & (top > 0)).double()
        unit = torch.pow(2.0, (e - 2).clamp(-127, 127))
        mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)
        best, value = torch.full_like(b, math.inf), torch.zeros_like(b)
        for i in range(8):
            d = (b.abs() / unit - mags[i]).abs() + (1e-12 if i % 2 else 0.0)
            value = torch.where(d < best, mags[i], value)
            best = torch.minimum(best, d)
        out.append((torch.copysign(value, b) * unit).reshape(rows.shape))
    return torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _round_trip(s["x"])
    x = s["x"].double() if case["act"] == "bf16" else _round_trip(s["x"])
    if case["op"] == "linear":
        return x @ _bytes_to_values(*s["w"]).t()
    ids, k = s["ids"].long(), case["top_k"]
    routes = torch.arange(ids.numel(), device=DEV)
    flat = ids.reshape(-1)
    if case["op"] == "grouped":
        y = torch.zeros((ids.numel(), case["N"]), dtype=torch.float64, device=DEV)
        for e in range(case["E"]):
            mine = routes[flat == e]
            y[mine] = x[mine // k] @ _bytes_to_values(s["w"][0][e], s["w"][1][e]).t()
        return y
    a = torch.zeros((ids.numel(), case["I"]), dtype=torch.float64, device=DEV)
    for e in range(case["E"]):
        mine = routes[flat == e]
        h = x[mine // k] @ _bytes_to_values(s["gate_up"][0][e], s["gate_up"][1][e]).t()
        g, u = h[:, :case["I"]], h[:, case["I"]:]
        a[mine] = g * torch.sigmoid(g) * u
    a = a.to(torch.bfloat16)
    a = a.double() if case["act"] == "bf16" else _round_trip(a)
    y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device=DEV)
    weights = s["router"].double().reshape(-1)
    for e in range(case["E"]):
        mine = routes[flat == e]
        r = a[mine] @ _bytes_to_values(s["down"][0][e], s["down"][1][e]).t()
        y.index_add_(0, mine // k, r * weights[mine].unsqueeze(1))
    return y
