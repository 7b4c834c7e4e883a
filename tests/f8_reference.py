"""FP8 with scales for blocks of 128, and the router, in float64 numpy from their definitions
(include/fp8.h), with the tolerances of products: the plain implementation that the FP8 tests
compare the library with."""
import numpy as np

# magnitudes of codes 0 .. 0x7E
MAGS = np.array([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])
TABLE = np.concatenate([MAGS, [np.nan], -MAGS, [np.nan]])
MIDS = (MAGS[1:] + MAGS[:-1]) / 2


def blocks(n):
    return -(-n // 128)


def encode(q):
    """Nearest codes of finite values, ties to the even code, saturating."""
    a = np.abs(np.asarray(q, np.float64))
    code = np.searchsorted(MIDS, a)  # a value between two: the lower one at a tie
    tie = (code < 126) & (a == MIDS[np.minimum(code, 125)]) & (code % 2 == 1)
    return (code + tie + 128 * np.signbit(q)).astype(np.uint8)


def quantize(x, rows=1, pow2=False):
    """x [M][K] of fp32 values -> codes [M][K] uint8, scales fp32 [ceil(M/rows)][ceil(K/128)]."""
    x = np.asarray(x, np.float32)
    M, K = x.shape
    pad = np.zeros((-(-M // rows) * rows, 128 * blocks(K)), np.float32)
    pad[:M, :K] = x
    b = pad.reshape(-1, rows, blocks(K), 128)
    bad = ~np.isfinite(b).all((1, 3))
    b = np.where(bad[:, None, :, None], np.float32(0), b)
    s = np.abs(b).max((1, 3)) / np.float32(448)
    if pow2:
        m, e = np.frexp(s.astype(np.float64))
        s = np.where(s > 0, np.ldexp(1.0, e - (m == 0.5)), 0).astype(np.float32)
    d = s[:, None, :, None]
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        q = np.where(d > 0, b / d, np.copysign(np.float32(0), b))
    assert q.dtype == np.float32
    codes = np.where(bad[:, None, :, None], 0, encode(np.clip(q, -448, 448)))
    return codes.reshape(pad.shape)[:M, :K].astype(np.uint8), np.where(bad, np.float32(np.nan), s)


def dequantize(codes, scales, rows=1):
    """The exact values in float64 (codes [..., M, K])."""
    M, K = codes.shape[-2:]
    s = scales.astype(np.float64)[..., np.arange(M) // rows, :][..., np.arange(K) // 128]
    return TABLE[codes] * s


def linear(x, w):
    """(x W^T, sum of |x w|) in float64, x [M][K], w [N][K]."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def tolerance(y, mag, K, bf16=False):
    """How far a product's result may be from y. Products of codes, and of codes with BF16 values,
    are exact in fp32. A sum is a chain of at most K/32 matrix instructions, K/128 products with
    scales and as many additions, and some joins of partial sums (64 allowed for, and for the
    product of the two scales), each a rounding (or truncation: 2^-23) of at most the sum of
    magnitudes. A BF16 result is rounded once more, by half a step (2^-8)."""
    t = (K / 16 + 64) * 2.0 ** -23 * mag + 1e-37
    return t + 2.0 ** -8 * (np.abs(y) + t) if bf16 else t


def dropped(x, w):
    """What W8A8's products in BF16 may lose: the FP8 matrix instruction drops, of eight products
    of consecutive k, what lies below 2^-13 of the largest one's power of two: seven products may
    lose up to that much each. (k of one lane lie in runs of 16 from a multiple of 16 on.)"""
    t = np.zeros((x.shape[0], w.shape[0]))
    for k in range(0, x.shape[1], 8):
        a, b = np.abs(x[:, k:k + 8]), np.abs(w[:, k:k + 8])
        most = np.zeros_like(t)
        for i in range(a.shape[1]):
            np.maximum(most, np.multiply.outer(a[:, i], b[:, i]), out=most)
        t += most
    return 7 * 2.0 ** -13 * t


def route(logits, k, scoring="softmax", bias=None, groups=1, top_groups=None, group_score="max", renormalize=True, scale=1.0):
    """(ids, weights) of moe_route: scores in long double, places by stable sorts."""
    T, E = logits.shape
    rows = np.arange(T)[:, None]
    top_groups = groups if top_groups is None else top_groups
    l = logits.astype(np.longdouble)
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max))
    there = l > -np.inf
    with np.errstate(over="ignore", invalid="ignore"):
        if scoring == "softmax":
            p = np.where(there, np.exp(l - np.where(there.any(1), l.max(1), 0)[:, None]), 0)
            p = p / np.where(there.any(1), p.sum(1), 1)[:, None]
        else:
            p = np.where(there, 1 / (1 + np.exp(-l)), 0)
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    is_open = there & ~np.isnan(b) & (b > -np.inf)
    # without a bias the order is that of the logits
    c = l if bias is None and (groups == 1 or group_score == "max") else p + np.where(np.isnan(b), 0, b)
    c = np.where(is_open, c, -np.inf)
    if groups > 1:
        best = -np.sort(-c.reshape(T, groups, -1), axis=2)
        score = best[:, :, 0]
        if group_score == "top2" and best.shape[2] > 1:
            score = score + np.where(best[:, :, 1] > -np.inf, best[:, :, 1], 0)
        kept = np.zeros((T, groups), bool)
        kept[rows, np.argsort(-score, axis=1, kind="stable")[:, :top_groups]] = True
        c = np.where(np.repeat(kept, E // groups, 1), c, -np.inf)
    ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
    got = c[rows, ids] > -np.inf
    w = np.where(got, p[rows, ids], 0)
    if renormalize:
        total = w.sum(1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1), 0)
    return np.where(got, ids, -1).astype(np.int32), w * scale
