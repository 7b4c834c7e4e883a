"""MXFP4 in float64 numpy, from the format's definition (include/mxfp4.h), and the tolerances
of products: the plain implementation that the MXFP4 tests compare the library with."""
import numpy as np

MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """x [M][K] finite or not -> codes [M][K/2], scales [M][K/32] (uint8)."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    e = np.frexp(np.where(amax > 0, amax, 1.0))[1] - 1 - 2
    s = np.where(amax > 0, np.clip(e + 127, 0, 254), 0)
    q = np.ldexp(np.abs(b), (127 - s)[..., None])
    # distance to each magnitude; among equal distances the even code wins
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])
    d = np.abs(q[..., None] - MAGS[order])
    code = order[np.argmin(d, -1)] + 8 * np.signbit(np.where(bad[..., None], 0.0, x.reshape(b.shape)))
    code = np.where(bad[..., None], 0, code).reshape(x.shape).astype(np.uint8)
    s = np.where(bad, 255, s).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), s


def dequantize(codes, scales):
    """The values in float64; NaN where the scale is 0xFF."""
    table = np.concatenate([MAGS, -MAGS])
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = table[c].reshape(*scales.shape, 32)
    v = np.ldexp(v, (scales.astype(np.int64) - 127)[..., None])
    v = np.where((scales == 255)[..., None], np.nan, v)
    return v.reshape(c.shape)


def linear(x, w):
    """(x W^T, sum of |x w|) in float64, x [M][K], w [N][K]."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def tolerance(y, mag, K, bf16=False):
    """How far a product's result may be from y. Products of codes, and of codes with BF16
    values, are exact in fp32; a sum is a chain of at most K/32 matrix instructions and some
    joins of partial sums (32 allowed for), each a rounding (or truncation: 2^-23) of at most
    the sum of magnitudes. A BF16 result is rounded once more, by half a step (2^-8)."""
    t = (K / 32 + 64) * 2.0 ** -23 * mag + 1e-37
    return t + 2.0 ** -8 * (np.abs(y) + t) if bf16 else t


def swiglu(h, tol_h, half):
    """(silu(gate) * up, its tolerance before rounding to BF16) from h [R][2 * half]."""
    g, u = h[:, :half], h[:, half:]
    s = g / (1 + np.exp(-g))
    # |silu'| < 1.1; the hardware's exponential and reciprocal: a few fp32 steps (2^-20)
    t = 1.1 * tol_h[:, :half] * np.abs(u) + (np.abs(s) + 1.1 * tol_h[:, :half]) * tol_h[:, half:]
    return s * u, t + 2.0 ** -20 * np.abs(s * u)
