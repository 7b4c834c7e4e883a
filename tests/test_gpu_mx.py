"""The MXFP4 operators on the GPU against float64 numpy (mx_reference.py): quantization bit for
bit, products within the tolerance derived there, at the sizes and values where they can go
wrong."""
import numpy as np
import pytest
import torch

import mx_reference as ref
import nvfp4_block_scaled_linear_amd as nv
from gpu_helpers import device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return device()


def say(*a):
    print(*a, flush=True)


def rng_of(*key):
    return np.random.default_rng(list(key))


def acts(rng, M, K):
    """BF16 rows on the CPU: unit normal, a few loud channels."""
    x = rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.01, 20.0, 1.0)
    return torch.from_numpy(x).float().bfloat16()


def weight(rng, *shape):
    c, s = ref.quantize((0.02 * rng.standard_normal(shape)).reshape(-1, shape[-1]))
    return c.reshape(*shape[:-1], -1), s.reshape(*shape[:-1], -1)


def up(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def num(t):
    return t.double().cpu().numpy()


def act_operand(x, kind, dev):
    """(x, x_scales) for a call, and the values that the product sees."""
    if kind == "bf16":
        return (x.to(dev), None), num(x)
    c, s = ref.quantize(num(x))
    return (up(c, dev), up(s, dev)), ref.dequantize(c, s)


def assert_near(got, want, tol, what):
    got = num(got)
    assert got.shape == want.shape, (got.shape, want.shape)
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = np.argwhere(bad)[0]
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} values are off, first at {tuple(i)}: got {got[tuple(i)]}, want {want[tuple(i)]} +- {tol[tuple(i)]}")


# ------------------------------------------------------------------ quantize and back

def check_quantize(x, dev, what):
    c, s = nv.mxfp4_quantize(x)
    rc, rs = ref.quantize(num(x))
    assert np.array_equal(s.cpu().numpy(), rs), what
    assert np.array_equal(c.cpu().numpy(), rc), what
    return c, s


@pytest.mark.parametrize("M,K", [(1, 32), (1, 64), (3, 96), (5, 160), (7, 1056), (2, 4096), (1, 14336), (300, 288), (17, 6560)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_rows(dev, M, K, dtype):
    rng = rng_of(1, M, K)
    # rows of very different sizes, and blocks of very different sizes in a row
    x = rng.standard_normal((M, K)) * 2.0 ** rng.integers(-30, 30, (M, 1)) * 2.0 ** np.repeat(rng.integers(-20, 20, (M, K // 32)), 32, 1)
    check_quantize(torch.from_numpy(x).to(dtype).to(dev), dev, (M, K, dtype))


def test_quantize_every_bf16_value(dev):
    """Every finite BF16 value as the largest of its block, beside values on E2M1's decision
    points and their BF16 neighbours at that scale."""
    bits = np.arange(65536, dtype=np.int64)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    top = torch.from_numpy(bits.astype(np.uint16).view(np.int16)).view(torch.bfloat16)
    e = torch.frexp(top.float())[1].double() - 3
    points = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.2499, 0.2512, 1.242, 3.516, 4.98, -0.25, -0.75])
    rows = torch.ldexp(points.double()[None, :], e[:, None].int()).to(torch.bfloat16)
    rows = torch.where(rows.abs() <= top.abs()[:, None], rows, torch.zeros_like(rows))
    x = torch.zeros((bits.size, 32), dtype=torch.bfloat16)
    x[:, 3] = top
    x[:, 8:23] = rows
    check_quantize(x.to(dev), dev, "every BF16")


def test_quantize_fp32_decision_points(dev):
    """fp32 values next to every decision point, at scales from the least to the largest."""
    pts = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], np.float32)
    near = np.concatenate([pts, np.nextafter(pts, np.float32(0)), np.nextafter(pts, np.float32(9)), [np.float32(7.9999995)]])
    x = np.zeros((253, 32), np.float32)
    x[:, 0] = 4.0
    x[:, 1:1 + near.size] = near * np.where(np.arange(near.size) % 2, -1, 1)
    x = np.ldexp(x, (np.arange(253) - 127)[:, None]).astype(np.float32)
    check_quantize(up(x, dev), dev, "fp32 points")


def test_quantize_subnormal_zero_and_signed_zero(dev):
    x = np.zeros((4, 64), np.float32)
    x[0, ::2] = -0.0
    x[1, :32] = 2.0 ** -149 * np.arange(32)
    x[2, :32] = -(2.0 ** -127) * np.arange(32) / 16
    x[3] = np.ldexp(np.linspace(-1.9, 1.9, 64), -126)
    check_quantize(up(x, dev), dev, "subnormal")


def test_quantize_strided_rows_and_given_outputs(dev):
    rng = rng_of(2)
    for dtype in (torch.bfloat16, torch.float32):
        wide = torch.full((9, 512), float("nan"), dtype=dtype)
        wide[:, 64:64 + 160] = torch.from_numpy(rng.standard_normal((9, 160))).to(dtype)
        wide = wide.to(dev)
        x = wide[:, 64:64 + 160]
        codes = torch.full((11, 80), 0xA5, dtype=torch.uint8, device=dev)
        scales = torch.full((11, 5), 0xA5, dtype=torch.uint8, device=dev)
        nv.mxfp4_quantize(x, codes=codes[1:10], scales=scales[1:10])
        rc, rs = ref.quantize(num(x))
        assert np.array_equal(codes[1:10].cpu().numpy(), rc) and np.array_equal(scales[1:10].cpu().numpy(), rs)
        for t in (codes, scales):
            assert (t[0] == 0xA5).all() and (t[10] == 0xA5).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_quantize_non_finite(dev, dtype, bad):
    x = torch.from_numpy(rng_of(3).standard_normal((6, 128))).to(dtype)
    clean = x.clone().to(dev)
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    nv.mxfp4_quantize(clean, faults=word)
    assert int(word) == 0
    x[4, 37] = bad
    c, s = nv.mxfp4_quantize(x.to(dev), faults=word)
    assert int(word) == nv.FAULT_NONFINITE
    rc, rs = ref.quantize(num(x))
    assert rs[4, 1] == 255
    assert np.array_equal(c.cpu().numpy(), rc) and np.array_equal(s.cpu().numpy(), rs)
    y = nv.mxfp4_dequantize(c, s)
    assert torch.isnan(y[4, 32:64]).all() and int(torch.isnan(y).sum()) == 32


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dequantize_every_code_and_scale(dev, dtype):
    codes = np.tile(np.arange(256, dtype=np.uint8)[None, :], (256, 1))  # 16 blocks a row
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    y = nv.mxfp4_dequantize(up(codes, dev), up(scales, dev), dtype=dtype)
    assert y.dtype == dtype
    with np.errstate(over="ignore"):
        want = torch.from_numpy(ref.dequantize(codes, scales)).to(dtype)
    assert torch.equal(torch.isnan(y.cpu()), torch.isnan(want))
    ok = ~torch.isnan(want)
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
    assert torch.equal(y.cpu().view(bits)[ok], want.view(bits)[ok])  # -0 included


@pytest.mark.parametrize("M,K", [(1, 32), (3, 160), (1, 14336), (261, 1056)])
def test_dequantize_shapes_and_pitch(dev, M, K):
    rng = rng_of(4, M, K)
    c, s = weight(rng, M, K)
    want = ref.dequantize(c, s)
    assert np.array_equal(num(nv.mxfp4_dequantize(up(c, dev), up(s, dev))), want)
    out = torch.full((M, K + 64), 9.0, device=dev)
    nv.mxfp4_dequantize(up(c, dev), up(s, dev), out=out[:, 32:32 + K])
    assert np.array_equal(num(out[:, 32:32 + K]), want)
    assert (out[:, :32] == 9).all() and (out[:, 32 + K:] == 9).all()


# -------------------------------------------------------------------------- linear

LINEAR = [(1, 2048, 2048), (1, 1, 32), (1, 17, 64), (2, 33, 96), (4, 4096, 512), (7, 250, 160), (15, 31, 1056), (16, 1000, 4096),
          (17, 48, 288), (31, 96, 2048), (33, 1, 128), (48, 513, 416), (64, 256, 1024), (65, 130, 256), (100, 257, 352), (128, 384, 768),
          (130, 100, 4128), (257, 300, 544), (300, 1000, 32), (513, 515, 1024), (16, 24, 14336), (1, 12288, 96), (700, 259, 2080)]


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(dev, M, N, K, kind):
    say("linear", kind, M, N, K)
    rng = rng_of(5, M, N, K)
    x, (c, s) = acts(rng, M, K), weight(rng, N, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    want, mag = ref.linear(xv, ref.dequantize(c, s))
    cd, sd = up(c, dev), up(s, dev)
    y = nv.mxfp4_linear(xd, cd, sd, x_scales=xs)
    assert y.dtype == torch.float32
    assert_near(y, want, ref.tolerance(want, mag, K), (kind, M, N, K))
    yb = nv.mxfp4_linear(xd, cd, sd, x_scales=xs, out_dtype=torch.bfloat16)
    assert torch.equal(yb, y.bfloat16())
    assert torch.equal(nv.mxfp4_linear(xd, cd, sd, x_scales=xs), y)  # the same on every run


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_linear_offsets_past_32_bits(dev, kind):
    """A weight, and activations, of more than 2^31 bytes: 509 rows over and over."""
    K, P = 8192, 509
    rng = rng_of(15)
    c, s = weight(rng, P, K)
    x = acts(rng, P, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    want, mag = ref.linear(xv, ref.dequantize(c, s))
    tol = ref.tolerance(want, mag, K)
    cd, sd = up(c, dev), up(s, dev)
    N = 2 ** 19 + 77
    which = torch.arange(N, device=dev) % P
    wc, ws = cd[which], sd[which]
    cols = np.r_[0:300, N // 2:N // 2 + 300, N - 300:N]
    for M in (1, 3, 33, 130):
        say("weight past 2^31 bytes", kind, M)
        y = nv.mxfp4_linear(xd[:M], wc, ws, x_scales=None if xs is None else xs[:M], out_dtype=torch.float32)
        assert_near(y[:, cols], want[:M, cols % P], tol[:M, cols % P], ("weight", M))
    del wc, ws, y
    M = 2 ** 17 + 77 if kind == "bf16" else 2 ** 19 + 77
    which = torch.arange(M, device=dev) % P
    big, bs = xd[which], None if xs is None else xs[which]
    rows = np.r_[0:300, M // 2:M // 2 + 300, M - 300:M]
    for N in (1, 70):
        say("activations past 2^31 bytes", kind, N)
        y = nv.mxfp4_linear(big, cd[:N], sd[:N], x_scales=bs)
        assert_near(y[rows], want[rows % P][:, :N], tol[rows % P][:, :N], ("activations", N))
    if kind == "bf16":
        qc, qs = nv.mxfp4_quantize(big)
        rc, rs = (up(a, dev) for a in ref.quantize(num(xd)))
        assert torch.equal(qc[rows], rc[rows % P]) and torch.equal(qs[rows], rs[rows % P])
        back = nv.mxfp4_dequantize(qc, qs)
        assert np.array_equal(num(back[rows]), ref.dequantize(rc.cpu().numpy(), rs.cpu().numpy())[rows % P])


# enough rows and columns for LDS tiles of 64 x 128, 128 x 128, 128 x 256 and 256 x 256, ragged
# in both, each with K of whole stages, of a part of one, and with scale rows off the dword
@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("K", [32, 160, 256, 416, 768, 1536])
@pytest.mark.parametrize("M,N", [(330, 4001), (1000, 3300), (1500, 4404), (2500, 5400)])
def test_linear_tiles(dev, M, N, K, kind):
    say("linear tiles", kind, M, N, K)
    rng = rng_of(15, M, N, K)
    x, (c, s) = acts(rng, M, K), weight(rng, N, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    keep = np.unique(np.concatenate([np.arange(0, M, 37), [M - 1, M - 2]]))  # rows for the reference
    want, mag = ref.linear(xv[keep], ref.dequantize(c, s))
    cd, sd = up(c, dev), up(s, dev)
    y = nv.mxfp4_linear(xd, cd, sd, x_scales=xs)
    assert_near(y[torch.from_numpy(keep).to(dev)], want, ref.tolerance(want, mag, K), (kind, M, N, K))
    # every row against the same rows in calls of 32, which stream the weight: both are within
    # the tolerance of the true value; the magnitudes from the codes without their signs
    parts = torch.cat([nv.mxfp4_linear(xd[i:i + 32], cd, sd, x_scales=None if xs is None else xs[i:i + 32]) for i in range(0, M, 32)])
    mags = num(nv.mxfp4_linear(xd.abs() if xs is None else xd & 0x77, cd & 0x77, sd, x_scales=xs)) * 1.01
    assert_near(y, num(parts), 2 * ref.tolerance(num(parts), mags, K), "rows")
    yb = nv.mxfp4_linear(xd, cd, sd, x_scales=xs, out_dtype=torch.bfloat16)
    assert torch.equal(yb, y.bfloat16())
    buf = torch.full((s.size + 3,), 255, dtype=torch.uint8, device=dev)
    off = buf[3:].view(N, K // 32)
    off.copy_(sd)
    wide = torch.full((M, N + 3), 5.0, device=dev)
    nv.mxfp4_linear(xd, cd, off, x_scales=xs, out=wide[:, 1:1 + N])
    assert_near(wide[:, 1:1 + N], num(y), 2 * ref.tolerance(num(y), mags, K), "offset scales and columns")
    assert (wide[:, 0] == 5).all() and (wide[:, N + 1:] == 5).all()


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,E,k,N,K", [(4200, 8, 2, 1088, 416), (1800, 3, 2, 640, 768), (2100, 40, 2, 576, 288)])
def test_grouped_tiles(dev, T, E, k, N, K, kind):
    """Prompt-sized groups: rows against float64, the other forms against the rows."""
    say("grouped tiles", kind, T, E, k, N, K)
    rng = rng_of(16, T, E)
    ids, tw = routes(rng, T, E, k)
    ids[5] = -1
    x, (c, s) = acts(rng, T, K), weight(rng, E, N, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    args = (xd, up(c, dev), up(s, dev), up(ids, dev))
    rows = nv.mxfp4_grouped_linear(*args, x_scales=xs)
    flat, tok = ids.reshape(-1), np.arange(T * k) // k
    for e in (0, E // 2, E - 1):
        mine = np.flatnonzero(flat == e)[::11]
        y, mag = ref.linear(xv[tok[mine]], ref.dequantize(c[e], s[e]))
        assert_near(rows[torch.from_numpy(mine).to(dev)], y, ref.tolerance(y, mag, K), ("expert", e))
    assert not rows[5 * k:6 * k].any()
    assert torch.equal(nv.mxfp4_grouped_linear(*args, x_scales=xs, out_dtype=torch.bfloat16), rows.bfloat16())
    a = nv.mxfp4_grouped_linear(*args, x_scales=xs, out_mode=nv.OUT_SWIGLU_BF16)
    h = num(rows)
    want, t = ref.swiglu(h, 0 * h, N // 2)
    assert_near(a, want, t + 2.0 ** -8 * (np.abs(want) + t) + 1e-37, "swiglu")
    if N % 64 == 0:
        qc, qs = nv.mxfp4_grouped_linear(*args, x_scales=xs, out_mode=nv.OUT_SWIGLU_MXFP4)
        rc, rs = nv.mxfp4_quantize(a)
        assert torch.equal(qs, rs) and torch.equal(qc, rc)
    out = num(nv.mxfp4_grouped_linear(*args, x_scales=xs, topk_w=up(tw, dev), out_mode=nv.OUT_COMBINE))
    terms = h.reshape(T, k, N) * tw[..., None].astype(np.float64)
    assert np.all(np.abs(out - terms.sum(1)) <= (k + 1) * 2.0 ** -24 * np.abs(terms).sum(1) + 1e-37)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_linear_pitched_views_and_what_lies_around(dev, M, kind):
    """x rows inside a wider NaN buffer, y columns inside a wider one; scales at odd addresses."""
    N, K = 75, 352
    rng = rng_of(6, M)
    x, (c, s) = acts(rng, M, K), weight(rng, N, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    if kind == "bf16":
        wide = torch.full((M + 1, K + 64), float("nan"), dtype=torch.bfloat16, device=dev)
        wide[:M, 8:8 + K] = xd
        xd = wide[:M, 8:8 + K]
    buf = torch.full((s.size + 2,), 255, dtype=torch.uint8, device=dev)
    sd = buf[1:-1].view(N, K // 32)
    sd.copy_(up(s, dev))
    want, mag = ref.linear(xv, ref.dequantize(c, s))
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((M + 2, N + 9), 7.0, dtype=dtype, device=dev)
        nv.mxfp4_linear(xd, up(c, dev), sd, x_scales=xs, out=out[1:M + 1, 3:3 + N])
        assert_near(out[1:M + 1, 3:3 + N], want, ref.tolerance(want, mag, K, dtype == torch.bfloat16), (kind, M, dtype))
        rest = out.clone()
        rest[1:M + 1, 3:3 + N] = 7.0
        assert (rest == 7).all()


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("M", [1, 20, 150])
def test_linear_extreme_scales(dev, M, kind):
    """Weight scales over the whole E8M0 range, each in a row of its own."""
    N, K = 255, 64
    rng = rng_of(7, M)
    c = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    s = np.repeat(np.arange(255, dtype=np.uint8)[:, None], 2, 1)
    x = acts(rng, M, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    w = ref.dequantize(c, s)
    want, mag = ref.linear(xv, w)
    y = num(nv.mxfp4_linear(xd, up(c, dev), up(s, dev), x_scales=xs))
    # results of 2^126 and more may overflow on the way, in a partial sum or in the decode
    safe = (mag.max(0) < 2.0 ** 126) & (np.abs(w).max(1) < 2.0 ** 126)
    # a value below fp32's and BF16's smallest normal may be taken as zero
    tol = ref.tolerance(want, mag, K) + 2.0 ** -126 * np.abs(xv).sum(1)[:, None]
    assert safe.sum() > 240
    assert np.all(np.abs(y - want)[:, safe] <= tol[:, safe])


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("M", [1, 20, 150])
def test_linear_nan_scales_and_check_mode(dev, M, kind):
    N, K = 70, 288
    rng = rng_of(8, M)
    x, (c, s) = acts(rng, M, K), weight(rng, N, K)
    (xd, xs), _ = act_operand(x, kind, dev)
    cd, sd = up(c, dev), up(s, dev)
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    clean = nv.mxfp4_linear(xd, cd, sd, x_scales=xs, check=True, faults=word)
    assert int(word) == 0
    sd[69, 8] = 255
    y = nv.mxfp4_linear(xd, cd, sd, x_scales=xs, faults=word)
    assert int(word) == 0  # nothing is scanned without the flag
    assert torch.isnan(y[:, 69]).all() and torch.equal(y[:, :69], clean[:, :69])
    assert torch.equal(nv.mxfp4_linear(xd, cd, sd, x_scales=xs, check=True, faults=word)[:, :69], clean[:, :69])
    assert int(word) == nv.FAULT_NAN_SCALE
    sd = up(s, dev)
    word.zero_()
    if kind == "bf16":
        xd[M - 1, 100] = float("inf")
        nv.mxfp4_linear(xd, cd, sd, check=True, faults=word)
        assert int(word) == nv.FAULT_NONFINITE
    else:
        xs[M - 1, 5] = 255
        y = nv.mxfp4_linear(xd, cd, sd, x_scales=xs, check=True, faults=word)
        assert int(word) == nv.FAULT_NAN_SCALE
        assert torch.isnan(y[M - 1]).all() and torch.equal(y[:M - 1], clean[:M - 1])


def test_linear_non_finite_rows_stay_in_their_rows(dev):
    M, N, K = 37, 90, 160
    rng = rng_of(9)
    x, (c, s) = acts(rng, M, K), weight(rng, N, K)
    cd, sd = up(c, dev), up(s, dev)
    clean = nv.mxfp4_linear(x.to(dev), cd, sd)
    x[5, 3], x[20, 159] = float("nan"), float("inf")
    y = nv.mxfp4_linear(x.to(dev), cd, sd)
    assert torch.isnan(y[5]).all() and not torch.isfinite(y[20]).all()
    keep = [m for m in range(M) if m not in (5, 20)]
    assert torch.equal(y[keep], clean[keep])


# ------------------------------------------------------------------------- grouped

def routes(rng, T, E, k, skew=1.0):
    liking = skew * rng.standard_normal(E)
    noise = rng.gumbel(size=(T, E))
    ids = np.argsort(-(liking + noise), axis=1)[:, :k].astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    return np.ascontiguousarray(ids), w / w.sum(1, keepdims=True)


def route_rows(xv, w, ids, per_route):
    """float64 rows [R][N] of the routes and their magnitudes; zeros for ids out of range and
    for repeats of an id within a token."""
    T, k = ids.shape
    y, mag = np.zeros((T * k, w.shape[1])), np.zeros((T * k, w.shape[1]))
    kept = np.zeros(T * k, bool)
    for r in range(T * k):
        t, j = divmod(r, k)
        e = ids[t, j]
        kept[r] = 0 <= e < w.shape[0] and e not in ids[t, :j]
    for e in range(w.shape[0]):
        mine = np.flatnonzero(kept & (ids.reshape(-1) == e))
        y[mine], mag[mine] = ref.linear(xv[mine if per_route else mine // k], w[e])
    return y, mag, kept


GROUPED = [(1, 4, 1, 64, 32), (1, 128, 8, 128, 2048), (16, 128, 8, 192, 256), (5, 3, 3, 130, 96), (40, 6, 2, 64, 1056),
           (333, 24, 3, 66, 160), (200, 2, 1, 256, 512), (64, 300, 4, 128, 64), (700, 8, 2, 320, 288), (1500, 5, 2, 130, 128),
           (100, 128, 4, 128, 160), (300, 64, 2, 66, 544), (256, 40, 1, 192, 64), (257, 40, 1, 64, 96), (90, 200, 64, 64, 32), (4, 70, 64, 64, 64)]


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,E,k,N,K", GROUPED)
def test_grouped_routes_swiglu_combine(dev, T, E, k, N, K, kind):
    say("grouped", kind, T, E, k, N, K)
    rng = rng_of(10, T, E, k, N, K)
    ids, tw = routes(rng, T, E, k)
    x, (c, s) = acts(rng, T, K), weight(rng, E, N, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    y, mag, _ = route_rows(xv, ref.dequantize(c, s), ids, False)
    tol = ref.tolerance(y, mag, K)
    args = (xd, up(c, dev), up(s, dev), up(ids, dev))
    rows = nv.mxfp4_grouped_linear(*args, x_scales=xs)
    assert rows.dtype == torch.float32
    assert_near(rows, y, tol, "routes")
    assert torch.equal(nv.mxfp4_grouped_linear(*args, x_scales=xs, out_dtype=torch.bfloat16), rows.bfloat16())
    # SwiGLU
    want, t = ref.swiglu(y, tol, N // 2)
    a = nv.mxfp4_grouped_linear(*args, x_scales=xs, out_mode=nv.OUT_SWIGLU_BF16)
    assert a.dtype == torch.bfloat16
    assert_near(a, want, t + 2.0 ** -8 * (np.abs(want) + t), "swiglu")
    if N % 64 == 0:  # to MXFP4: bit for bit the quantizer's view of the BF16 rows
        qc, qs = nv.mxfp4_grouped_linear(*args, x_scales=xs, out_mode=nv.OUT_SWIGLU_MXFP4)
        rc, rs = nv.mxfp4_quantize(a)
        assert torch.equal(qs, rs) and torch.equal(qc, rc)
    # combine
    want = (y.reshape(T, k, N) * tw[..., None].astype(np.float64)).sum(1)
    absw = (np.abs(y).reshape(T, k, N) * tw[..., None]).sum(1)
    t = (tol.reshape(T, k, N) * tw[..., None]).sum(1) + (k + 1) * 2.0 ** -24 * absw + 1e-37
    out = nv.mxfp4_grouped_linear(*args, x_scales=xs, topk_w=up(tw, dev), out_mode=nv.OUT_COMBINE)
    assert_near(out, want, t, "combine")
    outb = nv.mxfp4_grouped_linear(*args, x_scales=xs, topk_w=up(tw, dev), out_mode=nv.OUT_COMBINE, out_dtype=torch.bfloat16)
    assert torch.equal(outb, out.bfloat16())


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,E,k", [(9, 7, 3), (120, 40, 5), (300, 7, 3), (2500, 4, 2)])
def test_grouped_bad_routes(dev, T, E, k, kind):
    """Ids out of range and repeated: flagged, their rows zero, the others as without them."""
    N, K = 128, 96
    rng = rng_of(11, T)
    ids, tw = routes(rng, T, E, k)
    ids[0, 0], ids[T // 2, 1], ids[T - 1, k - 1] = -1, E, 2 ** 31 - 1
    ids[1, 1] = ids[1, 0]
    ids[T // 3] = -5  # a token without any route
    x, (c, s) = acts(rng, T, K), weight(rng, E, N, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    y, mag, kept = route_rows(xv, ref.dequantize(c, s), ids, False)
    args = (xd, up(c, dev), up(s, dev), up(ids, dev))
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    out = torch.full((T * k, N), float("nan"), device=dev)
    nv.mxfp4_grouped_linear(*args, x_scales=xs, out=out, faults=word)
    assert int(word) == nv.FAULT_BAD_ROUTE
    assert_near(out, y, ref.tolerance(y, mag, K), "bad routes")
    assert (out.cpu().numpy()[~kept] == 0).all()
    qc = torch.full((T * k, N // 4), 0xA5, dtype=torch.uint8, device=dev)
    qs = torch.full((T * k, N // 64), 0xA5, dtype=torch.uint8, device=dev)
    nv.mxfp4_grouped_linear(*args, x_scales=xs, out_mode=nv.OUT_SWIGLU_MXFP4, out=qc, out_scales=qs)
    assert not qc.cpu().numpy()[~kept].any() and not qs.cpu().numpy()[~kept].any()
    rc, rs = nv.mxfp4_quantize(nv.mxfp4_grouped_linear(*args, x_scales=xs, out_mode=nv.OUT_SWIGLU_BF16))
    assert torch.equal(qc, rc) and torch.equal(qs, rs)
    comb = nv.mxfp4_grouped_linear(*args, x_scales=xs, topk_w=up(tw, dev), out_mode=nv.OUT_COMBINE)
    assert (comb[T // 3] == 0).all()
    want = (y.reshape(T, k, N) * tw[..., None].astype(np.float64)).sum(1)
    t = ((ref.tolerance(y, mag, K) + (k + 1) * 2.0 ** -24 * np.abs(y)).reshape(T, k, N) * tw[..., None]).sum(1) + 1e-37
    assert_near(comb, want, t, "combine")


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,E,k", [(24, 40, 5), (300, 40, 3), (400, 7, 4), (2500, 4, 2)])
@pytest.mark.parametrize("real", [0, 1, 0.4])
def test_grouped_padded_batch(dev, T, E, k, kind, real):
    """A batch whose last tokens have no expert: zeros there in every form, whatever lay there,
    and the other tokens' rows as in a batch of theirs alone."""
    K, n = 96, int(T * real) if real < 1 else 1
    rng = rng_of(14, T)
    ids, tw = routes(rng, T, E, k)
    ids[n:] = -1
    x = acts(rng, T, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    ids_d, tw_d = up(ids, dev), up(tw, dev)
    for N, mode, dtype in ((193, nv.OUT_ROUTES, torch.bfloat16), (193, nv.OUT_ROUTES, torch.float32),
                           (130, nv.OUT_SWIGLU_BF16, torch.bfloat16), (134, nv.OUT_SWIGLU_BF16, torch.bfloat16),
                           (192, nv.OUT_SWIGLU_MXFP4, torch.uint8), (193, nv.OUT_COMBINE, torch.float32)):
        c, s = weight(rng, E, N, K)
        per = 1 if mode == nv.OUT_COMBINE else k
        cols = {nv.OUT_SWIGLU_BF16: N // 2, nv.OUT_SWIGLU_MXFP4: N // 4}.get(mode, N)
        out = torch.full((T * per, cols), 77, dtype=dtype, device=dev)
        osc = torch.full((T * k, N // 64), 77, dtype=torch.uint8, device=dev) if mode == nv.OUT_SWIGLU_MXFP4 else None
        word = torch.zeros(1, dtype=torch.int32, device=dev)
        cd, sd = up(c, dev), up(s, dev)
        nv.mxfp4_grouped_linear(xd, cd, sd, ids_d, topk_w=tw_d, x_scales=xs, out_mode=mode, out=out, out_scales=osc, faults=word)
        assert int(word) == nv.FAULT_BAD_ROUTE
        assert not out[n * per:].any() and (osc is None or not osc[n * k:].any())
        if mode == nv.OUT_ROUTES and dtype == torch.float32 and n:
            y, mag, _ = route_rows(xv[:n], ref.dequantize(c, s), ids[:n], False)
            assert_near(out[:n * k], y, ref.tolerance(y, mag, K), "kept rows")
        elif n:
            assert out[:n * per].any()


def test_grouped_all_on_one_expert_and_one_row_each(dev):
    N, K, E = 96, 128, 40
    rng = rng_of(12)
    c, s = weight(rng, E, N, K)
    w = ref.dequantize(c, s)
    for ids in (np.full((200, 1), 39, np.int32), np.full((259, 1), 17, np.int32), np.full((2000, 1), 0, np.int32),
                np.arange(E, dtype=np.int32)[:, None]):
        x = acts(rng, ids.shape[0], K)
        y, mag, _ = route_rows(num(x), w, ids, False)
        got = nv.mxfp4_grouped_linear(x.to(dev), up(c, dev), up(s, dev), up(ids, dev))
        assert_near(got, y, ref.tolerance(y, mag, K), ids.shape)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 16, 100, 1200])
def test_moe_layer(dev, T, kind):
    """A layer as it is used: quantize, gate_up with SwiGLU, down with the combine reusing the
    grouping, one workspace; each step against float64 on its own inputs."""
    E, k, H, I = 16, 4, 256, 160
    rng = rng_of(13, T)
    ids, tw = routes(rng, T, E, k)
    gu, dn = weight(rng, E, 2 * I, H), weight(rng, E, H, I)
    x = acts(rng, T, H).to(dev)
    idd, twd = up(ids, dev), up(tw, dev)
    size = max(nv.mxfp4_grouped_workspace_size(T, k, 2 * I, H, E, nv.OUT_SWIGLU_BF16), nv.mxfp4_grouped_workspace_size(T, k, H, I, E, nv.OUT_COMBINE))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=dev)
    if kind == "bf16":
        xv = num(x)
        a = nv.mxfp4_grouped_linear(x, up(gu[0], dev), up(gu[1], dev), idd, out_mode=nv.OUT_SWIGLU_BF16, workspace=ws)
        a_s, av = None, num(a)
    else:
        xq = nv.mxfp4_quantize(x)
        xv = ref.dequantize(*(t.cpu().numpy() for t in xq))
        a, a_s = nv.mxfp4_grouped_linear(xq[0], up(gu[0], dev), up(gu[1], dev), idd, x_scales=xq[1], out_mode=nv.OUT_SWIGLU_MXFP4, workspace=ws)
        av = ref.dequantize(a.cpu().numpy(), a_s.cpu().numpy())
    y, mag, _ = route_rows(xv, ref.dequantize(*gu), ids, False)
    want, t = ref.swiglu(y, ref.tolerance(y, mag, H), I)
    if kind == "bf16":
        assert_near(a, want, t + 2.0 ** -8 * (np.abs(want) + t), "gate_up")
    else:
        rc, rs = ref.quantize(torch.from_numpy(want).bfloat16().double().numpy())
        # one BF16 step may move a value over a decision point, or its block's scale
        assert np.mean(ref.dequantize(rc, rs) != av) < 0.01
    out = nv.mxfp4_grouped_linear(a, up(dn[0], dev), up(dn[1], dev), idd, x_scales=a_s, topk_w=twd, out_mode=nv.OUT_COMBINE,
                                  rows_per_route=True, workspace=ws, reuse_grouping=True)
    again = nv.mxfp4_grouped_linear(a, up(dn[0], dev), up(dn[1], dev), idd, x_scales=a_s, topk_w=twd, out_mode=nv.OUT_COMBINE,
                                    rows_per_route=True)
    assert torch.equal(out, again)
    y, mag, _ = route_rows(av, ref.dequantize(*dn), ids, True)
    want = (y.reshape(T, k, H) * tw[..., None].astype(np.float64)).sum(1)
    t = ((ref.tolerance(y, mag, I) + (k + 1) * 2.0 ** -24 * np.abs(y)).reshape(T, k, H) * tw[..., None]).sum(1) + 1e-37
    assert_near(out, want, t, "down")


# ------------------------------------------------- streams, graphs, calls side by side

def layer_calls(dev, T, seed):
    """A closure that runs quantize, linear and a W4A4 layer into given buffers."""
    E, k, H, I = 8, 2, 128, 64
    rng = rng_of(14, T, seed)
    ids, tw = routes(rng, T, E, k)
    x = acts(rng, T, H).to(dev)
    lin, gu, dn = ([up(t, dev) for t in weight(rng, *shape)] for shape in ((90, H), (E, 2 * I, H), (E, H, I)))
    idd, twd = up(ids, dev), up(tw, dev)
    size = max(nv.mxfp4_grouped_workspace_size(T, k, 2 * I, H, E, nv.OUT_SWIGLU_BF16), nv.mxfp4_grouped_workspace_size(T, k, H, I, E, nv.OUT_COMBINE))
    u8 = dict(dtype=torch.uint8, device=dev)
    ws = torch.empty(size, **u8)
    xc, xs, a, a_s = torch.empty((T, H // 2), **u8), torch.empty((T, H // 32), **u8), torch.empty((T * k, I // 2), **u8), torch.empty((T * k, I // 32), **u8)
    y, y16, out, back = torch.empty((T, 90), device=dev), torch.empty((T, 90), device=dev), torch.empty((T, H), device=dev), torch.empty((T, H), device=dev)

    def run():
        nv.mxfp4_quantize(x, codes=xc, scales=xs)
        nv.mxfp4_dequantize(xc, xs, out=back)
        nv.mxfp4_linear(xc, *lin, x_scales=xs, out=y)
        nv.mxfp4_linear(x, *lin, out=y16)
        nv.mxfp4_grouped_linear(xc, *gu, idd, x_scales=xs, out_mode=nv.OUT_SWIGLU_MXFP4, out=a, out_scales=a_s, workspace=ws)
        nv.mxfp4_grouped_linear(a, *dn, idd, x_scales=a_s, topk_w=twd, out_mode=nv.OUT_COMBINE, rows_per_route=True, out=out, workspace=ws, reuse_grouping=True)

    return run, [xc, xs, back, y, y16, a, a_s, out]


@pytest.mark.parametrize("T", [1, 12, 70, 600, 2500])
def test_graph_replays(dev, T):
    run, outs = layer_calls(dev, T, 0)
    other, _ = layer_calls(dev, T + 3, 1)
    run()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for i in range(4):
        for o in outs:
            o.view(torch.uint8).fill_(0xA5)
        other()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o.view(torch.uint8), w.view(torch.uint8)), f"replay {i}"


def test_two_streams_at_once(dev):
    """Two layers with workspaces of their own on two streams, several times, give what each
    gives alone."""
    pairs = [layer_calls(dev, 200, 2), layer_calls(dev, 310, 3)]
    for run, _ in pairs:
        run()
    torch.cuda.synchronize()
    want = [[o.clone() for o in outs] for _, outs in pairs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _, outs in pairs:
        for o in outs:
            o.view(torch.uint8).fill_(0xA5)
    torch.cuda.synchronize()
    for _ in range(5):
        for (run, _), st in zip(pairs, streams):
            with torch.cuda.stream(st):
                run()
    torch.cuda.synchronize()
    for (_, outs), ws in zip(pairs, want):
        for o, w in zip(outs, ws):
            assert torch.equal(o.view(torch.uint8), w.view(torch.uint8))


# ------------------------------------------------------------------------ refusals

def test_binding_refusals(dev):
    u8 = dict(dtype=torch.uint8, device=dev)
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=dev)
    c, s = torch.zeros((8, 32), **u8), torch.zeros((8, 2), **u8)
    ids = torch.zeros((4, 1), dtype=torch.int32, device=dev)
    for call in (
        lambda: nv.mxfp4_quantize(x.half()), lambda: nv.mxfp4_quantize(x.t()), lambda: nv.mxfp4_quantize(x[0]),
        lambda: nv.mxfp4_quantize(x, codes=c), lambda: nv.mxfp4_quantize(x, faults=torch.zeros(1, device=dev)),
        lambda: nv.mxfp4_dequantize(c, s[:, :1]), lambda: nv.mxfp4_dequantize(c[:, ::2], s), lambda: nv.mxfp4_dequantize(c, s, dtype=torch.half),
        lambda: nv.mxfp4_linear(x[:, :32], c, s), lambda: nv.mxfp4_linear(x.float(), c, s), lambda: nv.mxfp4_linear(x, c, s.int()),
        lambda: nv.mxfp4_linear(x, c, s, x_scales=s), lambda: nv.mxfp4_linear(x, c, s, out_dtype=torch.half),
        lambda: nv.mxfp4_linear(x, c, s, out=torch.empty((4, 7), device=dev)), lambda: nv.mxfp4_linear(x, c[:, :8], s),
        lambda: nv.mxfp4_linear(x.cpu(), c, s), lambda: nv.mxfp4_linear(c[:4, :16], c, s, x_scales=s[:4]),
        lambda: nv.mxfp4_grouped_linear(x, c[None], s[None], ids.long()), lambda: nv.mxfp4_grouped_linear(x[:3], c[None], s[None], ids),
        lambda: nv.mxfp4_grouped_linear(x, c, s, ids), lambda: nv.mxfp4_grouped_linear(x, c[None], s[None], ids, out_mode=9),
        lambda: nv.mxfp4_grouped_linear(x, c[None], s[None], ids, reuse_grouping=True),
        lambda: nv.mxfp4_grouped_linear(x, c[None], s[None], ids, out_scales=s),
        lambda: nv.mxfp4_grouped_linear(x, c[None], s[None], ids, out=torch.empty((4, 9), device=dev)),
    ):
        with pytest.raises(ValueError):
            call()
    for call, name in (
        (lambda: nv.mxfp4_quantize(x[:, :40]), "SHAPE"), (lambda: nv.mxfp4_quantize(x[:0]), "SHAPE"), (lambda: nv.mxfp4_quantize(x[:, 4:36]), "ALIGN"),
        (lambda: nv.mxfp4_linear(x[:0], c, s), "SHAPE"), (lambda: nv.mxfp4_linear(x, c, s, check=True), "NULL"),
        (lambda: nv.mxfp4_grouped_linear(x, c[None], s[None], ids, out_mode=nv.OUT_COMBINE), "NULL"),
        (lambda: nv.mxfp4_grouped_linear(x, c[None], s[None], ids, out_mode=nv.OUT_SWIGLU_MXFP4), "SHAPE"),
        (lambda: nv.mxfp4_grouped_linear(x, c[None], s[None], ids, out_mode=nv.OUT_SWIGLU_BF16, out_dtype=torch.float32), "ARG"),
        (lambda: nv.mxfp4_grouped_linear(x, c[None], s[None], ids, workspace=torch.empty(128, **u8)), "WORKSPACE"),
        (lambda: nv.mxfp4_grouped_linear(x, c[None], s[None], torch.zeros((4, 2), dtype=torch.int32, device=dev)), "ARG"),
    ):
        with pytest.raises(nv.NVFP4Error, match=name):
            call()
