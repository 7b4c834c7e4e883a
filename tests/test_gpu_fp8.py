"""The FP8 operators on the GPU against float64 numpy (f8_reference.py): quantization bit for bit,
products within the tolerance derived there, at the sizes and values where they can go wrong."""
import numpy as np
import pytest
import torch

import f8_reference as ref
import nvfp4_block_scaled_linear_amd as nv
from gpu_helpers import device

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    return device()


def say(*a):
    print(*a, flush=True)


def rng_of(*key):
    return np.random.default_rng([8, *key])


def acts(rng, M, K):
    """BF16 rows on the CPU: unit normal, a few loud channels."""
    x = rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.01, 20.0, 1.0)
    return torch.from_numpy(x).float().bfloat16()


def weight(rng, *shape):
    """Codes and scales of a normal weight whose rows differ in size (a stack: [E][N][K])."""
    w = 0.02 * rng.standard_normal(shape) * np.exp(0.5 * rng.standard_normal((*shape[:-1], 1)))
    parts = [ref.quantize(one, 128) for one in w.reshape(-1, *shape[-2:])]
    c, s = np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts])
    return c.reshape(shape), s.reshape(*shape[:-2], *s.shape[1:])


def up(a, dev):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    return t.view(F8) if t.dtype == torch.uint8 else t


def raw(t):
    return t.view(torch.uint8)


def num(t):
    return t.double().cpu().numpy()


def act_operand(x, kind, dev):
    """(x, x_scales) for a call, and the values that the product sees."""
    if kind == "bf16":
        return (x.to(dev), None), num(x)
    c, s = ref.quantize(num(x))
    return (up(c, dev), up(s, dev)), ref.dequantize(c, s)


def assert_near(got, want, tol, what):
    got = num(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (got.shape, want.shape)
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} values are off, first at {i}: got {got[i]}, want {want[i]} +- {tol[i]}")


# ------------------------------------------------------------------ quantize and back

def check_quantize(x, dev, what, rows=1, pow2=False):
    c, s = nv.fp8_quantize(x, block_rows=rows, pow2_scales=pow2)
    rc, rs = ref.quantize(x.float().cpu().numpy(), rows, pow2)
    assert c.dtype == F8 and s.dtype == torch.float32
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True), what
    assert np.array_equal(raw(c).cpu().numpy(), rc), what
    return c, s


@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (5, 272), (130, 1056), (2, 4096), (1, 14336), (300, 304), (257, 48)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantize(dev, M, K, dtype, rows, pow2):
    rng = rng_of(1, M, K)
    # rows of very different sizes, and blocks of very different sizes in a row
    x = rng.standard_normal((M, K)) * 2.0 ** rng.integers(-30, 30, (M, 1)) * 2.0 ** np.repeat(rng.integers(-20, 20, (M, -(-K // 128))), 128, 1)[:, :K]
    check_quantize(torch.from_numpy(x).to(dtype).to(dev), dev, (M, K, dtype), rows, pow2)


def test_quantize_every_bf16_value(dev):
    """Every finite BF16 value as the largest of its block, beside values on E4M3's decision
    points and next to them at that scale."""
    bits = np.arange(65536, dtype=np.int64)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    top = torch.from_numpy(bits.astype(np.uint16).view(np.int16)).view(torch.bfloat16)
    s = top.double().abs() / 448
    points = torch.from_numpy(np.concatenate([ref.MIDS[:118:2], -ref.MIDS[1:118:2], [448, 0.0009, -0.00098]]))
    rows = (points[None, :] * s[:, None]).to(torch.bfloat16)
    x = torch.zeros((bits.size, 128), dtype=torch.bfloat16)
    x[:, 3] = top
    x[:, 6:6 + points.numel()] = torch.where(rows.abs() <= top.abs()[:, None], rows, torch.zeros_like(rows))
    check_quantize(x.to(dev), dev, "every BF16")
    check_quantize(x.to(dev), dev, "every BF16", pow2=True)


def test_quantize_fp32_decision_points(dev):
    """fp32 values on and next to every decision point of E4M3, at scales from subnormal to the
    largest, powers of two and others."""
    pts = ref.MIDS.astype(np.float32)
    near = np.concatenate([pts, np.nextafter(pts, np.float32(0)), np.nextafter(pts, np.float32(999))])
    near = near[:384].reshape(3, 128) if near.size >= 384 else np.resize(near, (3, 128))
    near[:, 0] = 448
    near[1] *= -1
    with np.errstate(over="ignore"):
        x = np.concatenate([np.ldexp(near, e) for e in range(-158, 120)] + [near * np.float32(f) for f in rng_of(2).lognormal(0, 30, 400)])
    x = x[np.isfinite(x).all(1)].astype(np.float32)
    check_quantize(torch.from_numpy(x).to(dev), dev, "fp32 points")
    check_quantize(torch.from_numpy(x).to(dev), dev, "fp32 points", pow2=True)


def test_quantize_random_bits(dev):
    """Any finite fp32 bits, most blocks of few exponents."""
    rng = rng_of(3)
    bits = rng.integers(0, 1 << 32, (4096, 128), dtype=np.uint64).astype(np.uint32)
    e = np.clip(rng.integers(0, 255, (4096, 1)) - rng.integers(0, 24, (4096, 128)), 0, 254).astype(np.uint32)
    x = ((bits & 0x807FFFFF) | e << 23).view(np.float32)
    check_quantize(torch.from_numpy(x).to(dev), dev, "random bits")


def test_quantize_strided_rows_and_given_outputs(dev):
    rng = rng_of(4)
    for dtype in (torch.bfloat16, torch.float32):
        wide = torch.full((9, 512), float("nan"), dtype=dtype)
        wide[:, 64:64 + 176] = torch.from_numpy(rng.standard_normal((9, 176))).to(dtype)
        x = wide.to(dev)[:, 64:64 + 176]
        for rows in (1, 128):
            codes = torch.full((11, 176), 0xA5, dtype=torch.uint8, device=dev).view(F8)
            n = 9 if rows == 1 else 1
            scales = torch.full((n + 2, 2), 77.0, device=dev)
            nv.fp8_quantize(x, block_rows=rows, codes=codes[1:10], scales=scales[1:1 + n])
            rc, rs = ref.quantize(x.float().cpu().numpy(), rows)
            assert np.array_equal(raw(codes)[1:10].cpu().numpy(), rc) and np.array_equal(scales[1:1 + n].cpu().numpy(), rs)
            assert (raw(codes)[[0, 10]] == 0xA5).all() and (scales[[0, n + 1]] == 77).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_quantize_non_finite(dev, dtype, rows, bad):
    x = torch.from_numpy(rng_of(5).standard_normal((150, 272))).to(dtype)
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    nv.fp8_quantize(x.to(dev), block_rows=rows, faults=word)
    assert int(word) == 0
    x[140, 137] = bad
    c, s = nv.fp8_quantize(x.to(dev), block_rows=rows, faults=word)
    assert int(word) == nv.FAULT_NONFINITE
    check_quantize(x.to(dev), dev, "non-finite", rows)
    y = nv.fp8_dequantize(c, s, block_rows=rows)
    assert int(torch.isnan(y).sum()) == (128 if rows == 1 else 22 * 128) and torch.isnan(y[140, 128:256]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [1, 128])
def test_dequantize(dev, dtype, rows):
    """Every code at scales of every exponent; the product rounded to fp32, then to the type."""
    M, K = 300, 512
    codes = np.tile(np.arange(256, dtype=np.uint8), (M, 2))
    rng = rng_of(6)
    s = np.ldexp(rng.random((M if rows == 1 else 3, 4)) + 1, rng.integers(-149, 118, (M if rows == 1 else 3, 4))).astype(np.float32)
    s[0, 1] = np.inf
    y = nv.fp8_dequantize(up(codes, dev), up(s, dev), block_rows=rows, dtype=dtype)
    with np.errstate(over="ignore", invalid="ignore"):
        want = torch.from_numpy(ref.dequantize(codes, s, rows).astype(np.float32)).to(dtype)
    assert y.dtype == dtype
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(y.cpu()), nan)
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
    assert torch.equal(y.cpu().view(bits)[~nan], want.view(bits)[~nan])  # -0 included


@pytest.mark.parametrize("M,K", [(1, 16), (3, 160), (1, 14336), (261, 1056)])
def test_dequantize_shapes_and_pitch(dev, M, K):
    c, s = weight(rng_of(7, M, K), M, K)
    want = torch.from_numpy(ref.dequantize(c, s, 128).astype(np.float32))
    assert torch.equal(nv.fp8_dequantize(up(c, dev), up(s, dev), block_rows=128).cpu(), want.bfloat16())
    out = torch.full((M, K + 64), 9.0, device=dev)
    nv.fp8_dequantize(up(c, dev), up(s, dev), block_rows=128, out=out[:, 32:32 + K])
    assert torch.equal(out[:, 32:32 + K].cpu(), want)
    assert (out[:, :32] == 9).all() and (out[:, 32 + K:] == 9).all()


# -------------------------------------------------------------------------- linear

LINEAR = [(1, 2048, 2048), (1, 1, 16), (1, 17, 64), (2, 33, 112), (4, 4096, 512), (7, 250, 144), (15, 31, 1056), (16, 1000, 4096),
          (17, 48, 272), (31, 96, 2048), (33, 1, 128), (48, 513, 400), (64, 256, 1024), (65, 130, 256), (100, 257, 368), (128, 384, 768),
          (130, 100, 4112), (257, 300, 528), (300, 1000, 32), (513, 515, 1024), (16, 24, 14336), (3, 40, 36000), (1, 12288, 80), (700, 259, 2080)]


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(dev, M, N, K, kind):
    say("linear", kind, M, N, K)
    rng = rng_of(10, M, N, K)
    x, (c, s) = acts(rng, M, K), weight(rng, N, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    want, mag = ref.linear(xv, ref.dequantize(c, s, 128))
    cd, sd = up(c, dev), up(s, dev)
    y = nv.fp8_linear(xd, cd, sd, x_scales=xs)
    assert y.dtype == torch.float32
    assert_near(y, want, ref.tolerance(want, mag, K), (kind, M, N, K))
    yb = nv.fp8_linear(xd, cd, sd, x_scales=xs, out_dtype=torch.bfloat16)
    check_bf16(yb, y, want, ref.tolerance(want, mag, K), kind, xv, ref.dequantize(c, s, 128))
    assert torch.equal(nv.fp8_linear(xd, cd, sd, x_scales=xs), y)  # the same on every run
    assert torch.equal(nv.fp8_linear(xd, cd, sd, x_scales=xs, out_dtype=torch.bfloat16), yb)


def check_bf16(yb, y, want, tol, kind, xv, w):
    """A BF16 result: the fp32 one rounded, or W8A8's own sums (ref.dropped), rounded."""
    if kind == "bf16":
        assert torch.equal(yb, y.bfloat16())
        return
    tol = tol + ref.dropped(xv, w)
    assert_near(yb, want, tol + 2.0 ** -8 * (np.abs(want) + tol), "BF16")


# enough rows and columns for every tile, ragged in both
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("K", [16, 128, 240, 384, 640, 1600])
@pytest.mark.parametrize("M,N", [(330, 4001), (1000, 3300), (1500, 4404), (2500, 5400)])
def test_linear_tiles(dev, M, N, K, kind):
    say("linear tiles", kind, M, N, K)
    rng = rng_of(11, M, N, K)
    x, (c, s) = acts(rng, M, K), weight(rng, N, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    keep = np.unique(np.concatenate([np.arange(0, M, 37), [M - 1, M - 2]]))  # rows for the reference
    want, mag = ref.linear(xv[keep], ref.dequantize(c, s, 128))
    cd, sd = up(c, dev), up(s, dev)
    y = nv.fp8_linear(xd, cd, sd, x_scales=xs)
    assert_near(y[torch.from_numpy(keep).to(dev)], want, ref.tolerance(want, mag, K), (kind, M, N, K))
    # every row against the same rows in calls of 16, which stream the weight: both are within
    # the tolerance of the true value; the magnitudes from the values without their signs
    parts = torch.cat([nv.fp8_linear(xd[i:i + 16], cd, sd, x_scales=None if xs is None else xs[i:i + 16]) for i in range(0, M, 16)])
    plus = lambda t: (raw(t) & 0x7F).view(F8)  # noqa: E731
    mags = num(nv.fp8_linear(xd.abs() if xs is None else plus(xd), plus(cd), sd, x_scales=xs)) * 1.01
    assert_near(y, num(parts), 2 * ref.tolerance(num(parts), mags, K), "rows")
    yb = nv.fp8_linear(xd, cd, sd, x_scales=xs, out_dtype=torch.bfloat16)
    some = keep[::4]
    check_bf16(yb if kind == "bf16" else yb[torch.from_numpy(some).to(dev)], y, want[::4], ref.tolerance(want, mag, K)[::4], kind, xv[some],
               ref.dequantize(c, s, 128))
    if kind == "fp8":  # every row: eights' largest products are at most all of their magnitudes
        t = ref.tolerance(num(y), mags, K) + 7 * 2.0 ** -13 * mags
        assert_near(yb, num(y), t + 2.0 ** -8 * (np.abs(num(y)) + t), "BF16 rows")
    wide = torch.full((M, N + 3), 5.0, device=dev)
    nv.fp8_linear(xd, cd, sd, x_scales=xs, out=wide[:, 1:1 + N])
    assert torch.equal(wide[:, 1:1 + N], y)
    assert (wide[:, 0] == 5).all() and (wide[:, N + 1:] == 5).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("M,N,K", [(700, 2100, 8336), (400, 3400, 16400)])
def test_linear_tiles_long_rows(dev, M, N, K, kind):
    """More blocks along K than a wave has lanes."""
    say("linear tiles, long rows", kind, M, N, K)
    rng = rng_of(16, M, N, K)
    x, (c, s) = acts(rng, M, K), weight(rng, N, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    w = ref.dequantize(c, s, 128)
    keep = np.arange(0, M, 61)
    want, mag = ref.linear(xv[keep], w)
    at = torch.from_numpy(keep).to(dev)
    y = nv.fp8_linear(xd, up(c, dev), up(s, dev), x_scales=xs)
    assert_near(y[at], want, ref.tolerance(want, mag, K), (kind, M, N, K))
    yb = nv.fp8_linear(xd, up(c, dev), up(s, dev), x_scales=xs, out_dtype=torch.bfloat16)
    check_bf16(yb if kind == "bf16" else yb[at], y, want, ref.tolerance(want, mag, K), kind, xv[keep], w)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_linear_offsets_past_32_bits(dev, kind):
    """A weight, and activations, of more than 2^31 bytes: 512 and 509 rows over and over."""
    K, P, W = 8192, 509, 512
    rng = rng_of(12)
    c, s = weight(rng, W, K)
    x = acts(rng, P, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    want, mag = ref.linear(xv, ref.dequantize(c, s, 128))
    tol = ref.tolerance(want, mag, K)
    cd, sd = up(c, dev), up(s, dev)
    N = 2 ** 18 + 77
    wc = raw(cd).repeat(N // W + 1, 1)[:N].view(F8)
    ws = sd.repeat(N // W + 1, 1)[:ref.blocks(N)].contiguous()
    cols = np.r_[0:300, N // 2:N // 2 + 300, N - 300:N]
    for M in (1, 3, 33, 130):
        say("weight past 2^31 bytes", kind, M)
        y = nv.fp8_linear(xd[:M], wc, ws, x_scales=None if xs is None else xs[:M])
        assert_near(y[:, cols], want[:M, cols % W], tol[:M, cols % W], ("weight", M))
    del wc, ws, y
    M = 2 ** 17 + 77 if kind == "bf16" else 2 ** 18 + 77
    which = torch.arange(M, device=dev) % P
    big, bs = raw(xd)[which].view(xd.dtype), None if xs is None else xs[which]
    rows = np.r_[0:300, M // 2:M // 2 + 300, M - 300:M]
    for N in (1, 70):
        say("activations past 2^31 bytes", kind, N)
        y = nv.fp8_linear(big, cd[:N], sd[:1], x_scales=bs)
        assert_near(y[rows], want[rows % P][:, :N], tol[rows % P][:, :N], ("activations", N))
    if kind == "bf16":
        for block in (1, 128):
            qc, qs = nv.fp8_quantize(big, block_rows=block)
            if block == 1:
                rc, rs = (up(a, dev) for a in ref.quantize(x.float().numpy()))
                assert torch.equal(raw(qc)[rows], raw(rc)[rows % P]) and torch.equal(qs[rows], rs[rows % P])
            back = nv.fp8_dequantize(qc, qs, block_rows=block)
            assert np.abs(num(back[rows]) - num(big[rows])).max() <= 2.0 ** -4 * 1.01 * float(big.abs().max())


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_linear_pitched_views_and_what_lies_around(dev, M, kind):
    """x rows inside a wider buffer of NaNs, y columns inside a wider one, scales off 16 bytes."""
    N, K = 75, 368
    rng = rng_of(13, M)
    x, (c, s) = acts(rng, M, K), weight(rng, N, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    wide = torch.full((M + 1, 2 * K + 64), 0xFF, dtype=torch.uint8, device=dev).view(xd.dtype)
    view = wide[:M, 16:16 + K]
    raw(view).copy_(raw(xd)) if kind == "fp8" else view.copy_(xd)
    around = torch.full((s.size + 2,), float("nan"), device=dev)
    sd = around[1:-1].view(s.shape)
    sd.copy_(up(s, dev))
    if xs is not None:
        buf = torch.full((xs.numel() + 2,), float("nan"), device=dev)
        at = buf[1:-1].view(xs.shape)
        at.copy_(xs)
        xs = at
    want, mag = ref.linear(xv, ref.dequantize(c, s, 128))
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((M + 2, N + 9), 7.0, dtype=dtype, device=dev)
        nv.fp8_linear(view, up(c, dev), sd, x_scales=xs, out=out[1:M + 1, 3:3 + N])
        if dtype == torch.float32:
            assert_near(out[1:M + 1, 3:3 + N], want, ref.tolerance(want, mag, K), (kind, M))
            y = out[1:M + 1, 3:3 + N].clone()
        else:
            check_bf16(out[1:M + 1, 3:3 + N], y, want, ref.tolerance(want, mag, K), kind, xv, ref.dequantize(c, s, 128))
        rest = out.clone()
        rest[1:M + 1, 3:3 + N] = 7.0
        assert (rest == 7).all()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (9, 33)])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_linear_every_pair_of_codes(dev, kind, rows, cols, out):
    """Rows of one code each, subnormal ones among them: 144 equal products, whose sums of at most 128 are
    exact in 32 bits, as are these times powers of two, and of which no instruction drops anything."""
    K, n = 144, 254
    codes = np.concatenate([np.arange(127), np.arange(128, 255)]).astype(np.uint8)
    x, w = (np.tile(np.repeat(codes[:, None], K, 1), (many, 1)) for many in (rows, cols))
    xs, ws = np.full((rows * n, 2), 2.0 ** -3, np.float32), np.full((ref.blocks(cols * n), 2), 4.0, np.float32)
    want = torch.from_numpy(K * 0.5 * np.multiply.outer(ref.TABLE[codes], ref.TABLE[codes])).float().to(out).to(dev)
    if kind == "bf16":
        a, a_s = torch.from_numpy(ref.dequantize(x, xs)).to(torch.bfloat16).to(dev), None
    else:
        a, a_s = up(x, dev), up(xs, dev)
    y = nv.fp8_linear(a, up(w, dev), up(ws, dev), x_scales=a_s, out_dtype=out)
    assert torch.equal(y.view(rows, n, cols, n), want[None, :, None, :].expand(rows, n, cols, n))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("M", [1, 20, 150, 400])
def test_linear_scales_of_every_size(dev, M, kind):
    """Each block has a scale of its own, from tiny to huge along K and down N, powers of two or
    not; each block's share is found in the sum."""
    N, K = 520, 1040
    rng = rng_of(14, M)
    c, s = weight(rng, N, K)
    s = (s * 2.0 ** rng.integers(-40, 40, s.shape)).astype(np.float32)
    (xd, xs), xv = act_operand(acts(rng, M, K), kind, dev)
    if kind == "fp8":
        t = xs.cpu().numpy() * (2.0 ** rng.integers(-20, 20, tuple(xs.shape))).astype(np.float32)
        xv, xs = ref.dequantize(raw(xd).cpu().numpy(), t), up(t, dev)
    want, mag = ref.linear(xv, ref.dequantize(c, s, 128))
    y = nv.fp8_linear(xd, up(c, dev), up(s, dev), x_scales=xs)
    assert_near(y, want, ref.tolerance(want, mag, K), (kind, M))
    yb = nv.fp8_linear(xd, up(c, dev), up(s, dev), x_scales=xs, out_dtype=torch.bfloat16)
    check_bf16(yb, y, want, ref.tolerance(want, mag, K), kind, xv, ref.dequantize(c, s, 128))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [1, 20, 150, 400])
def test_linear_nan_and_check_mode(dev, M, out, kind):
    N, K = 300, 400
    rng = rng_of(15, M)
    x, (c, s) = acts(rng, M, K), weight(rng, N, K)
    (xd, xs), _ = act_operand(x, kind, dev)
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    cd, sd = up(c, dev), up(s, dev)
    clean = nv.fp8_linear(xd, cd, sd, x_scales=xs, out_dtype=out, check=True, faults=word)
    assert int(word) == 0
    sd[2, 3] = float("nan")  # rows 256 and on
    y = nv.fp8_linear(xd, cd, sd, x_scales=xs, out_dtype=out, faults=word)
    assert int(word) == 0  # nothing is scanned without the flag
    assert torch.isnan(y[:, 256:]).all() and torch.equal(y[:, :256], clean[:, :256])
    nv.fp8_linear(xd, cd, sd, x_scales=xs, out_dtype=out, check=True, faults=word)
    assert int(word) == nv.FAULT_NAN_SCALE
    word.zero_()
    cd, sd = up(c, dev), up(s, dev)
    raw(cd)[77, 399] = 0xFF
    y = nv.fp8_linear(xd, cd, sd, x_scales=xs, out_dtype=out, check=True, faults=word)
    assert int(word) == nv.FAULT_NONFINITE
    keep = [n for n in range(N) if n != 77]
    assert torch.isnan(y[:, 77]).all() and torch.equal(y[:, keep], clean[:, keep])
    word.zero_()
    cd = up(c, dev)
    if kind == "bf16":
        xd[M - 1, 100] = float("inf")
    else:
        raw(xd)[M - 1, 100] = 0x7F
    y = nv.fp8_linear(xd, cd, sd, x_scales=xs, out_dtype=out, check=True, faults=word)
    assert int(word) == nv.FAULT_NONFINITE
    assert not torch.isfinite(y[M - 1]).any() and torch.equal(y[:M - 1], clean[:M - 1])
    if kind == "fp8":
        word.zero_()
        raw(xd)[M - 1, 100] = 0
        xs[M - 1, 1] = float("inf")
        nv.fp8_linear(xd, cd, sd, x_scales=xs, out_dtype=out, check=True, faults=word)
        assert int(word) == nv.FAULT_NAN_SCALE


# ------------------------------------------------------------------------- grouped

def routes(rng, T, E, k, skew=1.0):
    ids = np.argsort(-(skew * rng.standard_normal(E) + rng.gumbel(size=(T, E))), axis=1)[:, :k].astype(np.int32)
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
        kept[r] = 0 <= ids[t, j] < w.shape[0] and ids[t, j] not in ids[t, :j]
    for e in range(w.shape[0]):
        mine = np.flatnonzero(kept & (ids.reshape(-1) == e))
        y[mine], mag[mine] = ref.linear(xv[mine if per_route else mine // k], w[e])
    return y, mag, kept


def check_forms(args, xs, y, mag, tw, T, k, N, K, dev, lost):
    """Every output form of a grouped call against the float64 rows; lost: what W8A8's sums of
    results that are not fp32 may be off more (0 for BF16 activations)."""
    tol = ref.tolerance(y, mag, K)
    tol_b = tol + lost
    rows = nv.fp8_grouped_linear(*args, x_scales=xs)
    assert rows.dtype == torch.float32
    assert_near(rows, y, tol, "routes")
    rows_b = nv.fp8_grouped_linear(*args, x_scales=xs, out_dtype=torch.bfloat16)
    assert_near(rows_b, y, tol_b + 2.0 ** -8 * (np.abs(y) + tol_b), "routes in BF16")
    if N % 256 == 0:
        want, t = swiglu(y, tol)
        a = nv.fp8_grouped_linear(*args, x_scales=xs, out_mode=nv.OUT_SWIGLU_BF16)
        assert a.dtype == torch.bfloat16
        assert_near(a, want, t + 2.0 ** -8 * (np.abs(want) + t) + 1e-37, "swiglu")
        qc, qs = nv.fp8_grouped_linear(*args, x_scales=xs, out_mode=nv.OUT_SWIGLU_FP8)
        rc, rs = nv.fp8_quantize(a)  # bit for bit the quantizer's view of the BF16 rows
        assert torch.equal(qs, rs) and torch.equal(raw(qc), raw(rc))
    want = (y.reshape(T, k, N) * tw[..., None].astype(np.float64)).sum(1)
    absw = (np.abs(y).reshape(T, k, N) * tw[..., None]).sum(1)
    of = lambda t: (t.reshape(T, k, N) * tw[..., None]).sum(1) + (k + 1) * 2.0 ** -24 * absw + 1e-37  # noqa: E731
    out = nv.fp8_grouped_linear(*args, x_scales=xs, topk_w=up(tw, dev), out_mode=nv.OUT_COMBINE)
    assert_near(out, want, of(tol), "combine")
    out = nv.fp8_grouped_linear(*args, x_scales=xs, topk_w=up(tw, dev), out_mode=nv.OUT_COMBINE, out_dtype=torch.bfloat16)
    assert_near(out, want, of(tol_b) + 2.0 ** -8 * (np.abs(want) + of(tol_b)), "combine in BF16")


def swiglu(y, tol):
    """(silu(gate) * up, its tolerance before rounding) from rows y [R][2 * half]. |silu'| < 1.1;
    the hardware's exponential and reciprocal: a few fp32 steps (2^-20)."""
    half = y.shape[1] // 2
    g, u = y[:, :half], y[:, half:]
    silu = g / (1 + np.exp(-g))
    t = 1.1 * tol[:, :half] * np.abs(u) + (np.abs(silu) + 1.1 * tol[:, :half]) * tol[:, half:]
    return silu * u, t + 2.0 ** -20 * np.abs(silu * u)


def lost_of(kind, xv, w, ids, per_route=False):
    """ref.dropped of each route's row."""
    T, k = ids.shape
    t = np.zeros((T * k, w.shape[1]))
    if kind == "bf16":
        return t
    flat = ids.reshape(-1)
    for e in range(w.shape[0]):
        mine = np.flatnonzero(flat == e)
        if mine.size:
            t[mine] = ref.dropped(xv[mine if per_route else mine // k], w[e])
    return t


GROUPED = [(1, 4, 1, 64, 32), (1, 128, 8, 256, 2048), (16, 128, 8, 256, 272), (5, 3, 3, 130, 112), (40, 6, 2, 64, 1056),
           (333, 24, 3, 66, 160), (200, 2, 1, 256, 512), (64, 300, 4, 256, 64), (700, 8, 2, 320, 288), (1500, 5, 2, 130, 128),
           (100, 128, 4, 128, 160), (300, 64, 2, 66, 528), (256, 40, 1, 512, 64), (257, 40, 1, 64, 80), (90, 200, 64, 64, 32), (4, 70, 64, 256, 64),
           (900, 6, 3, 768, 400), (260, 2, 2, 256, 8336)]


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("T,E,k,N,K", GROUPED)
def test_grouped_every_form(dev, T, E, k, N, K, kind):
    say("grouped", kind, T, E, k, N, K)
    rng = rng_of(20, T, E, k, N, K)
    ids, tw = routes(rng, T, E, k)
    x, (c, s) = acts(rng, T, K), weight(rng, E, N, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    w = ref.dequantize(c, s, 128)
    y, mag, _ = route_rows(xv, w, ids, False)
    check_forms((xd, up(c, dev), up(s, dev), up(ids, dev)), xs, y, mag, tw, T, k, N, K, dev, lost_of(kind, xv, w, ids))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("T,E,k,N,K", [(4200, 8, 2, 1088, 416), (1800, 3, 2, 768, 784), (2100, 40, 2, 512, 288)])
def test_grouped_prompts(dev, T, E, k, N, K, kind):
    """Prompt-sized groups, a token without experts among them."""
    say("grouped prompts", kind, T, E, k, N, K)
    rng = rng_of(21, T, E)
    ids, tw = routes(rng, T, E, k)
    ids[5] = -1
    x, (c, s) = acts(rng, T, K), weight(rng, E, N, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    w = ref.dequantize(c, s, 128)
    y, mag, _ = route_rows(xv, w, ids, False)
    check_forms((xd, up(c, dev), up(s, dev), up(ids, dev)), xs, y, mag, tw, T, k, N, K, dev, lost_of(kind, xv, w, ids))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("popular", [False, True])
@pytest.mark.parametrize("T,E,k,N,K", [(20, 40, 5, 256, 1296), (28, 40, 5, 130, 640), (42, 40, 5, 256, 784), (47, 40, 5, 64, 2064),
                                       (110, 200, 5, 256, 1296), (160, 200, 5, 128, 656), (235, 200, 5, 256, 400), (240, 200, 5, 128, 400)])
def test_grouped_a_few_routes_an_expert(dev, T, E, k, N, K, popular, kind):
    """Two to six routes an expert, or one with many: more of them than a workgroup takes at once."""
    say("grouped few routes", kind, T, E, k, N, K, popular)
    rng = rng_of(26, T, E, k, N, K, popular)
    ids, tw = routes(rng, T, E, k)
    if popular:
        at = np.flatnonzero((ids != 7).all(axis=1))[: T // 2]
        ids[at, 1] = 7
    x, (c, s) = acts(rng, T, K), weight(rng, E, N, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    w = ref.dequantize(c, s, 128)
    y, mag, _ = route_rows(xv, w, ids, False)
    check_forms((xd, up(c, dev), up(s, dev), up(ids, dev)), xs, y, mag, tw, T, k, N, K, dev, lost_of(kind, xv, w, ids))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("T,E,k", [(9, 7, 3), (120, 40, 5), (300, 7, 3), (2500, 4, 2)])
def test_grouped_bad_routes(dev, T, E, k, kind):
    """Ids out of range and repeated: flagged, their rows zero, the others as without them."""
    N, K = 256, 112
    rng = rng_of(22, T)
    ids, tw = routes(rng, T, E, k)
    ids[0, 0], ids[T // 2, 1], ids[T - 1, k - 1] = -1, E, 2 ** 31 - 1
    ids[1, 1] = ids[1, 0]
    ids[T // 3] = -5  # a token without any route
    x, (c, s) = acts(rng, T, K), weight(rng, E, N, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    y, mag, kept = route_rows(xv, ref.dequantize(c, s, 128), ids, False)
    args = (xd, up(c, dev), up(s, dev), up(ids, dev))
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    out = torch.full((T * k, N), float("nan"), device=dev)
    nv.fp8_grouped_linear(*args, x_scales=xs, out=out, faults=word)
    assert int(word) == nv.FAULT_BAD_ROUTE
    assert (out.cpu().numpy()[~kept] == 0).all()
    qc = torch.full((T * k, N // 2), 0xA5, dtype=torch.uint8, device=dev).view(F8)
    qs = torch.full((T * k, N // 256), 77.0, device=dev)
    nv.fp8_grouped_linear(*args, x_scales=xs, out_mode=nv.OUT_SWIGLU_FP8, out=qc, out_scales=qs)
    assert not raw(qc).cpu().numpy()[~kept].any() and not qs.cpu().numpy()[~kept].any()
    comb = nv.fp8_grouped_linear(*args, x_scales=xs, topk_w=up(tw, dev), out_mode=nv.OUT_COMBINE)
    assert (comb[T // 3] == 0).all()
    check_forms(args, xs, y, mag, tw, T, k, N, K, dev, lost_of(kind, xv, ref.dequantize(c, s, 128), ids))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("T,E,k", [(24, 40, 5), (300, 40, 3), (400, 7, 4), (2500, 4, 2)])
@pytest.mark.parametrize("real", [0, 1, 0.4])
def test_grouped_padded_batch(dev, T, E, k, kind, real):
    """A batch whose last tokens have no expert: zeros there in every form, whatever lay there."""
    K, n = 96, int(T * real) if real < 1 else 1
    rng = rng_of(23, T)
    ids, tw = routes(rng, T, E, k)
    ids[n:] = -1
    x = acts(rng, T, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    ids_d, tw_d = up(ids, dev), up(tw, dev)
    for N, mode, dtype in ((193, nv.OUT_ROUTES, torch.bfloat16), (193, nv.OUT_ROUTES, torch.float32),
                           (256, nv.OUT_SWIGLU_BF16, torch.bfloat16), (512, nv.OUT_SWIGLU_FP8, F8), (193, nv.OUT_COMBINE, torch.float32)):
        c, s = weight(rng, E, N, K)
        per = 1 if mode == nv.OUT_COMBINE else k
        cols = N // 2 if mode in (nv.OUT_SWIGLU_BF16, nv.OUT_SWIGLU_FP8) else N
        out = torch.full((T * per, cols), 77, dtype=torch.float32, device=dev).to(dtype)
        osc = torch.full((T * k, N // 256), 77.0, device=dev) if mode == nv.OUT_SWIGLU_FP8 else None
        word = torch.zeros(1, dtype=torch.int32, device=dev)
        nv.fp8_grouped_linear(xd, up(c, dev), up(s, dev), ids_d, topk_w=tw_d, x_scales=xs, out_mode=mode, out=out, out_scales=osc, faults=word)
        assert int(word) == nv.FAULT_BAD_ROUTE
        bits = raw(out) if dtype == F8 else out
        assert not bits[n * per:].any() and (osc is None or not osc[n * k:].any())
        if mode == nv.OUT_ROUTES and dtype == torch.float32 and n:
            y, mag, _ = route_rows(xv[:n], ref.dequantize(c, s, 128), ids[:n], False)
            assert_near(out[:n * k], y, ref.tolerance(y, mag, K), "kept rows")
        elif n:
            assert bits[:n * per].any()


def test_grouped_all_on_one_expert_and_one_row_each(dev):
    N, K, E = 96, 128, 40
    rng = rng_of(24)
    c, s = weight(rng, E, N, K)
    w = ref.dequantize(c, s, 128)
    for kind in ("bf16", "fp8"):
        for ids in (np.full((200, 1), 39, np.int32), np.full((259, 1), 17, np.int32), np.full((2000, 1), 0, np.int32),
                    np.arange(E, dtype=np.int32)[:, None]):
            (xd, xs), xv = act_operand(acts(rng, ids.shape[0], K), kind, dev)
            y, mag, _ = route_rows(xv, w, ids, False)
            got = nv.fp8_grouped_linear(xd, up(c, dev), up(s, dev), up(ids, dev), x_scales=xs)
            assert_near(got, y, ref.tolerance(y, mag, K), ids.shape)


def test_grouped_swiglu_to_fp8_non_finite(dev):
    """A token with an infinite activation: its blocks' scales are NaN and their codes 0."""
    T, E, k, N, K = 600, 4, 2, 512, 128
    rng = rng_of(25)
    ids, _ = routes(rng, T, E, k)
    c, s = weight(rng, E, N, K)
    for kind in ("bf16", "fp8"):
        for n in (3, T):
            (xd, xs), _ = act_operand(acts(rng, n, K), kind, dev)
            if kind == "bf16":
                xd[2, 7] = float("inf")
            else:
                xs[2, 0] = float("inf")
            args = (xd, up(c, dev), up(s, dev), up(ids[:n], dev))
            qc, qs = nv.fp8_grouped_linear(*args, x_scales=xs, out_mode=nv.OUT_SWIGLU_FP8)
            assert torch.isnan(qs[4:6]).all() and not raw(qc)[4:6].any() and torch.isfinite(qs[:4]).all() and torch.isfinite(qs[6:]).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("T", [1, 16, 100, 1200])
def test_moe_layer(dev, T, kind):
    """A layer as it is used: route, quantize, gate_up with SwiGLU, down with the combine reusing
    the grouping, one workspace; each step against float64 on its own inputs."""
    E, k, H, I = 16, 4, 272, 256
    rng = rng_of(26, T)
    gu, dn = weight(rng, E, 2 * I, H), weight(rng, E, H, I)
    x = acts(rng, T, H).to(dev)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    idd, twd = nv.moe_route(up(logits, dev), k)
    ids, tw = ref.route(logits, k)
    assert np.array_equal(idd.cpu().numpy(), ids)
    assert np.all(np.abs(num(twd) - tw) <= 2.0 ** -23 * tw)
    tw = twd.cpu().numpy()
    mid = nv.OUT_SWIGLU_BF16 if kind == "bf16" else nv.OUT_SWIGLU_FP8
    size = max(nv.fp8_grouped_workspace_size(T, k, 2 * I, H, E, mid), nv.fp8_grouped_workspace_size(T, k, H, I, E, nv.OUT_COMBINE))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=dev)
    if kind == "bf16":
        xv = num(x)
        a, a_s = nv.fp8_grouped_linear(x, up(gu[0], dev), up(gu[1], dev), idd, out_mode=mid, workspace=ws), None
        av = num(a)
    else:
        xc, xs = nv.fp8_quantize(x)
        xv = ref.dequantize(raw(xc).cpu().numpy(), xs.cpu().numpy())
        a, a_s = nv.fp8_grouped_linear(xc, up(gu[0], dev), up(gu[1], dev), idd, x_scales=xs, out_mode=mid, workspace=ws)
        av = ref.dequantize(raw(a).cpu().numpy(), a_s.cpu().numpy())
    y, mag, _ = route_rows(xv, ref.dequantize(*gu, 128), ids, False)
    want, t = swiglu(y, ref.tolerance(y, mag, H))
    t = t + 2.0 ** -8 * (np.abs(want) + t)
    if kind == "fp8":  # half a step of E4M3: 2^-4 of the value or 2^-10 of the scale
        top = np.repeat((np.abs(want) + t).reshape(T * k, I // 128, 128).max(-1), 128, 1)
        t = t + 2.0 ** -4 * (np.abs(want) + t) + 1.01 * 2.0 ** -10 * top / 448
    assert_near(av, want, t, "gate_up")
    out = nv.fp8_grouped_linear(a, up(dn[0], dev), up(dn[1], dev), idd, x_scales=a_s, topk_w=twd, out_mode=nv.OUT_COMBINE,
                                rows_per_route=True, workspace=ws, reuse_grouping=True)
    again = nv.fp8_grouped_linear(a, up(dn[0], dev), up(dn[1], dev), idd, x_scales=a_s, topk_w=twd, out_mode=nv.OUT_COMBINE,
                                  rows_per_route=True)
    assert torch.equal(out, again)
    y, mag, _ = route_rows(av, ref.dequantize(*dn, 128), ids, True)
    want = (y.reshape(T, k, H) * tw[..., None].astype(np.float64)).sum(1)
    t = ((ref.tolerance(y, mag, I) + (k + 1) * 2.0 ** -24 * np.abs(y)).reshape(T, k, H) * tw[..., None]).sum(1) + 1e-37
    assert_near(out, want, t, "down")


def test_routes_feed_every_format(dev):
    """moe_route's ids and weights, a padded row's among them, in the grouped calls of all three
    formats: the padded row comes out as zeros, the others as of the same weights."""
    T, E, k, N, K = 37, 12, 3, 128, 256
    rng = rng_of(27)
    logits = torch.from_numpy(rng.standard_normal((T, E))).float().to(dev)
    logits[11] = float("-inf")
    ids, tw = nv.moe_route(logits, k, scoring="sigmoid", groups=3, top_groups=2)
    x = acts(rng, T, K).to(dev)
    w = torch.from_numpy(0.02 * rng.standard_normal((E, N, K))).float().to(dev)
    f8 = [nv.fp8_quantize(one, block_rows=128) for one in w]
    mx = [nv.mxfp4_quantize(one) for one in w]
    n4 = [nv.quantize_act(one, per_tensor=True) for one in w]
    stack = lambda parts: [torch.stack([raw(p[i]) if p[i].dtype == F8 else p[i] for p in parts]) for i in range(len(parts[0]))]  # noqa: E731
    f8, mx, n4 = stack(f8), stack(mx), stack(n4)
    f8[0] = f8[0].view(F8)
    outs = [nv.fp8_grouped_linear(x, *f8, ids, topk_w=tw, out_mode=nv.OUT_COMBINE), nv.mxfp4_grouped_linear(x, *mx, ids, topk_w=tw, out_mode=nv.OUT_COMBINE),
            nv.grouped_linear(x, n4[0], n4[1], n4[2].reshape(E), ids, topk_w=tw, out_mode=nv.OUT_COMBINE)]
    xv, idn, twn = num(x), ids.cpu().numpy(), num(tw)
    want = np.stack([sum(twn[t, j] * (num(w[idn[t, j]]) @ xv[t]) for j in range(k) if idn[t, j] >= 0) + np.zeros(N) for t in range(T)])
    for y, rel in zip(outs, (0.05, 0.2, 0.2)):  # 3 and 1 mantissa bits: about 0.025 and 0.1 of the whole
        assert not y[11].any()
        assert np.linalg.norm(num(y) - want) < rel * np.linalg.norm(want)


# ------------------------------------------------- streams, graphs, calls side by side

def layer_calls(dev, T, seed):
    """A closure that runs a router, quantize, linear and a W8A8 layer into given buffers."""
    E, k, H, I = 8, 2, 144, 128
    rng = rng_of(28, T, seed)
    x = acts(rng, T, H).to(dev)
    logits, bias = (torch.from_numpy(rng.standard_normal(n)).float().to(dev) for n in ((T, E), (E,)))
    lin, gu, dn = ([up(t, dev) for t in weight(rng, *shape)] for shape in ((90, H), (E, 2 * I, H), (E, H, I)))
    size = max(nv.fp8_grouped_workspace_size(T, k, 2 * I, H, E, nv.OUT_SWIGLU_FP8), nv.fp8_grouped_workspace_size(T, k, H, I, E, nv.OUT_COMBINE))
    new = lambda shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
    ws = new((size,), torch.uint8)
    ids, tw = new((T, k), torch.int32), new((T, k))
    xc, xs, a, a_s = new((T, H), F8), new((T, 2)), new((T * k, I), F8), new((T * k, 1))
    y, y16, out, back = new((T, 90)), new((T, 90)), new((T, H)), new((T, H))

    def run():
        nv.moe_route(logits, k, scoring="sigmoid", bias=bias, groups=2, top_groups=1, group_score="top2", topk_ids=ids, topk_w=tw)
        nv.fp8_quantize(x, codes=xc, scales=xs)
        nv.fp8_dequantize(xc, xs, out=back)
        nv.fp8_linear(xc, *lin, x_scales=xs, out=y)
        nv.fp8_linear(x, *lin, out=y16)
        nv.fp8_grouped_linear(xc, *gu, ids, x_scales=xs, out_mode=nv.OUT_SWIGLU_FP8, out=a, out_scales=a_s, workspace=ws)
        nv.fp8_grouped_linear(a, *dn, ids, x_scales=a_s, topk_w=tw, out_mode=nv.OUT_COMBINE, rows_per_route=True, out=out, workspace=ws, reuse_grouping=True)

    return run, [ids, tw, xc, xs, back, y, y16, a, a_s, out]


@pytest.mark.parametrize("T", [1, 12, 70, 600, 2500])
def test_graph_replays(dev, T):
    run, outs = layer_calls(dev, T, 0)
    other, _ = layer_calls(dev, T + 3, 1)
    run()
    torch.cuda.synchronize()
    want = [raw(o).clone() for o in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for i in range(4):
        for o in outs:
            raw(o).fill_(0xA5)
        other()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(raw(o), w), f"replay {i}"


def test_two_streams_at_once(dev):
    """Two layers with workspaces of their own on two streams, several times, give what each
    gives alone."""
    pairs = [layer_calls(dev, 200, 2), layer_calls(dev, 310, 3)]
    for run, _ in pairs:
        run()
    torch.cuda.synchronize()
    want = [[raw(o).clone() for o in outs] for _, outs in pairs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _, outs in pairs:
        for o in outs:
            raw(o).fill_(0xA5)
    torch.cuda.synchronize()
    for _ in range(5):
        for (run, _), st in zip(pairs, streams):
            with torch.cuda.stream(st):
                run()
    torch.cuda.synchronize()
    for (_, outs), ws in zip(pairs, want):
        for o, w in zip(outs, ws):
            assert torch.equal(raw(o), w)


# a grouping that is reused: whatever the workspace holds, the product stays inside its buffers
# (tokens, experts, top_k): by slots with and without list tiles, tiles of 64 and of 128
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("T,E,k", [(16, 64, 17), (100, 64, 4), (700, 512, 8), (300, 40, 4), (1100, 16, 4)])
def test_any_workspace_stays_in_bounds(dev, T, E, k, kind):
    N, K, guard = 64, 96, 1 << 20
    rng = rng_of(30, T, E, k)
    ids, tw = routes(rng, T, E, k)
    (xd, xs), _ = act_operand(acts(rng, T, K), kind, dev)
    wd, idd, twd = [up(a, dev) for a in weight(rng, E, N, K)], up(ids, dev), up(tw, dev)
    size = nv.fp8_grouped_workspace_size(T, k, N, K, E, nv.OUT_COMBINE)
    arena = torch.full((guard + size + guard,), 0xA5, dtype=torch.uint8, device=dev)
    ws = arena[guard:guard + size]
    board = torch.full((T + 8192, N), 7.0, device=dev)
    out = board[4096:4096 + T]

    def combine(**kw):
        return nv.fp8_grouped_linear(xd, *wd, idd, topk_w=twd, x_scales=xs, out_mode=nv.OUT_COMBINE, out=out, workspace=ws, **kw)

    want = combine().clone()
    ints = lambda low, high: torch.from_numpy(rng.integers(low, high, size // 4, dtype=np.int64).astype(np.int32)).to(dev).view(torch.uint8)  # noqa: E731
    fills = {
        "zeros": lambda: ws.zero_(), "ones": lambda: ws.fill_(0xFF), "large": lambda: ws.fill_(0x7F),
        "least": lambda: ws.copy_(torch.full((size // 4,), -2 ** 31, dtype=torch.int32, device=dev).view(torch.uint8)),
        "any": lambda: ws.copy_(ints(-2 ** 31, 2 ** 31)), "near": lambda: ws.copy_(ints(-3, T * k + 3)), "experts": lambda: ws.copy_(ints(0, E)),
    }
    for name, fill in fills.items():
        say("reused workspace", kind, T, E, k, name)
        fill()
        combine(reuse_grouping=True)
        torch.cuda.synchronize()
        assert (arena[:guard] == 0xA5).all() and (arena[guard + size:] == 0xA5).all(), name
        assert (board[:4096] == 7).all() and (board[4096 + T:] == 7).all(), name
        assert torch.equal(combine(), want), name


# ------------------------------------------------------------------------ refusals

def test_binding_refusals(dev):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=dev)
    c, s = torch.zeros((256, 64), dtype=F8, device=dev), torch.zeros((2, 1), device=dev)
    xs = torch.zeros((4, 1), device=dev)
    x8 = c[:4]
    ids = torch.zeros((4, 1), dtype=torch.int32, device=dev)
    for call in (
        lambda: nv.fp8_quantize(x.half()), lambda: nv.fp8_quantize(x.t()), lambda: nv.fp8_quantize(x[0]), lambda: nv.fp8_quantize(x, block_rows=64),
        lambda: nv.fp8_quantize(x, codes=c), lambda: nv.fp8_quantize(x, scales=s), lambda: nv.fp8_quantize(x, faults=torch.zeros(1, device=dev)),
        lambda: nv.fp8_dequantize(c, s), lambda: nv.fp8_dequantize(c, s, block_rows=2), lambda: nv.fp8_dequantize(raw(c), s, block_rows=128),
        lambda: nv.fp8_dequantize(c[:, ::2], s, block_rows=128), lambda: nv.fp8_dequantize(c, s, block_rows=128, dtype=torch.half),
        lambda: nv.fp8_dequantize(c[0], s, block_rows=128),
        lambda: nv.fp8_linear(x[:, :32], c, s), lambda: nv.fp8_linear(x.float(), c, s), lambda: nv.fp8_linear(x, raw(c), s), lambda: nv.fp8_linear(x, c, s.double()),
        lambda: nv.fp8_linear(x, c, s[:1]), lambda: nv.fp8_linear(x, c, s, x_scales=xs), lambda: nv.fp8_linear(x8, c, s), lambda: nv.fp8_linear(x8, c, s, x_scales=s),
        lambda: nv.fp8_linear(x, c, s, out_dtype=torch.half), lambda: nv.fp8_linear(x, c, s, out=torch.empty((4, 7), device=dev)),
        lambda: nv.fp8_linear(x, c[:, :16], s), lambda: nv.fp8_linear(x.cpu(), c, s), lambda: nv.fp8_linear(x8.t(), c, s, x_scales=xs),
        lambda: nv.fp8_grouped_linear(x, c[None], s[None], ids.long()), lambda: nv.fp8_grouped_linear(x[:3], c[None], s[None], ids),
        lambda: nv.fp8_grouped_linear(x, c, s, ids), lambda: nv.fp8_grouped_linear(x, c[None], s[None], ids, out_mode=3),
        lambda: nv.fp8_grouped_linear(x, c[None], s[None], ids, reuse_grouping=True), lambda: nv.fp8_grouped_linear(x, c[None], s[None], ids, out_scales=xs),
        lambda: nv.fp8_grouped_linear(x, c[None], s[None], ids, out_mode=nv.OUT_SWIGLU_FP8, out_dtype=torch.float32),
        lambda: nv.fp8_grouped_linear(x, c[None], s[None], ids, out=torch.empty((4, 9), device=dev)),
    ):
        with pytest.raises(ValueError):
            call()
    for call, name in (
        (lambda: nv.fp8_quantize(x[:, :40]), "SHAPE"), (lambda: nv.fp8_quantize(x[:0]), "SHAPE"), (lambda: nv.fp8_quantize(x[:, 4:36]), "ALIGN"),
        (lambda: nv.fp8_linear(x[:0], c, s), "SHAPE"), (lambda: nv.fp8_linear(x, c, s, check=True), "NULL"),
        (lambda: nv.fp8_linear(x[:, 8:24], c[:, 8:24].contiguous(), s), None),
        (lambda: nv.fp8_linear(c[:4, 8:24], c[:, 8:24].contiguous(), s, x_scales=xs), "ALIGN"),
        (lambda: nv.fp8_grouped_linear(x, c[None], s[None], ids, out_mode=nv.OUT_COMBINE), "NULL"),
        (lambda: nv.fp8_grouped_linear(x, c[None, :128].contiguous(), s[None, :1], ids, out_mode=nv.OUT_SWIGLU_BF16), "SHAPE"),
        (lambda: nv.fp8_grouped_linear(x, c[None], s[None], ids, out_mode=nv.OUT_SWIGLU_BF16, out_dtype=torch.float32), "ARG"),
        (lambda: nv.fp8_grouped_linear(x, c[None], s[None], ids, workspace=torch.empty(128, dtype=torch.uint8, device=dev)), "WORKSPACE"),
        (lambda: nv.fp8_grouped_linear(x, c[None], s[None], torch.zeros((4, 2), dtype=torch.int32, device=dev)), "ARG"),
    ):
        if name is None:
            call()
            continue
        with pytest.raises(nv.NVFP4Error, match=name):
            call()
