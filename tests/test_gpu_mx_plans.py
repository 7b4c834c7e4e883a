"""The MXFP4 grouped product in each way it goes about its routes, against float64 numpy: few
routes, found by the workgroups themselves (up to 256, fewer than 16 per active expert); slot
records (more routes, still fewer than 16 per active expert); tiles. And what a call may meet in
each: popular experts, padding, NaN scales, large expert stacks."""
import numpy as np
import pytest
import torch

import mx_reference as ref
import nvfp4_block_scaled_linear_amd as nv
from test_gpu_mx import act_operand, acts, assert_near, dev, num, rng_of, route_rows, routes, say, up, weight  # noqa: F401

pytestmark = pytest.mark.gpu


def popular(rng, T, E, k, most):
    """ids of T tokens: expert E - 1 is picked by `most` of them, E - 2 by half as many, E - 3 by
    a quarter, the rest at random."""
    ids = np.argsort(rng.random((T, E - 3)), 1)[:, :k].astype(np.int32)
    for i in range(min(3, k)):
        at = rng.permutation(T)[:max(1, most >> i)]
        ids[at, rng.integers(0, k, at.size)] = E - 1 - i
    for t in range(T):  # an expert once a token: a later repeat becomes one that is free
        free = [e for e in rng.permutation(E - 3) if e not in ids[t]]
        for j in range(k):
            if ids[t, j] in ids[t, :j]:
                ids[t, j] = free.pop()
    return np.ascontiguousarray(ids)


def weights_of(rng, T, k):
    w = rng.random((T, k)).astype(np.float32)
    return w / w.sum(1, keepdims=True)


def check_forms(dev, kind, ids, tw, E, N, K, rng, per_route=False):
    """Every output form over every row: kept rows against float64, dropped ones zero, whatever
    lay there. N is a multiple of 64."""
    T, k = ids.shape
    x, (c, s) = acts(rng, T * k if per_route else T, K), weight(rng, E, N, K)
    (xd, xs), xv = act_operand(x, kind, dev)
    y, mag, kept = route_rows(xv, ref.dequantize(c, s), ids, per_route)
    tol = ref.tolerance(y, mag, K)
    args, kw = (xd, up(c, dev), up(s, dev), up(ids, dev)), dict(x_scales=xs, rows_per_route=per_route)
    nan = dict(device=dev)

    def call(mode, out, **more):
        word = torch.zeros(1, dtype=torch.int32, device=dev)
        nv.mxfp4_grouped_linear(*args, out_mode=mode, out=out, faults=word, **kw, **more)
        assert int(word) == (0 if kept.all() else nv.FAULT_BAD_ROUTE)
        return out

    rows = call(nv.OUT_ROUTES, torch.full((T * k, N), float("nan"), **nan))
    assert_near(rows, y, tol, "routes")
    gone = torch.from_numpy(~kept).to(dev)
    assert not rows[gone].any()
    assert torch.equal(call(nv.OUT_ROUTES, torch.full((T * k, N), float("nan"), dtype=torch.bfloat16, **nan)), rows.bfloat16())
    want, t = ref.swiglu(y, tol, N // 2)
    a = call(nv.OUT_SWIGLU_BF16, torch.full((T * k, N // 2), float("nan"), dtype=torch.bfloat16, **nan))
    assert_near(a, want, t + 2.0 ** -8 * (np.abs(want) + t) + 1e-37, "swiglu")
    assert not a[gone].any()
    qs = torch.full((T * k, N // 64), 0xA5, dtype=torch.uint8, **nan)
    qc = call(nv.OUT_SWIGLU_MXFP4, torch.full((T * k, N // 4), 0xA5, dtype=torch.uint8, **nan), out_scales=qs)
    rc, rs = nv.mxfp4_quantize(a)
    assert torch.equal(qs, rs) and torch.equal(qc, rc)
    want = (y.reshape(T, k, N) * tw[..., None].astype(np.float64)).sum(1)
    t = ((tol + (k + 1) * 2.0 ** -24 * np.abs(y)).reshape(T, k, N) * tw[..., None]).sum(1) + 1e-37
    out = call(nv.OUT_COMBINE, torch.full((T, N), float("nan"), **nan), topk_w=up(tw, dev))
    assert_near(out, want, t, "combine")
    outb = call(nv.OUT_COMBINE, torch.full((T, N), float("nan"), dtype=torch.bfloat16, **nan), topk_w=up(tw, dev))
    assert torch.equal(outb, out.bfloat16())


# (tokens, experts, top_k, tokens of the most popular expert)
SCAN = [(16, 24, 4, 16), (32, 128, 8, 32), (60, 300, 4, 60), (128, 40, 2, 100), (256, 128, 1, 256), (85, 17, 3, 85), (64, 4096, 4, 64), (250, 17, 1, 240)]
SLOTS = [(40, 256, 8, 40), (33, 256, 8, 3), (64, 64, 8, 60), (700, 512, 8, 300), (300, 1200, 2, 200), (2000, 400, 3, 1900), (500, 512, 10, 17), (300, 512, 20, 60)]
TILES = [(300, 40, 4, 300), (1100, 17, 2, 900), (900, 24, 20, 500)]


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,E,k,most", SCAN + SLOTS + TILES)
def test_popular_experts(dev, T, E, k, most, kind):
    say("popular", kind, T, E, k, most)
    rng = rng_of(20, T, E, k)
    ids = popular(rng, T, E, k, most) if k > 1 else np.where(np.arange(T) < most, E - 1, rng.integers(0, E, T)).astype(np.int32)[:, None]
    check_forms(dev, kind, ids, weights_of(rng, T, k), E, 64, 96, rng)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,E,k,most", [(32, 128, 8, 30), (200, 100, 1, 200), (60, 300, 4, 60), (40, 256, 8, 40), (700, 512, 8, 300), (300, 40, 4, 300)])
def test_popular_experts_among_bad_routes(dev, T, E, k, most, kind):
    """Ids out of range, repeats, and tokens without an expert among routes of popular ones; one
    activation row per route."""
    say("popular, bad", kind, T, E, k, most)
    rng = rng_of(21, T, E, k)
    ids = popular(rng, T, E, k, most) if k > 1 else np.full((T, 1), E - 1, np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    ids[rng.random((T, k)) < 0.03] = E
    ids[T // 2] = E - 1  # the popular expert, over and over
    ids[T - 3:] = -7
    check_forms(dev, kind, ids, weights_of(rng, T, k), E, 64, 160, rng, per_route=True)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,E,k", [(24, 40, 5), (300, 40, 3), (600, 64, 1), (400, 7, 4), (2500, 4, 2)])
@pytest.mark.parametrize("real", [0, 1, 0.4])
def test_padded_batch_in_every_form(dev, T, E, k, real, kind):
    say("padded", kind, T, E, k, real)
    rng = rng_of(22, T, E, k)
    ids, tw = routes(rng, T, E, k)
    ids[int(T * real) if real < 1 else 1:] = -1
    check_forms(dev, kind, ids, tw, E, 192, 96, rng)


# ------------------------------------------------------------- whole layers and their reuse

PLANS = [(12, 64, 4), (100, 64, 4), (40, 256, 8), (700, 512, 8), (300, 16, 4), (600, 40, 17)]


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,E,k", PLANS)
def test_layer_with_reused_grouping(dev, T, E, k, kind):
    """gate_up and down with one workspace and one grouping: against float64 and against calls
    that group for themselves, eager and replayed, on every replay."""
    H, I = 128, 64
    say("layer", kind, T, E, k)
    rng = rng_of(23, T, E, k)
    ids, tw = routes(rng, T, E, k)
    gu, dn = weight(rng, E, 2 * I, H), weight(rng, E, H, I)
    (xd, xs), xv = act_operand(acts(rng, T, H), kind, dev)
    gud, dnd, idd, twd = [up(a, dev) for a in gu], [up(a, dev) for a in dn], up(ids, dev), up(tw, dev)
    mode = nv.OUT_SWIGLU_BF16 if kind == "bf16" else nv.OUT_SWIGLU_MXFP4
    size = max(nv.mxfp4_grouped_workspace_size(T, k, 2 * I, H, E, mode), nv.mxfp4_grouped_workspace_size(T, k, H, I, E, nv.OUT_COMBINE))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=dev)
    a_s = None if kind == "bf16" else torch.empty((T * k, I // 32), dtype=torch.uint8, device=dev)
    a = torch.empty((T * k, I), dtype=torch.bfloat16, device=dev) if kind == "bf16" else torch.empty((T * k, I // 2), dtype=torch.uint8, device=dev)
    out = torch.empty((T, H), device=dev)

    def layer():
        nv.mxfp4_grouped_linear(xd, *gud, idd, x_scales=xs, out_mode=mode, out=a, out_scales=a_s, workspace=ws)
        nv.mxfp4_grouped_linear(a, *dnd, idd, x_scales=a_s, topk_w=twd, out_mode=nv.OUT_COMBINE, rows_per_route=True, out=out, workspace=ws, reuse_grouping=True)

    layer()
    alone = nv.mxfp4_grouped_linear(a, *dnd, idd, x_scales=a_s, topk_w=twd, out_mode=nv.OUT_COMBINE, rows_per_route=True)
    assert torch.equal(out, alone)
    av = num(a) if kind == "bf16" else ref.dequantize(a.cpu().numpy(), a_s.cpu().numpy())
    y, mag, _ = route_rows(av, ref.dequantize(*dn), ids, True)
    want = (y.reshape(T, k, H) * tw[..., None].astype(np.float64)).sum(1)
    t = ((ref.tolerance(y, mag, I) + (k + 1) * 2.0 ** -24 * np.abs(y)).reshape(T, k, H) * tw[..., None]).sum(1) + 1e-37
    assert_near(out, want, t, "down")
    keep = [t.clone() for t in (a, out)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for i in range(4):
        a.view(torch.uint8).fill_(0xA5)
        out.fill_(float("nan"))
        ws.fill_(0x5A if i % 2 else 0xFF)
        nv.mxfp4_grouped_linear(xd, *gud, idd, x_scales=xs)  # the program's own work in between
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.view(torch.uint8), keep[0].view(torch.uint8)) and torch.equal(out, keep[1]), f"replay {i}"


# --------------------------------------------------- check mode and NaN scales in one expert

@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,E,k", [(20, 30, 4), (100, 64, 4), (300, 12, 4)])
def test_nan_scale_in_one_expert_and_check_mode(dev, T, E, k, kind):
    N, K = 70, 288
    rng = rng_of(24, T)
    ids, _ = routes(rng, T, E, k)
    x, (c, s) = acts(rng, T, K), weight(rng, E, N, K)
    (xd, xs), _ = act_operand(x, kind, dev)
    cd, sd, idd = up(c, dev), up(s, dev), up(ids, dev)
    word = torch.zeros(1, dtype=torch.int32, device=dev)

    def call(**kw):
        return nv.mxfp4_grouped_linear(xd, cd, sd, idd, x_scales=xs, faults=word, **kw)

    clean = call(check=True)
    assert int(word) == 0 and torch.isfinite(clean).all()
    e = int(ids[T // 2, 1])
    sd[e, 69, 8] = 255
    y = call()
    assert int(word) == 0  # nothing is scanned without the flag
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[torch.from_numpy(ids.reshape(-1) == e).to(dev), 69] = True
    assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], clean[~hit])
    assert torch.equal(call(check=True)[~hit], clean[~hit])
    assert int(word) == nv.FAULT_NAN_SCALE
    sd[e, 69, 8] = int(s[e, 69, 8])
    word.zero_()
    if kind == "bf16":
        xd[T - 1, 100] = float("-inf")
    else:
        xs[T - 1, 5] = 255
    y = call(check=True)
    assert int(word) == (nv.FAULT_NONFINITE if kind == "bf16" else nv.FAULT_NAN_SCALE)
    assert torch.equal(y[:(T - 1) * k], clean[:(T - 1) * k]) and not torch.isfinite(y[(T - 1) * k:]).all()


# ----------------------------------------------------------- experts past 32-bit offsets

@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_experts_past_32_bit_offsets(dev, kind):
    """4096 experts' weights of more than 2^31 bytes in all: those of 13 experts over and over."""
    E, N, K, P = 4096, 520, 2048, 13
    rng = rng_of(25)
    c, s = weight(rng, P, N, K)
    which = torch.arange(E, device=dev) % P
    wc, ws = up(c, dev)[which], up(s, dev)[which]
    assert wc.numel() > 2 ** 31
    w = ref.dequantize(c, s)
    for T, k in ((8, 4), (100, 4), (17000, 4)):  # by routes, by slots, in tiles
        say("experts past 2^31 bytes", kind, T, k)
        ids = np.argsort(rng.random((T, 8)), 1)[:, :k].astype(np.int32)
        ids = ids * (E // 8) + rng.integers(0, E // 8, (T, k)).astype(np.int32)
        ids[::3, 0] = rng.integers(E - 30, E, ids[::3, 0].size)
        for t in np.flatnonzero([len(set(r)) < k for r in ids.tolist()]):
            ids[t] = [0, E - 1, E // 2, 5]
        (xd, xs), xv = act_operand(acts(rng, T, K), kind, dev)
        y = nv.mxfp4_grouped_linear(xd, wc, ws, up(ids, dev), x_scales=xs)
        flat = ids.reshape(-1)
        some = np.unique(np.r_[np.arange(min(T * k, 64)), np.argsort(-flat, kind="stable")[:40], T * k - 3:T * k])
        for e in range(P):
            mine = some[flat[some] % P == e]
            want, mag = ref.linear(xv[mine // k], w[e])
            assert_near(y[torch.from_numpy(mine).to(dev)], want, ref.tolerance(want, mag, K), (kind, T, e))


# -------------------------------------------------------------------- the smallest scales

@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("M", [1, 20, 150, 3000])
def test_linear_smallest_scales_are_exact(dev, M, kind):
    """Weight values down to 2^-128, below BF16's and fp32's smallest normal, times activations of
    about 2^100: no value of the weight is taken as zero."""
    N, K = 520, 64
    rng = rng_of(26, M)
    c = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    s = np.repeat((np.arange(N) % 20).astype(np.uint8)[:, None], 2, 1)
    (xd, xs), xv = act_operand(torch.ldexp(acts(rng, M, K).float(), torch.tensor(100)).bfloat16(), kind, dev)
    want, mag = ref.linear(xv, ref.dequantize(c, s))
    y = nv.mxfp4_linear(xd, up(c, dev), up(s, dev), x_scales=xs)
    assert_near(y, want, ref.tolerance(want, mag, K), (kind, M))


@pytest.mark.parametrize("M,N,K", [(3, 75, 352), (20, 75, 256), (60, 130, 1024), (300, 4001, 288), (1000, 3300, 512)])
def test_linear_activation_scales_at_any_address(dev, M, N, K):
    """Activations in MXFP4 whose scale rows begin at any byte, between scales that are NaN."""
    rng = rng_of(27, M)
    c, s = weight(rng, N, K)
    (xd, xs), xv = act_operand(acts(rng, M, K), "mxfp4", dev)
    want, mag = ref.linear(xv, ref.dequantize(c, s))
    cd, sd = up(c, dev), up(s, dev)
    for at in (1, 2, 3, 4):
        buf = torch.full((xs.numel() + 8,), 255, dtype=torch.uint8, device=dev)
        moved = buf[at:at + xs.numel()].view(xs.shape)
        moved.copy_(xs)
        assert_near(nv.mxfp4_linear(xd, cd, sd, x_scales=moved), want, ref.tolerance(want, mag, K), (M, N, K, at))
