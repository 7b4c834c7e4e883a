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
