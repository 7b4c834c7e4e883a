"""moe_route on the GPU against the definition in long double (f8_reference.route): ids have to be
equal, weights within a rounding to fp32."""
import numpy as np
import pytest
import torch

import f8_reference as ref
import nvfp4_block_scaled_linear_amd as nv
from gpu_helpers import device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return device()


def check(logits, k, dev, bias=None, dtype=torch.float32, **kw):
    l = torch.from_numpy(np.asarray(logits, np.float32)).to(dtype)
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32))
    ids, w = nv.moe_route(l.to(dev), k, bias=None if b is None else b.to(dev), **kw)
    want, ww = ref.route(l.float().numpy(), k, bias=None if b is None else b.numpy(), **kw)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    got = ids.cpu().numpy()
    bad = np.flatnonzero((got != want).any(1))
    assert not bad.size, f"{bad.size} rows differ, first {bad[0]}: {got[bad[0]]} for {want[bad[0]]}"
    # 64-bit sums and a rounding to fp32 (half a step), which may be subnormal
    assert np.all(np.abs(w.double().cpu().numpy() - ww) <= (2.0 ** -24 + 1e-12) * np.abs(ww) + 2.0 ** -150)
    return ids, w


CASES = [
    dict(E=1, k=1), dict(E=2, k=2), dict(E=7, k=3), dict(E=64, k=8), dict(E=65, k=6), dict(E=128, k=8), dict(E=160, k=6, groups=8, top_groups=3),
    dict(E=256, k=8, groups=8, top_groups=4, group_score="top2"), dict(E=384, k=8), dict(E=512, k=64, groups=64, top_groups=20), dict(E=60, k=4),
    dict(E=1000, k=17, groups=5, top_groups=2, group_score="top2"), dict(E=4096, k=64), dict(E=2050, k=9, groups=1025, top_groups=30, group_score="top2"),
    dict(E=12, k=6, groups=6, top_groups=3), dict(E=12, k=2, groups=12, top_groups=7, group_score="top2"), dict(E=96, k=96 // 2, groups=2, top_groups=1),
    dict(E=100, k=5, groups=4, top_groups=4), dict(E=72, k=3, groups=3, top_groups=1), dict(E=192, k=8, groups=6, top_groups=2, group_score="top2"),
    dict(E=300, k=4, groups=100, top_groups=3), dict(E=4096, k=3, groups=4096, top_groups=5),
]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_routes(dev, case, scoring, with_bias):
    print("route", case, scoring, with_bias, flush=True)
    case = dict(case)
    E, k = case.pop("E"), case.pop("k")
    rng = np.random.default_rng([9, E, k])
    bias = 0.1 * rng.standard_normal(E) if with_bias else None
    for T in (1, 3, 33) if E > 600 else (1, 5, 257):
        logits = 2 * rng.standard_normal((T, E))
        for dtype in (torch.float32, torch.bfloat16):
            check(logits, k, dev, bias, dtype, scoring=scoring, **case)
        check(logits, k, dev, bias, scoring=scoring, renormalize=False, scale=2.5, **case)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top", [(128, 8, 1, 1), (256, 8, 8, 4), (48, 5, 6, 2), (600, 6, 1, 1)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_equal_scores_go_to_the_lowest_index(dev, E, k, groups, top, scoring, group_score):
    """Few different values, all equal, and -0 beside +0, with and without a bias of few values."""
    rng = np.random.default_rng([10, E])
    logits = rng.integers(-2, 3, (200, E)) * 0.5
    logits[::7] = 0.25
    logits[1::7] = np.where(rng.random((len(logits[1::7]), E)) < 0.5, -0.0, 0.0)
    kw = dict(scoring=scoring, groups=groups, top_groups=top, group_score=group_score)
    check(logits, k, dev, **kw)
    check(logits, k, dev, np.zeros(E), **kw)
    check(logits, k, dev, rng.integers(0, 2, E) * 0.5, **kw)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top", [(64, 8, 1, 1), (256, 8, 8, 4), (30, 6, 5, 2), (1024, 8, 1, 1)])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_masks_and_non_finite_logits(dev, E, k, groups, top, scoring, with_bias, group_score):
    """Rows with all, most or some experts masked by -inf, by the type's lowest value and by NaN,
    +inf among them; biases of -inf, NaN and +inf."""
    rng = np.random.default_rng([11, E])
    l = rng.standard_normal((120, E)).astype(np.float32)
    l[0], l[1], l[2] = -np.inf, np.nan, np.finfo(np.float32).min
    l[3, 1:], l[4, :-1] = -np.inf, np.nan
    l[5:30][rng.random((25, E)) < 0.5] = -np.inf
    l[30:60][rng.random((30, E)) < 0.97] = -np.inf
    l[60:70][rng.random((10, E)) < 0.5] = np.finfo(np.float32).min
    l[70:80][rng.random((10, E)) < 0.05] = np.inf
    l[80:90][rng.random((10, E)) < 0.3] = np.nan
    l[90, :] = np.inf
    l[91] = np.finfo(np.float32).max
    l[92:95] *= 1e30
    bias = None
    if with_bias:
        bias = 0.1 * rng.standard_normal(E)
        bias[:4] = -np.inf, np.nan, np.inf, -3.0
    kw = dict(scoring=scoring, groups=groups, top_groups=top, group_score=group_score)
    for renormalize in (True, False):
        ids, w = check(l, k, dev, bias, renormalize=renormalize, **kw)
        assert (ids[:2] == -1).all() and (w[:2] == 0).all()
    check(np.clip(l, -3e38, 3e38), k, dev, bias, torch.bfloat16, **kw)


MANY = [dict(E=8, k=2), dict(E=16, k=15), dict(E=60, k=4), dict(E=64, k=8, groups=2, top_groups=1), dict(E=96, k=6, groups=3, top_groups=2),
        dict(E=128, k=8), dict(E=128, k=8, groups=8, top_groups=3), dict(E=160, k=6, groups=8, top_groups=3), dict(E=250, k=13),
        dict(E=256, k=8, groups=8, top_groups=4), dict(E=256, k=1, groups=16, top_groups=15), dict(E=256, k=15, groups=4, top_groups=4), dict(E=256, k=16)]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("case", MANY, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_many_tokens(dev, case, scoring, with_bias, group_score):
    """Enough tokens for four to a wave: spread and close logits, equal ones, masked and padded rows."""
    print("many tokens", case, scoring, with_bias, group_score, flush=True)
    case = dict(case)
    E, k = case.pop("E"), case.pop("k")
    rng = np.random.default_rng([14, E, k])
    T = 4099
    l = 2 * rng.standard_normal((T, E))
    l[100:200] = 0.5 * rng.integers(-2, 3, (100, E))
    l[200:300] = rng.standard_normal((100, 1)) + 1e-6 * rng.standard_normal((100, E))
    l[300:500][rng.random((200, E)) < 0.6] = -np.inf
    l[500:520], l[520:540] = 0.0, np.finfo(np.float32).min
    l[540:600][rng.random((60, E)) < 0.2] = np.nan
    l[600:620][rng.random((20, E)) < 0.1] = np.inf
    l[4000:] = -np.inf
    bias = 0.1 * rng.standard_normal(E) if with_bias else None
    kw = dict(scoring=scoring, group_score=group_score, **case)
    ids, w = check(l, k, dev, bias, **kw)
    assert (ids[4000:] == -1).all() and not w[4000:].any()
    check(l, k, dev, bias, renormalize=False, scale=2.5, **kw)
    check(np.clip(l, -3e38, None), k, dev, bias, torch.bfloat16, **kw)
    if with_bias:
        check(l, k, dev, 0.5 * rng.integers(0, 2, E), torch.bfloat16, **kw)


def extreme_logits(T, E, rng):
    """fp32 rows, a quarter each: scores that round to 1 in 64 bits, scores that round to 0, logits that differ in
    their last bits only, and logits near 0 whose scores are all alike; most have ties among the best."""
    l = np.empty((T, E), np.float32)
    a, b, c = T // 4, T // 2, 3 * T // 4
    l[:a] = 0.5 * rng.integers(60, 161, (a, E))
    l[a:b] = 50.0 * rng.integers(-40, 41, (b - a, E))
    l[b:c] = np.float32(45) + np.spacing(np.float32(45)) * rng.integers(-40, 41, (c - b, E))
    l[c:] = 1e-30 * rng.integers(-40, 41, (T - c, E))
    return l


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top", [(60, 4, 1, 1), (64, 8, 2, 1), (96, 6, 3, 2), (128, 8, 1, 1), (128, 1, 8, 3), (256, 8, 8, 4), (256, 15, 1, 1)])
def test_without_bias_the_order_is_that_of_the_logits(dev, E, k, groups, top, scoring):
    """Also where scores in 64 bits are equal, for few tokens and for many."""
    l = extreme_logits(4100, E, np.random.default_rng([15, E, k]))
    kw = dict(scoring=scoring, groups=groups, top_groups=top)
    ids, _ = check(l, k, dev, **kw)
    few, _ = check(l[:4095], k, dev, **kw)
    assert torch.equal(ids[:4095], few)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias,groups,top,group_score", [(False, 1, 1, "max"), (True, 1, 1, "max"), (False, 4, 2, "max"), (True, 4, 2, "max"),
                                                               (False, 4, 2, "top2"), (True, 4, 2, "top2")])
def test_a_tokens_experts_do_not_depend_on_the_others(dev, with_bias, groups, top, group_score, scoring):
    rng = np.random.default_rng([16, groups])
    E = 128
    l = extreme_logits(4400, E, rng)
    l[4100:] = 2 * rng.standard_normal((300, E))
    l = torch.from_numpy(l[rng.permutation(len(l))]).to(dev)
    bias = torch.from_numpy((0.25 * rng.integers(0, 3, E)).astype(np.float32)).to(dev) if with_bias else None
    kw = dict(scoring=scoring, bias=bias, groups=groups, top_groups=top, group_score=group_score)
    ids, _ = nv.moe_route(l, 8, **kw)
    parts = [nv.moe_route(part, 8, **kw)[0] for part in l.split(1100)]
    assert torch.equal(ids, torch.cat(parts))

@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [5, 4099])
@pytest.mark.parametrize("E", [64, 128, 256])
def test_groups_masked_by_low_biases(dev, E, T, scoring):
    """Groups whose biases are the type's lowest value, or low enough for the sum of two to pass it, come
    before closed ones and in the order of their sums in 64 bits."""
    rng = np.random.default_rng([17, E, T])
    l = rng.standard_normal((T, E))
    least = float(np.finfo(np.float32).min)
    group = np.arange(E) // (E // 4)
    for low in ([-np.inf, least, -2e38, -3e38], [least, -np.inf, -2.5e38, -np.inf], [-np.inf, least, -np.inf, 0.1], [least, -2e38, least, -2e38]):
        for top in (1, 2, 3):
            check(l, 15, dev, np.array(low)[group], scoring=scoring, groups=4, top_groups=top, group_score="top2")


@pytest.mark.parametrize("T", [3, 4099])
def test_scores_that_round_to_the_same_number_are_equals(dev, T):
    """Groups by their two best, or a bias, compare scores: sigmoids of 40 and of 60 are both 1 in 64 bits, and
    softmax's of -800 and of -900 below 0 both 0. Without either the logits count."""
    l = torch.full((T, 32), 40.0, device=dev)
    l[:, 5] = 60.0
    l[:, 20] = 50.0
    kw = dict(scoring="sigmoid", groups=2)
    for more in (dict(group_score="top2"), dict(bias=torch.zeros(32, device=dev)), dict(group_score="top2", bias=torch.zeros(32, device=dev))):
        assert (nv.moe_route(l, 3, **kw, **more)[0].cpu() == torch.tensor([0, 1, 2])).all()
    assert (nv.moe_route(l, 3, **kw)[0].cpu() == torch.tensor([5, 20, 0])).all()
    l = torch.full((T, 32), -900.0, device=dev)
    l[:, 7], l[:, 9] = 0.0, -800.0
    for more in (dict(group_score="top2"), dict(bias=torch.zeros(32, device=dev))):
        assert (nv.moe_route(l, 3, groups=2, **more)[0].cpu() == torch.tensor([7, 0, 1])).all()
    assert (nv.moe_route(l, 3, groups=2)[0].cpu() == torch.tensor([7, 9, 0])).all()


def test_close_scores(dev):
    """Scores with a bias that differ by less than fp32 can hold are told apart."""
    rng = np.random.default_rng(12)
    T, E = 300, 128
    base = rng.standard_normal((T, 1))
    logits = (base + 1e-6 * rng.standard_normal((T, E))).astype(np.float32)
    for scoring in ("softmax", "sigmoid"):
        check(logits, 8, dev, np.full(E, 0.3), scoring=scoring)
        check(logits, 8, dev, scoring=scoring, groups=8, top_groups=2, group_score="top2")


def test_strided_rows_given_outputs_and_many_tokens(dev):
    rng = np.random.default_rng(13)
    T, E, k = 5001, 96, 6
    logits = rng.standard_normal((T, E)).astype(np.float32)
    wide = torch.full((T, E + 5), float("nan"), device=dev)
    wide[:, 3:3 + E] = torch.from_numpy(logits).to(dev)
    ids = torch.full((T + 2, k), 77, dtype=torch.int32, device=dev)
    w = torch.full((T + 2, k), 77.0, device=dev)
    got = nv.moe_route(wide[:, 3:3 + E], k, topk_ids=ids[1:-1], topk_w=w[1:-1])
    assert got[0].data_ptr() == ids[1:].data_ptr()
    want, ww = ref.route(logits, k)
    assert np.array_equal(ids[1:-1].cpu().numpy(), want)
    assert np.all(np.abs(w[1:-1].double().cpu().numpy() - ww) <= (2.0 ** -24 + 1e-12) * ww)
    for t in (ids, w):
        assert (t[[0, -1]] == 77).all()


def test_binding_refusals(dev):
    l = torch.zeros((4, 16), device=dev)
    for call in (
        lambda: nv.moe_route(l.half(), 2), lambda: nv.moe_route(l.t(), 2), lambda: nv.moe_route(l[0], 2), lambda: nv.moe_route(l, 2, scoring="relu"),
        lambda: nv.moe_route(l, 2, group_score="sum"), lambda: nv.moe_route(l, 2, bias=l[0].double()), lambda: nv.moe_route(l, 2, bias=l[0, :8]),
        lambda: nv.moe_route(l, 2, topk_ids=torch.zeros((4, 2), device=dev)), lambda: nv.moe_route(l, 2, topk_w=torch.zeros((4, 3), device=dev)),
        lambda: nv.moe_route(l, 2, topk_w=torch.zeros((4, 2))),
    ):
        with pytest.raises(ValueError):
            call()
    for call, name in (
        (lambda: nv.moe_route(l, 0), "ARG"), (lambda: nv.moe_route(l, 17), "ARG"), (lambda: nv.moe_route(l, 2, groups=3), "ARG"),
        (lambda: nv.moe_route(l, 2, groups=4, top_groups=5), "ARG"), (lambda: nv.moe_route(l, 9, groups=2, top_groups=1), "ARG"),
        (lambda: nv.moe_route(l[:0], 2), "SHAPE"),
    ):
        with pytest.raises(nv.NVFP4Error, match=name):
            call()
