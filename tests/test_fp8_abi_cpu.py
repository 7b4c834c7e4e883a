"""The C ABI of the FP8 operators and the router on the host (no GPU needed): every declared call
is exported, and bad arguments are refused by name before anything is enqueued. Every call here
fails host-side validation; the fake device addresses are never dereferenced."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import f8_reference as ref
import nvfp4_block_scaled_linear_amd as nv
from nvfp4_block_scaled_linear_amd import _fp8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ARG, ERR_WORKSPACE = 0, 1, 2, 3, 4, 5
P = 0x7F0000000000  # an aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_block_scaled_linear_amd import build
        build.build()
    return _fp8._load()


def test_header_and_binding_name_the_same_calls(lib):
    text = open(os.path.join(ROOT, "include", "fp8.h")).read()
    names = set(re.findall(r"^nvfp4_status\s+(\w+)\(", text, re.M))
    assert names == set(nv.FP8_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", nv.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert names <= exported


def test_header_compiles_as_c():
    code = '#include "fp8.h"\n#include "mxfp4.h"\nint main(void) { return FP8_OUT_SWIGLU_FP8 - 4 + ROUTE_SOFTMAX; }\n'
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-x", "c", "-I", os.path.join(ROOT, "include"), "-"],
                       input=code, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("kw,status", [
    (dict(t=2), ERR_ARG), (dict(t=-1), ERR_ARG), (dict(rows=2), ERR_ARG), (dict(rows=0), ERR_ARG), (dict(rule=2), ERR_ARG),
    (dict(K=0), ERR_SHAPE), (dict(K=24), ERR_SHAPE), (dict(K=-16), ERR_SHAPE), (dict(K=1 << 23, ld=1 << 23), ERR_SHAPE),
    (dict(M=0), ERR_SHAPE), (dict(M=-1), ERR_SHAPE), (dict(M=1 << 31), ERR_SHAPE), (dict(ld=4064), ERR_SHAPE), (dict(ld=1 << 31), ERR_SHAPE),
    (dict(x=None), ERR_NULL), (dict(c=None), ERR_NULL), (dict(s=None), ERR_NULL), (dict(x=P + 8), ERR_ALIGN), (dict(ld=4100), ERR_ALIGN),
    (dict(t=1, ld=4098), ERR_ALIGN), (dict(c=P + 8), ERR_ALIGN), (dict(s=P + 2), ERR_ALIGN), (dict(f=P + 2), ERR_ALIGN),
])
def test_quantize_refusals(lib, kw, status):
    def call(t=0, x=P, ld=4096, M=4, K=4096, rows=1, rule=0, c=P, s=P, f=None):
        return lib.fp8_quantize(t, x, ld, M, K, rows, rule, c, s, f, None)
    assert call(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(t=2), ERR_ARG), (dict(rows=64), ERR_ARG), (dict(K=40), ERR_SHAPE), (dict(M=0), ERR_SHAPE), (dict(ld=100), ERR_SHAPE),
    (dict(y=None), ERR_NULL), (dict(c=None), ERR_NULL), (dict(s=None), ERR_NULL), (dict(y=P + 8), ERR_ALIGN), (dict(ld=4100), ERR_ALIGN),
    (dict(t=1, ld=4098), ERR_ALIGN), (dict(c=P + 4), ERR_ALIGN), (dict(s=P + 1), ERR_ALIGN),
])
def test_dequantize_refusals(lib, kw, status):
    def call(t=0, c=P, s=P, M=4, K=4096, rows=1, y=P, ld=4096):
        return lib.fp8_dequantize(c, s, M, K, rows, t, y, ld, None)
    assert call(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(K=0), ERR_SHAPE), (dict(K=40), ERR_SHAPE), (dict(M=0), ERR_SHAPE), (dict(N=0), ERR_SHAPE), (dict(M=1 << 31), ERR_SHAPE),
    (dict(N=1 << 31), ERR_SHAPE), (dict(act=2), ERR_ARG), (dict(act=-1), ERR_ARG), (dict(t=2), ERR_ARG), (dict(x=None), ERR_NULL),
    (dict(x=P + 8), ERR_ALIGN), (dict(ldx=4000), ERR_SHAPE), (dict(ldx=4100), ERR_ALIGN), (dict(ldx=1 << 29), ERR_SHAPE), (dict(xs=P), ERR_ARG),
    (dict(act=1), ERR_NULL), (dict(act=1, xs=P + 2), ERR_ALIGN), (dict(act=1, xs=P, ldx=4104), ERR_ALIGN), (dict(act=1, xs=P, ldx=1 << 30), ERR_SHAPE),
    (dict(wc=None), ERR_NULL), (dict(ws=None), ERR_NULL), (dict(wc=P + 4), ERR_ALIGN), (dict(ws=P + 2), ERR_ALIGN),
    (dict(y=None), ERR_NULL), (dict(ldy=100), ERR_SHAPE), (dict(y=P + 2), ERR_ALIGN), (dict(t=0, y=P + 1), ERR_ALIGN),
    (dict(flags=2), ERR_ARG), (dict(flags=1), ERR_NULL), (dict(flags=1, f=P + 2), ERR_ALIGN), (dict(f=P + 1), ERR_ALIGN),
])
def test_linear_refusals(lib, kw, status):
    def call(act=0, x=P, xs=None, ldx=4096, M=4, N=128, K=4096, wc=P, ws=P, t=1, y=P, ldy=128, flags=0, f=None):
        return lib.fp8_linear(act, x, xs, ldx, M, N, K, wc, ws, t, y, ldy, flags, f, None)
    assert call(**kw) == status


def grouped(lib, act=0, x=P, xs=None, ldx=2048, rows_mode=0, T=16, k=8, N=1536, K=2048, E=128, wc=P, ws=P, ids=P, tw=P,
            mode=0, t=1, y=P, ys=None, work=P, nbytes=1 << 40, flags=0, f=None, pass_nbytes=True):
    n = ctypes.c_size_t(nbytes)
    st = lib.fp8_grouped_linear(act, x, xs, ldx, rows_mode, T, k, N, K, E, wc, ws, ids, tw, mode, t, y, ys, work,
                                ctypes.byref(n) if pass_nbytes else None, flags, f, None)
    return st, n.value


@pytest.mark.parametrize("kw,status", [
    (dict(pass_nbytes=False), ERR_NULL), (dict(E=0), ERR_ARG), (dict(E=5000), ERR_ARG), (dict(k=0), ERR_ARG), (dict(k=129), ERR_ARG),
    (dict(E=128, k=65), ERR_ARG), (dict(rows_mode=2), ERR_ARG), (dict(mode=3), ERR_ARG), (dict(mode=5), ERR_ARG), (dict(mode=-1), ERR_ARG),
    (dict(t=2), ERR_ARG), (dict(mode=0x100), ERR_ARG), (dict(mode=0x101, t=0), ERR_ARG), (dict(mode=0x104, t=0), ERR_ARG),
    (dict(mode=1, t=1), ERR_ARG), (dict(mode=4, t=1), ERR_ARG), (dict(T=0), ERR_SHAPE), (dict(N=0), ERR_SHAPE), (dict(K=2047), ERR_SHAPE),
    (dict(T=1 << 22, k=2), ERR_SHAPE), (dict(mode=1, t=0, N=1408), ERR_SHAPE), (dict(mode=4, t=0, N=1664, ys=P), ERR_SHAPE),
    (dict(nbytes=100), ERR_WORKSPACE), (dict(T=4096, nbytes=100000), ERR_WORKSPACE), (dict(mode=2, nbytes=1000), ERR_WORKSPACE),
    (dict(work=P + 16), ERR_ALIGN), (dict(x=None), ERR_NULL), (dict(ids=None), ERR_NULL), (dict(y=None), ERR_NULL),
    (dict(mode=2, tw=None), ERR_NULL), (dict(mode=4, t=0), ERR_NULL), (dict(ys=P), ERR_ARG), (dict(ids=P + 2), ERR_ALIGN),
    (dict(tw=P + 2), ERR_ALIGN), (dict(wc=P + 8), ERR_ALIGN), (dict(ws=P + 2), ERR_ALIGN), (dict(mode=4, t=0, ys=P, y=P + 8), ERR_ALIGN),
    (dict(mode=4, t=0, ys=P + 2), ERR_ALIGN), (dict(y=P + 2), ERR_ALIGN), (dict(act=1), ERR_NULL), (dict(act=2), ERR_ARG), (dict(xs=P), ERR_ARG),
    (dict(ldx=2000), ERR_SHAPE), (dict(ldx=1 << 27), ERR_SHAPE), (dict(N=1 << 21), ERR_SHAPE),  # beyond 32-bit offsets
    (dict(flags=2), ERR_ARG), (dict(flags=1), ERR_NULL), (dict(f=P + 2), ERR_ALIGN),
])
def test_grouped_refusals(lib, kw, status):
    assert grouped(lib, **kw)[0] == status


def test_grouped_workspace_query(lib):
    needs = {m: grouped(lib, work=None, nbytes=0, mode=m, t=0) for m in (0, 1, 2, 4)}
    assert all(st == OK and n > 0 for st, n in needs.values())
    assert needs[0][1] == needs[1][1]  # rows go straight to y
    assert needs[2][1] >= needs[0][1] + 16 * 8 * 1536 * 4  # the combine keeps fp32 rows
    assert grouped(lib, work=None, nbytes=0, mode=0x102, t=0)[1] == needs[2][1]
    assert nv.fp8_grouped_workspace_size(16, 8, 1536, 2048, 128, nv.OUT_SWIGLU_FP8) == needs[4][1]


@pytest.mark.parametrize("kw,status", [
    (dict(t=2), ERR_ARG), (dict(E=0), ERR_ARG), (dict(E=4097, ld=5000), ERR_ARG), (dict(scoring=2), ERR_ARG), (dict(scoring=-1), ERR_ARG),
    (dict(gs=2), ERR_ARG), (dict(renorm=2), ERR_ARG), (dict(G=0), ERR_ARG), (dict(G=3, tg=1), ERR_ARG), (dict(G=256), ERR_ARG),
    (dict(tg=0), ERR_ARG), (dict(tg=2), ERR_ARG), (dict(k=0), ERR_ARG), (dict(k=-1), ERR_ARG), (dict(k=65), ERR_ARG), (dict(E=4, k=5), ERR_ARG),
    (dict(G=16, tg=1, k=9), ERR_ARG), (dict(T=0), ERR_SHAPE), (dict(T=-4), ERR_SHAPE), (dict(T=1 << 61), ERR_SHAPE), (dict(T=1 << 62, k=4), ERR_SHAPE), (dict(T=1 << 20), ERR_SHAPE), (dict(ld=127), ERR_SHAPE),
    (dict(ld=1 << 31), ERR_SHAPE), (dict(l=None), ERR_NULL), (dict(ids=None), ERR_NULL), (dict(w=None), ERR_NULL), (dict(l=P + 2), ERR_ALIGN),
    (dict(t=0, l=P + 1), ERR_ALIGN), (dict(ids=P + 2), ERR_ALIGN), (dict(w=P + 2), ERR_ALIGN), (dict(bias=P + 2), ERR_ALIGN),
])
def test_route_refusals(lib, kw, status):
    def call(t=1, l=P, ld=128, T=4, E=128, k=8, scoring=0, bias=None, G=1, tg=1, gs=0, renorm=1, ids=P, w=P):
        return lib.moe_route(t, l, ld, T, E, k, scoring, bias, G, tg, gs, renorm, 1.0, ids, w, None)
    assert call(**kw) == status


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    c, s = torch.zeros((8, 64), dtype=torch.float8_e4m3fn), torch.zeros((1, 1))
    for call in (lambda: nv.fp8_quantize(x), lambda: nv.fp8_dequantize(c, s, block_rows=128), lambda: nv.fp8_linear(x, c, s),
                 lambda: nv.fp8_grouped_linear(x, c[None], s[None], torch.zeros((4, 1), dtype=torch.int32)), lambda: nv.moe_route(x, 2)):
        with pytest.raises(ValueError, match="device tensors"):
            call()


# ------------------------------------------------------------ the reference's own pins

def test_reference_agrees_with_torch_on_every_code():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.TABLE, want, equal_nan=True)
    assert np.array_equal(ref.encode(want[:127]), codes[:127]) and np.array_equal(ref.encode(want[128:255]), codes[128:255])
    mids = np.concatenate([ref.MIDS, -ref.MIDS])
    assert np.array_equal(ref.encode(mids), torch.from_numpy(mids).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_reference_scales():
    x = np.zeros((3, 256), np.float32)
    x[0, 5], x[0, 200], x[1, 7], x[2, 130] = 448, -7, 2.0 ** -149, np.inf
    codes, s = ref.quantize(x)
    assert s[0, 0] == 1 and s[0, 1] == np.float32(7) / np.float32(448) and s[1, 0] == 0 and np.isnan(s[2, 1])
    assert codes[0, 5] == 0x7E and codes[0, 200] == 0xFE and not codes[1:].any()
    assert ref.quantize(x, pow2=True)[1][0].tolist() == [1, 1 / 64]
    codes, s = ref.quantize(x[:2], rows=128)
    assert s.shape == (1, 2) and s[0, 0] == 1


def test_reference_routes():
    l = np.array([[1.0, 3.0, 2.0, 3.0], [-np.inf, np.nan, 0.0, -np.inf], [np.inf, 0.0, 1.0, 2.0]], np.float32)
    ids, w = ref.route(l, 2)
    assert ids.tolist() == [[1, 3], [2, -1], [0, 3]] and np.allclose(w, [[0.5, 0.5], [1, 0], [1, 0]])
    ids, w = ref.route(l[:1], 2, scoring="sigmoid", bias=np.array([5, 0, 0, 0], np.float32), groups=2, top_groups=1, renormalize=False)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, 1 / (1 + np.exp([-1.0, -3.0])))
