"""The C ABI of the MXFP4 operators on the host (no GPU needed): every declared call is
exported, and bad arguments are refused by name before anything is enqueued. Every call here
fails host-side validation; the fake device addresses are never dereferenced."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import mx_reference as ref
import nvfp4_block_scaled_linear_amd as nv
from nvfp4_block_scaled_linear_amd import _mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ARG, ERR_WORKSPACE = 0, 1, 2, 3, 4, 5
P = 0x7F0000000000  # an aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_block_scaled_linear_amd import build
        build.build()
    return _mx._load()


def test_header_and_binding_name_the_same_calls(lib):
    text = open(os.path.join(ROOT, "include", "mxfp4.h")).read()
    names = set(re.findall(r"^nvfp4_status\s+(mxfp4_\w+)\(", text, re.M))
    assert names == set(nv.MX_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", nv.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert names <= exported


@pytest.mark.parametrize("kw,status", [
    (dict(t=2), ERR_ARG), (dict(t=-1), ERR_ARG), (dict(K=0), ERR_SHAPE), (dict(K=48), ERR_SHAPE), (dict(K=-32), ERR_SHAPE),
    (dict(K=1 << 23, ld=1 << 23), ERR_SHAPE), (dict(M=0), ERR_SHAPE), (dict(M=-1), ERR_SHAPE), (dict(M=1 << 31), ERR_SHAPE),
    (dict(ld=4064), ERR_SHAPE), (dict(ld=1 << 31), ERR_SHAPE), (dict(x=None), ERR_NULL), (dict(c=None), ERR_NULL),
    (dict(s=None), ERR_NULL), (dict(x=P + 8), ERR_ALIGN), (dict(ld=4100), ERR_ALIGN), (dict(t=1, ld=4098), ERR_ALIGN),
    (dict(c=P + 8), ERR_ALIGN), (dict(f=P + 2), ERR_ALIGN),
])
def test_quantize_refusals(lib, kw, status):
    def call(t=0, x=P, ld=4096, M=4, K=4096, c=P, s=P, f=None):
        return lib.mxfp4_quantize(t, x, ld, M, K, c, s, f, None)
    assert call(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(t=2), ERR_ARG), (dict(K=40), ERR_SHAPE), (dict(M=0), ERR_SHAPE), (dict(ld=100), ERR_SHAPE), (dict(y=None), ERR_NULL),
    (dict(c=None), ERR_NULL), (dict(s=None), ERR_NULL), (dict(y=P + 8), ERR_ALIGN), (dict(ld=4100), ERR_ALIGN),
    (dict(t=1, ld=4098), ERR_ALIGN), (dict(c=P + 4), ERR_ALIGN),
])
def test_dequantize_refusals(lib, kw, status):
    def call(t=0, c=P, s=P, M=4, K=4096, y=P, ld=4096):
        return lib.mxfp4_dequantize(c, s, M, K, t, y, ld, None)
    assert call(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(K=0), ERR_SHAPE), (dict(K=48), ERR_SHAPE), (dict(M=0), ERR_SHAPE), (dict(N=0), ERR_SHAPE), (dict(M=1 << 31), ERR_SHAPE),
    (dict(N=1 << 31), ERR_SHAPE), (dict(act=2), ERR_ARG), (dict(act=-1), ERR_ARG), (dict(t=2), ERR_ARG), (dict(x=None), ERR_NULL),
    (dict(x=P + 8), ERR_ALIGN), (dict(ldx=4000), ERR_SHAPE), (dict(ldx=4100), ERR_ALIGN), (dict(ldx=1 << 29), ERR_SHAPE), (dict(xs=P), ERR_ARG),
    (dict(act=1), ERR_NULL), (dict(wc=None), ERR_NULL), (dict(ws=None), ERR_NULL), (dict(wc=P + 4), ERR_ALIGN),
    (dict(y=None), ERR_NULL), (dict(ldy=100), ERR_SHAPE), (dict(y=P + 2), ERR_ALIGN), (dict(t=0, y=P + 1), ERR_ALIGN),
    (dict(flags=2), ERR_ARG), (dict(flags=1), ERR_NULL), (dict(flags=1, f=P + 2), ERR_ALIGN), (dict(f=P + 1), ERR_ALIGN),
])
def test_linear_refusals(lib, kw, status):
    def call(act=0, x=P, xs=None, ldx=4096, M=4, N=128, K=4096, wc=P, ws=P, t=1, y=P, ldy=128, flags=0, f=None):
        return lib.mxfp4_linear(act, x, xs, ldx, M, N, K, wc, ws, t, y, ldy, flags, f, None)
    assert call(**kw) == status


def grouped(lib, act=0, x=P, xs=None, ldx=2048, rows_mode=0, T=16, k=8, N=1536, K=2048, E=128, wc=P, ws=P, ids=P, tw=P,
            mode=0, t=1, y=P, ys=None, work=P, nbytes=1 << 40, flags=0, f=None, pass_nbytes=True):
    n = ctypes.c_size_t(nbytes)
    st = lib.mxfp4_grouped_linear(act, x, xs, ldx, rows_mode, T, k, N, K, E, wc, ws, ids, tw, mode, t, y, ys, work,
                                  ctypes.byref(n) if pass_nbytes else None, flags, f, None)
    return st, n.value


@pytest.mark.parametrize("kw,status", [
    (dict(pass_nbytes=False), ERR_NULL), (dict(E=0), ERR_ARG), (dict(E=5000), ERR_ARG), (dict(k=0), ERR_ARG), (dict(k=129), ERR_ARG),
    (dict(E=128, k=65), ERR_ARG), (dict(rows_mode=2), ERR_ARG), (dict(mode=4), ERR_ARG), (dict(mode=-1), ERR_ARG), (dict(t=2), ERR_ARG),
    (dict(mode=0x100), ERR_ARG), (dict(mode=0x101, t=0), ERR_ARG), (dict(mode=0x103, t=0), ERR_ARG), (dict(mode=1, t=1), ERR_ARG),
    (dict(mode=3, t=1), ERR_ARG), (dict(T=0), ERR_SHAPE), (dict(N=0), ERR_SHAPE), (dict(K=2047), ERR_SHAPE),
    (dict(T=1 << 22, k=2), ERR_SHAPE), (dict(mode=1, t=0, N=1535), ERR_SHAPE), (dict(mode=3, t=0, N=1568, ys=P), ERR_SHAPE),
    (dict(nbytes=100), ERR_WORKSPACE), (dict(T=4096, nbytes=100000), ERR_WORKSPACE), (dict(mode=2, nbytes=1000), ERR_WORKSPACE), (dict(work=P + 16), ERR_ALIGN), (dict(x=None), ERR_NULL), (dict(ids=None), ERR_NULL),
    (dict(y=None), ERR_NULL), (dict(mode=2, tw=None), ERR_NULL), (dict(mode=3, t=0), ERR_NULL), (dict(ys=P), ERR_ARG),
    (dict(ids=P + 2), ERR_ALIGN), (dict(tw=P + 2), ERR_ALIGN), (dict(wc=P + 8), ERR_ALIGN), (dict(mode=3, t=0, ys=P, y=P + 8), ERR_ALIGN),
    (dict(y=P + 2), ERR_ALIGN), (dict(act=1), ERR_NULL), (dict(act=2), ERR_ARG), (dict(xs=P), ERR_ARG), (dict(ldx=2000), ERR_SHAPE),
    (dict(ldx=1 << 27), ERR_SHAPE), (dict(N=1 << 22), ERR_SHAPE),  # beyond 32-bit offsets
    (dict(flags=2), ERR_ARG), (dict(flags=1), ERR_NULL), (dict(f=P + 2), ERR_ALIGN),
])
def test_grouped_refusals(lib, kw, status):
    assert grouped(lib, **kw)[0] == status


def test_grouped_workspace_query(lib):
    needs = {m: grouped(lib, work=None, nbytes=0, mode=m, t=0) for m in range(4)}
    assert all(st == OK and n > 0 for st, n in needs.values())
    assert needs[0][1] == needs[1][1] == needs[3][1]  # rows go straight to y
    assert needs[2][1] >= needs[0][1] + 16 * 8 * 1536 * 4  # the combine keeps fp32 rows
    assert grouped(lib, work=None, nbytes=0, mode=0x102, t=0)[1] == needs[2][1]
    assert nv.mxfp4_grouped_workspace_size(16, 8, 1536, 2048, 128, nv.OUT_SWIGLU_MXFP4) == needs[3][1]


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    c, s = torch.zeros((8, 32), dtype=torch.uint8), torch.zeros((8, 2), dtype=torch.uint8)
    for call in (lambda: nv.mxfp4_quantize(x), lambda: nv.mxfp4_dequantize(c, s), lambda: nv.mxfp4_linear(x, c, s),
                 lambda: nv.mxfp4_grouped_linear(x, c[None], s[None], torch.zeros((4, 1), dtype=torch.int32))):
        with pytest.raises(ValueError, match="device tensors"):
            call()


# ------------------------------------------------------------ the reference's own pins

def test_reference_codes_of_known_values():
    row = np.zeros((1, 64))
    row[0, :12] = [6.0, -6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.0, 0.26]
    row[0, 32:34] = [448.0, -1.0]
    codes, scales = ref.quantize(row)
    # 7.9 sets the first block's exponent to 2 - 2; ties go to the even code; 7.9 saturates
    assert scales.tolist() == [[127, 127 + 8 - 2]]
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(-1)
    assert nib[:12].tolist() == [7, 15, 0, 2, 2, 4, 4, 6, 6, 7, 8, 1]
    assert nib[32:34].tolist() == [7, 8]  # 448 / 64 = 7 saturates; -1/64 rounds to -0
    assert np.array_equal(ref.dequantize(codes, scales)[0, :8], [6, -6, 0, 1, 1, 2, 2, 4])


def test_reference_scale_edges():
    for top, scale in ((0.0, 0), (2.0 ** -149, 0), (2.0 ** -126, 0), (2.0 ** -125, 0), (2.0 ** -124, 1), (1.0, 125), (3.999, 126),
                       (4.0, 127), (np.finfo(np.float32).max, 252)):
        row = np.zeros((1, 32))
        row[0, 5] = top
        assert ref.quantize(row)[1][0, 0] == scale, top
    row[0, 9] = np.nan
    codes, scales = ref.quantize(row)
    assert scales[0, 0] == 255 and not codes.any() and np.isnan(ref.dequantize(codes, scales)).all()
