"""The FP8 operators and the router of libnvfp4.so (include/fp8.h) over torch tensors:
quantization with scales for blocks of 128 and its way back, the linear layer, its expert-grouped
form, and the routes that the grouped forms read. As in _mx.py, nothing is computed here, each
call runs on the current stream of its tensors' device, and the checks build no message before
one fails."""
from __future__ import annotations

import ctypes

import torch

from . import _binding
from ._binding import F_CHECK, OUT_COMBINE, OUT_REUSE_GROUPING, OUT_ROUTES, OUT_SWIGLU_BF16, _check
from ._mx import _BF16, _F32, _TYPES, _U8, _dense, _device, _new, _out, _rows, _run, _word

OUT_SWIGLU_FP8 = 4
FP8_EXPORTS = ("fp8_quantize", "fp8_dequantize", "fp8_linear", "fp8_grouped_linear", "moe_route")

_ACT_BF16, _ACT_FP8 = 0, 1
_F8, _I32 = torch.float8_e4m3fn, torch.int32
_X_TYPES, _X8_TYPES = (_BF16,), (_F8,)
_strided = torch.empty_strided
_BLOCK_ROWS = (1, 128)
_SCORING = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORE = {"max": 0, "top2": 1}
_lib = None


def _load():
    """The library, the argument types of these entry points set."""
    global _lib
    if _lib is None:
        lib = _binding.load_library()
        vp, i64, i32, u32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32
        lib.fp8_quantize.argtypes = [i32, vp, i64, i64, i64, i32, i32, vp, vp, vp, vp]
        lib.fp8_dequantize.argtypes = [vp, vp, i64, i64, i32, i32, vp, i64, vp]
        lib.fp8_linear.argtypes = [i32, vp, vp, i64, i64, i64, i64, vp, vp, i32, vp, i64, u32, vp, vp]
        lib.fp8_grouped_linear.argtypes = [i32, vp, vp, i64, i32, i64, i32, i64, i64, i32, vp, vp, vp, vp, i32, i32,
                                           vp, vp, vp, ctypes.POINTER(ctypes.c_size_t), u32, vp, vp]
        lib.moe_route.argtypes = [i32, vp, i64, i64, i32, i32, i32, vp, i32, i32, i32, i32, ctypes.c_float, vp, vp, vp]
        for name in FP8_EXPORTS:
            getattr(lib, name).restype = i32
        _lib = lib
    return _lib


def _blocks(n):
    return (n + 127) >> 7


def _codes(codes, scales, dims, index):
    """(shape of the codes, codes address, scales address) of a weight."""
    shape = codes.shape
    if len(shape) != dims or codes.dtype is not _F8 or not codes.is_contiguous():
        raise ValueError(f"w_codes: contiguous {_F8} of {dims} dimensions is needed, got {codes.dtype} {tuple(shape)}")
    blocks = ((shape[-2] + 127) >> 7, (shape[-1] + 127) >> 7)
    if dims == 3:
        blocks = (shape[0], *blocks)
    if scales.dtype is not _F32 or scales.shape != blocks or scales.get_device() != index or not scales.is_contiguous():
        _dense(scales, "w_scales", _F32, blocks, index)  # says what is wrong
    return shape, codes.data_ptr(), scales.data_ptr()


def _acts(x, x_scales, K, index):
    """(kind, rows, x address, scales address, row pitch) of the activations."""
    shape = x.shape
    if x_scales is None and x.dtype is _BF16 and len(shape) == 2 and shape[1] == K and x.get_device() == index and x.is_contiguous():
        return _ACT_BF16, shape[0], x.data_ptr(), None, K
    if x.get_device() != index:
        raise ValueError(f"x is on {x.device}, the weight on cuda:{index}")
    M, cols, ld = _rows(x, "x", _X_TYPES if x_scales is None else _X8_TYPES)
    if cols != K:
        raise ValueError(f"x: rows of {K} values are needed, got {cols}")
    if x_scales is None:
        return _ACT_BF16, M, x.data_ptr(), None, ld
    return _ACT_FP8, M, x.data_ptr(), _dense(x_scales, "x_scales", _F32, (M, (K + 127) >> 7), index), ld


def _check_block_rows(block_rows):
    if block_rows not in _BLOCK_ROWS:
        raise ValueError(f"block_rows: 1 or 128 is needed, got {block_rows}")


def fp8_quantize(x, *, block_rows=1, pow2_scales=False, faults=None, codes=None, scales=None):
    """Quantize x (BF16 or fp32, [M][K], rows may be strided) to FP8 on the device, a scale for
    each block of block_rows x 128 (1: activations, 128: weights); returns (codes [M][K]
    float8_e4m3fn, scales [ceil(M/block_rows)][ceil(K/128)] fp32). pow2_scales: scales are powers
    of two. `faults`: a device int32 that receives FAULT_NONFINITE."""
    index = _device(x)
    M, K, ld = _rows(x, "x", _TYPES)
    if block_rows not in _BLOCK_ROWS:
        _check_block_rows(block_rows)
    down, along = M if block_rows == 1 else (M + 127) >> 7, (K + 127) >> 7
    if codes is None:
        codes = _strided((M, K), (K, 1), dtype=_F8, device=x.device)
        cp = codes.data_ptr()
    else:
        cp = _dense(codes, "codes", _F8, (M, K), index)
    if scales is None:
        scales = _strided((down, along), (along, 1), dtype=_F32, device=x.device)
        sp = scales.data_ptr()
    else:
        sp = _dense(scales, "scales", _F32, (down, along), index)
    _run((_lib or _load()).fp8_quantize, "fp8_quantize", index, _TYPES[x.dtype], x.data_ptr(), ld, M, K, block_rows,
         1 if pow2_scales else 0, cp, sp, None if faults is None else _word(faults, index))
    return codes, scales


def fp8_dequantize(codes, scales, *, block_rows=1, dtype=_BF16, out=None):
    """The values of codes [M][K] float8_e4m3fn and scales [ceil(M/block_rows)][ceil(K/128)] fp32
    as [M][K] of `dtype` (BF16 or fp32; `out`'s, when that is given)."""
    index = _device(codes)
    if codes.dim() != 2:
        raise ValueError(f"codes: a matrix of {_F8} is needed, got {codes.dtype} {tuple(codes.shape)}")
    M, K = codes.shape
    cp = _dense(codes, "codes", _F8, (M, K), index)
    _check_block_rows(block_rows)
    sp = _dense(scales, "scales", _F32, (M if block_rows == 1 else _blocks(M), _blocks(K)), index)
    out, ld = _out(out, dtype, M, K, index, codes)
    _run((_lib or _load()).fp8_dequantize, "fp8_dequantize", index, cp, sp, M, K, block_rows, _TYPES[out.dtype],
         out.data_ptr(), ld)
    return out


def fp8_linear(x, w_codes, w_scales, *, x_scales=None, out=None, out_dtype=_F32, check=False, faults=None):
    """y = x W^T for an FP8 weight (codes [N][K] float8_e4m3fn, scales [ceil(N/128)][ceil(K/128)]
    fp32). x is BF16 [M][K] (W8A16) or FP8 codes [M][K] with x_scales [M][ceil(K/128)] (W8A8);
    its rows may be strided. y is [M][N] of out_dtype (fp32 or BF16; `out`'s, when that is given).
    check=True scans the operands first and ORs FAULT_* bits into `faults` (a device int32 word,
    required then)."""
    index = _device(w_codes)
    (N, K), cp, sp = _codes(w_codes, w_scales, 2, index)
    act, M, xp, xsp, ldx = _acts(x, x_scales, K, index)
    if out is None and out_dtype in _TYPES:
        out, y_type, ldy = _strided((M, N), (N, 1), dtype=out_dtype, device=w_codes.device), _TYPES[out_dtype], N
    else:
        out, ldy = _out(out, out_dtype, M, N, index, w_codes)
        y_type = _TYPES[out.dtype]
    _run((_lib or _load()).fp8_linear, "fp8_linear", index, act, xp, xsp, ldx, M, N, K, cp, sp, y_type, out.data_ptr(), ldy,
         1 if check else 0, None if faults is None else _word(faults, index))
    return out


def fp8_grouped_workspace_size(T: int, top_k: int, N: int, K: int, num_experts: int, out_mode: int) -> int:
    """Bytes of workspace that fp8_grouped_linear needs for these sizes."""
    n = ctypes.c_size_t(0)
    st = (_lib or _load()).fp8_grouped_linear(_ACT_BF16, None, None, K, 0, T, top_k, N, K, num_experts, None, None, None,
                                              None, out_mode, 0, None, None, None, ctypes.byref(n), 0, None, None)
    if st:
        _check(st, "fp8_grouped_linear (workspace query)")
    return n.value


def fp8_grouped_linear(x, w_codes, w_scales, topk_ids, *, topk_w=None, out_mode=OUT_ROUTES, rows_per_route=False,
                       x_scales=None, out=None, out_scales=None, out_dtype=None, workspace=None, faults=None,
                       reuse_grouping=False, check=False):
    """Expert-grouped FP8 linear. w_codes [E][N][K] float8_e4m3fn, w_scales
    [E][ceil(N/128)][ceil(K/128)] fp32, topk_ids [T][top_k] int32; x as in fp8_linear, one row per
    token (rows_per_route: per route). See include/fp8.h for the output forms. OUT_ROUTES and
    OUT_COMBINE write out_dtype (fp32 when None; `out`'s, when that is given), OUT_SWIGLU_BF16
    BF16; OUT_SWIGLU_FP8 returns (codes, scales) and takes them as out and out_scales.
    reuse_grouping (OUT_COMBINE with the workspace of the layer's earlier call on the same
    topk_ids) skips the route grouping."""
    index = _device(w_codes)
    (E, N, K), cp, sp = _codes(w_codes, w_scales, 3, index)
    shape = topk_ids.shape
    if len(shape) != 2:
        raise ValueError("topk_ids: [T][top_k] is needed")
    T, top_k = shape
    R = T * top_k
    ip = _dense(topk_ids, "topk_ids", _I32, shape, index)
    tp = None if topk_w is None else _dense(topk_w, "topk_w", _F32, shape, index)
    act, rows, xp, xsp, ldx = _acts(x, x_scales, K, index)
    if rows != (R if rows_per_route else T):
        raise ValueError(f"x: {R if rows_per_route else T} rows are needed, got {rows}")
    osp, y_type, kind = None, 0, _BF16
    if out_mode == OUT_SWIGLU_FP8:
        if out_dtype is not None and out_dtype is not _F8:
            raise ValueError(f"out_dtype: OUT_SWIGLU_FP8 writes {_F8}, got {out_dtype}")
        shape, kind = (R, N // 2), _F8
        if out_scales is None:
            out_scales = _new((R, N // 256), _F32, w_codes)
        osp = _dense(out_scales, "out_scales", _F32, (R, N // 256), index)
    else:
        if out_scales is not None:
            raise ValueError("out_scales: with OUT_SWIGLU_FP8 only")
        if out_mode == OUT_SWIGLU_BF16:
            shape = (R, N // 2)
        elif out_mode == OUT_ROUTES or out_mode == OUT_COMBINE:
            shape, kind = (R if out_mode == OUT_ROUTES else T, N), _F32
        else:
            raise ValueError(f"out_mode: one of the OUT_* forms is needed, got {out_mode}")
        if out_dtype is not None:
            kind = out_dtype
        elif out is not None:
            kind = out.dtype
        if kind not in _TYPES:
            raise ValueError(f"out_dtype: {_BF16} or {_F32} is needed, got {kind}")
        y_type = _TYPES[kind]
    if out is None:
        out = _new(shape, kind, w_codes)
        yp = out.data_ptr()
    else:
        yp = _dense(out, "out", kind, shape, index)
    if workspace is None:
        if reuse_grouping:
            raise ValueError("reuse_grouping needs the workspace that holds the grouping")
        size = fp8_grouped_workspace_size(T, top_k, N, K, E, out_mode)
        workspace = torch.empty(size, dtype=_U8, device=w_codes.device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace: contiguous, on cuda:{index}, is needed")
    nbytes = ctypes.c_size_t(workspace.nbytes)
    _run((_lib or _load()).fp8_grouped_linear, "fp8_grouped_linear", index, act, xp, xsp, ldx,
         1 if rows_per_route else 0, T, top_k, N, K, E, cp, sp, ip, tp,
         out_mode | OUT_REUSE_GROUPING if reuse_grouping else out_mode, y_type, yp, osp, workspace.data_ptr(),
         ctypes.byref(nbytes), F_CHECK if check else 0, None if faults is None else _word(faults, index))
    return (out, out_scales) if out_mode == OUT_SWIGLU_FP8 else out


def moe_route(logits, top_k, *, scoring="softmax", bias=None, groups=1, top_groups=None, group_score="max",
              renormalize=True, scale=1.0, topk_ids=None, topk_w=None):
    """Each token's top_k experts from router logits [T][E] (BF16 or fp32, rows may be strided);
    returns (topk_ids [T][top_k] int32, topk_w [T][top_k] fp32), as the grouped_linear calls of
    every format take them. Scores are a softmax over the experts or sigmoids; `bias` [E] fp32 is
    added to choose by, not to the weights. With groups > 1 only the top_groups (all when None)
    best of as many equal groups of experts are chosen from, a group's score being its best
    expert's ("max") or the sum of its two best ("top2"). With a bias, or groups by "top2", scores
    are compared in 64 bits, otherwise the logits; of equals the lower index comes first.
    renormalize divides the weights by their sum; `scale` multiplies them. Experts whose logit is -inf or NaN are not chosen: where
    they leave fewer than top_k, ids are -1 and weights 0, routes that grouped_linear drops."""
    index = _device(logits)
    T, E, ld = _rows(logits, "logits", _TYPES)
    if scoring not in _SCORING:
        raise ValueError(f"scoring: 'softmax' or 'sigmoid' is needed, got {scoring!r}")
    if group_score not in _GROUP_SCORE:
        raise ValueError(f"group_score: 'max' or 'top2' is needed, got {group_score!r}")
    bp = None if bias is None else _dense(bias, "bias", _F32, (E,), index)
    shape = (T, top_k)
    if topk_ids is None:
        topk_ids = _strided(shape, (top_k, 1), dtype=_I32, device=logits.device)
        ip = topk_ids.data_ptr()
    else:
        ip = _dense(topk_ids, "topk_ids", _I32, shape, index)
    if topk_w is None:
        topk_w = _strided(shape, (top_k, 1), dtype=_F32, device=logits.device)
        wp = topk_w.data_ptr()
    else:
        wp = _dense(topk_w, "topk_w", _F32, shape, index)
    _run((_lib or _load()).moe_route, "moe_route", index, _TYPES[logits.dtype], logits.data_ptr(), ld, T, E, top_k,
         _SCORING[scoring], bp, groups, groups if top_groups is None else top_groups, _GROUP_SCORE[group_score],
         1 if renormalize else 0, scale, ip, wp)
    return topk_ids, topk_w
