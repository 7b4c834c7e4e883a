"""The MXFP4 operators of libnvfp4.so (include/mxfp4.h) over torch tensors: quantization and
its way back, the linear layer and its expert-grouped form. As in _binding.py, nothing is
computed here. Each call runs on the current stream of its tensors' device.

A decode step makes these calls by the hundred, and a small one's kernel takes a few
microseconds, so the checks below build no message before one fails."""
from __future__ import annotations

import ctypes

import torch

from . import _binding
from ._binding import F_CHECK, OUT_COMBINE, OUT_REUSE_GROUPING, OUT_ROUTES, OUT_SWIGLU_BF16, _check

OUT_SWIGLU_MXFP4 = 3
MX_EXPORTS = ("mxfp4_quantize", "mxfp4_dequantize", "mxfp4_linear", "mxfp4_grouped_linear")

_ACT_BF16, _ACT_MXFP4 = 0, 1
_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8
_TYPES = {_BF16: 0, _F32: 1}
_X_TYPES = (_BF16,)
_lib = None


def _public_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


def _public_device():
    return torch.cuda.current_device()


# handle of a device's current stream, and the current device: where torch has them without the
# objects and checks of torch.cuda's forms, which cost as much as the rest of a call's host work
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", _public_device)


def _load():
    """The library, the argument types of these entry points set."""
    global _lib
    if _lib is None:
        lib = _binding.load_library()
        vp, i64, i32, u32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32
        lib.mxfp4_quantize.argtypes = [i32, vp, i64, i64, i64, vp, vp, vp, vp]
        lib.mxfp4_dequantize.argtypes = [vp, vp, i64, i64, i32, vp, i64, vp]
        lib.mxfp4_linear.argtypes = [i32, vp, vp, i64, i64, i64, i64, vp, vp, i32, vp, i64, u32, vp, vp]
        lib.mxfp4_grouped_linear.argtypes = [i32, vp, vp, i64, i32, i64, i32, i64, i64, i32, vp, vp, vp, vp, i32, i32,
                                             vp, vp, vp, ctypes.POINTER(ctypes.c_size_t), u32, vp, vp]
        for name in MX_EXPORTS:
            getattr(lib, name).restype = i32
        _lib = lib
    return _lib


def _run(fn, name, index, *args):
    """Calls an entry point on the current stream of device `index`."""
    if index == _current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st:
        _check(st, name)


def _device(t):
    """Index of the device that a tensor lies on."""
    index = t.get_device()
    if index < 0:
        raise ValueError("libnvfp4 takes device tensors only")
    return index


def _new(shape, dtype, like):
    """A dense matrix on the device of `like` (empty_strided: the least host work)."""
    return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=like.device)


def _dense(t, name, dtype, shape, index):
    """Address of a contiguous tensor of this type, shape and device."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: {dtype} of shape {tuple(shape)} is needed, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the call on cuda:{index}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, types):
    """(rows, columns, row pitch) of a matrix of one of `types` with unit inner stride."""
    if t.dim() != 2 or t.dtype not in types:
        raise ValueError(f"{name}: a matrix of {' or '.join(map(str, types))} is needed, got {t.dtype} {tuple(t.shape)}")
    rows, cols = t.shape
    if t.is_contiguous():
        return rows, cols, cols
    pitch, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} needs rows with unit inner stride")
    # a one-row view may carry any stride
    return rows, cols, pitch if rows > 1 else cols


def _out(out, dtype, M, N, index, like):
    """(out, its row pitch), made when None."""
    if out is None:
        if dtype not in _TYPES:
            raise ValueError(f"dtype: {_BF16} or {_F32} is needed, got {dtype}")
        return _new((M, N), dtype, like), N
    rows, cols, ld = _rows(out, "out", _TYPES)
    if rows != M or cols != N or out.get_device() != index:
        raise ValueError(f"out: shape {(M, N)} on cuda:{index} is needed, got {tuple(out.shape)} on {out.device}")
    return out, ld


def _word(faults, index):
    if faults.get_device() != index or faults.dtype is not torch.int32 or faults.numel() != 1:
        raise ValueError(f"faults: one int32 on cuda:{index} is needed")
    return faults.data_ptr()


def _codes(codes, scales, dims, what, index):
    """(shape of the codes, codes address, scales address) of a stored operand."""
    shape = codes.shape
    half = shape[-1] if shape else 0
    if len(shape) != dims or half & 15 or codes.dtype is not _U8 or not codes.is_contiguous():
        raise ValueError(f"{what}codes: contiguous {_U8} of {dims} dimensions, K a multiple of 32, is needed, got {codes.dtype} {tuple(shape)}")
    return shape, codes.data_ptr(), _dense(scales, what + "scales", _U8, (*shape[:-1], half >> 4), index)


def _acts(x, x_scales, half, index):
    """(kind, rows, x address, scales address, row pitch) of the activations."""
    if x.get_device() != index:
        raise ValueError(f"x is on {x.device}, the weight on cuda:{index}")
    if x_scales is not None:
        M = x.shape[0] if x.dim() else 0
        return _ACT_MXFP4, M, _dense(x, "x", _U8, (M, half), index), _dense(x_scales, "x_scales", _U8, (M, half >> 4), index), 2 * half
    M, K, ld = _rows(x, "x", _X_TYPES)
    if K != 2 * half:
        raise ValueError(f"x: rows of {2 * half} values are needed, got {K}")
    return _ACT_BF16, M, x.data_ptr(), None, ld


def mxfp4_quantize(x, *, faults=None, codes=None, scales=None):
    """Quantize x (BF16 or fp32, [M][K], rows may be strided) to MXFP4 on the device; returns
    (codes [M][K/2] u8, scales [M][K/32] u8). `faults`: a device int32 that receives
    FAULT_NONFINITE."""
    index = _device(x)
    M, K, ld = _rows(x, "x", _TYPES)
    if codes is None:
        codes = _new((M, K // 2), _U8, x)
        cp = codes.data_ptr()
    else:
        cp = _dense(codes, "codes", _U8, (M, K // 2), index)
    if scales is None:
        scales = _new((M, K // 32), _U8, x)
        sp = scales.data_ptr()
    else:
        sp = _dense(scales, "scales", _U8, (M, K // 32), index)
    _run((_lib or _load()).mxfp4_quantize, "mxfp4_quantize", index, _TYPES[x.dtype], x.data_ptr(), ld, M, K, cp, sp,
         None if faults is None else _word(faults, index))
    return codes, scales


def mxfp4_dequantize(codes, scales, *, dtype=_BF16, out=None):
    """The values of codes [M][K/2] u8 and scales [M][K/32] u8 as [M][K] of `dtype` (BF16 or
    fp32; `out`'s, when that is given)."""
    index = _device(codes)
    (M, half), cp, sp = _codes(codes, scales, 2, "", index)
    out, ld = _out(out, dtype, M, 2 * half, index, codes)
    _run((_lib or _load()).mxfp4_dequantize, "mxfp4_dequantize", index, cp, sp, M, 2 * half, _TYPES[out.dtype],
         out.data_ptr(), ld)
    return out


def mxfp4_linear(x, w_codes, w_scales, *, x_scales=None, out=None, out_dtype=_F32, check=False, faults=None):
    """y = x W^T for an MXFP4 weight (codes [N][K/2] u8, scales [N][K/32] u8). x is BF16
    [M][K] (W4A16; rows may be strided) or MXFP4 codes [M][K/2] with x_scales (W4A4). y is
    [M][N] of out_dtype (fp32 or BF16; `out`'s, when that is given). check=True scans the
    operands first and ORs FAULT_* bits into `faults` (a device int32 word, required then)."""
    index = _device(w_codes)
    (N, half), cp, sp = _codes(w_codes, w_scales, 2, "w_", index)
    act, M, xp, xsp, ldx = _acts(x, x_scales, half, index)
    out, ldy = _out(out, out_dtype, M, N, index, w_codes)
    _run((_lib or _load()).mxfp4_linear, "mxfp4_linear", index, act, xp, xsp, ldx, M, N, 2 * half, cp, sp,
         _TYPES[out.dtype], out.data_ptr(), ldy, F_CHECK if check else 0, None if faults is None else _word(faults, index))
    return out


def mxfp4_grouped_workspace_size(T: int, top_k: int, N: int, K: int, num_experts: int, out_mode: int) -> int:
    """Bytes of workspace that mxfp4_grouped_linear needs for these sizes."""
    n = ctypes.c_size_t(0)
    st = (_lib or _load()).mxfp4_grouped_linear(_ACT_BF16, None, None, K, 0, T, top_k, N, K, num_experts, None, None, None,
                                         None, out_mode, 0, None, None, None, ctypes.byref(n), 0, None, None)
    if st:
        _check(st, "mxfp4_grouped_linear (workspace query)")
    return n.value


def mxfp4_grouped_linear(x, w_codes, w_scales, topk_ids, *, topk_w=None, out_mode=OUT_ROUTES, rows_per_route=False,
                         x_scales=None, out=None, out_scales=None, out_dtype=None, workspace=None, faults=None,
                         reuse_grouping=False, check=False):
    """Expert-grouped MXFP4 linear. w_codes [E][N][K/2] u8, w_scales [E][N][K/32] u8, topk_ids
    [T][top_k] int32; x as in mxfp4_linear, one row per token (rows_per_route: per route).
    See include/mxfp4.h for the output forms. OUT_ROUTES and OUT_COMBINE write out_dtype
    (fp32 when None; `out`'s, when that is given), OUT_SWIGLU_BF16 BF16; OUT_SWIGLU_MXFP4
    returns (codes, scales) and takes them as out and out_scales. reuse_grouping
    (OUT_COMBINE with the workspace of the layer's earlier call on the same topk_ids) skips
    the route grouping."""
    index = _device(w_codes)
    (E, N, half), cp, sp = _codes(w_codes, w_scales, 3, "w_", index)
    shape = topk_ids.shape
    if len(shape) != 2:
        raise ValueError("topk_ids: [T][top_k] is needed")
    T, top_k = shape
    R = T * top_k
    ip = _dense(topk_ids, "topk_ids", torch.int32, shape, index)
    tp = None if topk_w is None else _dense(topk_w, "topk_w", _F32, shape, index)
    act, rows, xp, xsp, ldx = _acts(x, x_scales, half, index)
    if rows != (R if rows_per_route else T):
        raise ValueError(f"x: {R if rows_per_route else T} rows are needed, got {rows}")
    osp, y_type, kind = None, 0, _BF16
    if out_mode == OUT_SWIGLU_MXFP4:
        shape, kind = (R, N // 4), _U8
        if out_scales is None:
            out_scales = _new((R, N // 64), _U8, w_codes)
        osp = _dense(out_scales, "out_scales", _U8, (R, N // 64), index)
    else:
        if out_scales is not None:
            raise ValueError("out_scales: with OUT_SWIGLU_MXFP4 only")
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
        size = mxfp4_grouped_workspace_size(T, top_k, N, 2 * half, E, out_mode)
        workspace = torch.empty(size, dtype=_U8, device=w_codes.device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace: contiguous, on cuda:{index}, is needed")
    nbytes = ctypes.c_size_t(workspace.nbytes)
    _run((_lib or _load()).mxfp4_grouped_linear, "mxfp4_grouped_linear", index, act, xp, xsp, ldx,
         1 if rows_per_route else 0, T, top_k, N, 2 * half, E, cp, sp, ip, tp,
         out_mode | OUT_REUSE_GROUPING if reuse_grouping else out_mode, y_type, yp, osp, workspace.data_ptr(),
         ctypes.byref(nbytes), F_CHECK if check else 0, None if faults is None else _word(faults, index))
    return (out, out_scales) if out_mode == OUT_SWIGLU_MXFP4 else out
