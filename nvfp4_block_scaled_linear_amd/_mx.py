"""The MXFP4 operators of libnvfp4.so (include/mxfp4.h) over torch tensors: quantization and
its way back, the linear layer and its expert-grouped form. As in _binding.py, nothing is
computed here. Each call runs on the current stream of its tensors' device."""
from __future__ import annotations

import ctypes

import torch

from . import _binding
from ._binding import F_CHECK, OUT_COMBINE, OUT_REUSE_GROUPING, OUT_ROUTES, OUT_SWIGLU_BF16, _check

OUT_SWIGLU_MXFP4 = 3
MX_EXPORTS = ("mxfp4_quantize", "mxfp4_dequantize", "mxfp4_linear", "mxfp4_grouped_linear")

_ACT_BF16, _ACT_MXFP4 = 0, 1
_TYPES = {torch.bfloat16: 0, torch.float32: 1}
_lib = None


def _load():
    global _lib
    if _lib is None:
        lib = _binding.load_library()
        vp, i64, i32, u32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32
        lib.mxfp4_quantize.argtypes = [i32, vp, i64, i64, i64, vp, vp, vp, vp]
        lib.mxfp4_dequantize.argtypes = [vp, vp, i64, i64, i32, vp, i64, vp]
        lib.mxfp4_linear.argtypes = [i32, vp, vp, i64, i64, i64, i64, vp, vp, i32, vp, i64, u32, vp, vp]
        lib.mxfp4_grouped_linear.argtypes = [i32, vp, vp, i64, i32, i64, i32, i64, i64, i32, vp, vp, vp, vp,
                                             i32, i32, vp, vp, vp, ctypes.POINTER(ctypes.c_size_t), u32, vp, vp]
        for name in MX_EXPORTS:
            getattr(lib, name).restype = i32
        _lib = lib
    return _lib


def _run(device, name, *args):
    """Calls the entry point `name` on `device`'s current stream."""
    fn = getattr(_load(), name)
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            st = fn(*args, torch.cuda.current_stream().cuda_stream)
    else:
        st = fn(*args, torch.cuda.current_stream().cuda_stream)
    if st != 0:
        _check(st, name)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _dense(t, name, dtype, shape, device):
    """A contiguous device tensor of this type and shape."""
    _need(t.is_cuda, "libnvfp4 takes device tensors only")
    _need(t.dtype == dtype and t.shape == shape, f"{name}: {dtype} of shape {tuple(shape)} is needed, got {t.dtype} {tuple(t.shape)}")
    _need(t.is_contiguous(), f"{name} must be contiguous")
    _need(t.device == device, f"{name} is on {t.device}, the call on {device}")


def _rows(t, name, types):
    """A device matrix of one of `types` with unit inner stride; its row pitch."""
    _need(t.is_cuda, "libnvfp4 takes device tensors only")
    _need(t.dim() == 2 and t.dtype in types, f"{name}: a matrix of {' or '.join(map(str, types))} is needed, got {t.dtype} {tuple(t.shape)}")
    _need(t.stride(1) == 1 or t.shape[1] <= 1, f"{name} needs rows with unit inner stride")
    # a one-row view may carry any stride
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _word(faults, device):
    if faults is None:
        return None
    _need(faults.is_cuda and faults.device == device and faults.dtype == torch.int32 and faults.numel() == 1,
          f"faults: one int32 on {device} is needed")
    return faults.data_ptr()


def _weight(w_codes, w_scales, dims):
    _need(w_codes.dim() == dims, f"w_codes: {dims} dimensions are needed, got {w_codes.dim()}")
    device = w_codes.device
    _dense(w_codes, "w_codes", torch.uint8, w_codes.shape, device)
    _need(w_codes.shape[-1] % 16 == 0, "w_codes: K must be a multiple of 32")
    _dense(w_scales, "w_scales", torch.uint8, (*w_codes.shape[:-1], w_codes.shape[-1] // 16), device)
    return device


def _acts(x, x_scales, K, device):
    """(kind, x address, scales address, row pitch) of the activations."""
    _need(x.device == device, f"x is on {x.device}, the weight on {device}")
    if x_scales is None:
        ld = _rows(x, "x", (torch.bfloat16,))
        _need(x.shape[1] == K, f"x: rows of {K} values are needed, got {x.shape[1]}")
        return _ACT_BF16, x.data_ptr(), None, ld
    _dense(x, "x", torch.uint8, (x.shape[0], K // 2), device)
    _dense(x_scales, "x_scales", torch.uint8, (x.shape[0], K // 32), device)
    return _ACT_MXFP4, x.data_ptr(), x_scales.data_ptr(), K


def mxfp4_quantize(x, *, faults=None, codes=None, scales=None):
    """Quantize x (BF16 or fp32, [M][K], rows may be strided) to MXFP4 on the device; returns
    (codes [M][K/2] u8, scales [M][K/32] u8). `faults`: a device int32 that receives
    FAULT_NONFINITE."""
    ld = _rows(x, "x", (torch.bfloat16, torch.float32))
    M, K = x.shape
    dev = x.device
    if codes is None:
        codes = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    else:
        _dense(codes, "codes", torch.uint8, (M, K // 2), dev)
    if scales is None:
        scales = torch.empty((M, K // 32), dtype=torch.uint8, device=dev)
    else:
        _dense(scales, "scales", torch.uint8, (M, K // 32), dev)
    _run(dev, "mxfp4_quantize", _TYPES[x.dtype], x.data_ptr(), ld, M, K, codes.data_ptr(), scales.data_ptr(),
         _word(faults, dev))
    return codes, scales


def mxfp4_dequantize(codes, scales, *, dtype=torch.bfloat16, out=None):
    """The values of codes [M][K/2] u8 and scales [M][K/32] u8 as [M][K] of `dtype` (BF16 or
    fp32; `out`'s, when that is given)."""
    dev = _weight(codes, scales, 2)
    M, K = codes.shape[0], 2 * codes.shape[1]
    if out is None:
        _need(dtype in _TYPES, f"dtype: {' or '.join(map(str, _TYPES))}, got {dtype}")
        out = torch.empty((M, K), dtype=dtype, device=dev)
    ld = _rows(out, "out", tuple(_TYPES))
    _need(out.shape == (M, K) and out.device == dev, f"out: shape {(M, K)} on {dev} is needed")
    _run(dev, "mxfp4_dequantize", codes.data_ptr(), scales.data_ptr(), M, K, _TYPES[out.dtype], out.data_ptr(), ld)
    return out


def mxfp4_linear(x, w_codes, w_scales, *, x_scales=None, out=None, out_dtype=torch.float32, check=False, faults=None):
    """y = x W^T for an MXFP4 weight (codes [N][K/2] u8, scales [N][K/32] u8). x is BF16
    [M][K] (W4A16; rows may be strided) or MXFP4 codes [M][K/2] with x_scales (W4A4). y is
    [M][N] of out_dtype (fp32 or BF16; `out`'s, when that is given). check=True scans the
    operands first and ORs FAULT_* bits into `faults` (a device int32 word, required then)."""
    dev = _weight(w_codes, w_scales, 2)
    N, K = w_codes.shape[0], 2 * w_codes.shape[1]
    act, xp, xsp, ldx = _acts(x, x_scales, K, dev)
    M = x.shape[0]
    if out is None:
        _need(out_dtype in _TYPES, f"out_dtype: {' or '.join(map(str, _TYPES))}, got {out_dtype}")
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
        ldy = N
    else:
        ldy = _rows(out, "out", tuple(_TYPES))
        _need(out.shape == (M, N) and out.device == dev, f"out: shape {(M, N)} on {dev} is needed")
    _run(dev, "mxfp4_linear", act, xp, xsp, ldx, M, N, K, w_codes.data_ptr(), w_scales.data_ptr(),
         _TYPES[out.dtype], out.data_ptr(), ldy, F_CHECK if check else 0, _word(faults, dev))
    return out


def mxfp4_grouped_workspace_size(T: int, top_k: int, N: int, K: int, num_experts: int, out_mode: int) -> int:
    """Bytes of workspace that mxfp4_grouped_linear needs for these sizes."""
    n = ctypes.c_size_t(0)
    st = _load().mxfp4_grouped_linear(_ACT_BF16, None, None, K, 0, T, top_k, N, K, num_experts, None, None, None,
                                      None, out_mode, 0, None, None, None, ctypes.byref(n), 0, None, None)
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
    dev = _weight(w_codes, w_scales, 3)
    E, N, half = w_codes.shape
    K = 2 * half
    _need(topk_ids.dim() == 2, "topk_ids: [T][top_k] is needed")
    T, top_k = topk_ids.shape
    R = T * top_k
    _dense(topk_ids, "topk_ids", torch.int32, topk_ids.shape, dev)
    if topk_w is not None:
        _dense(topk_w, "topk_w", torch.float32, topk_ids.shape, dev)
    _need(not reuse_grouping or workspace is not None, "reuse_grouping needs the workspace that holds the grouping")
    act, xp, xsp, ldx = _acts(x, x_scales, K, dev)
    _need(x.shape[0] == (R if rows_per_route else T), f"x: {R if rows_per_route else T} rows are needed, got {x.shape[0]}")
    to_mx = out_mode == OUT_SWIGLU_MXFP4
    shape = {OUT_ROUTES: (R, N), OUT_SWIGLU_BF16: (R, N // 2), OUT_COMBINE: (T, N), OUT_SWIGLU_MXFP4: (R, N // 4)}.get(out_mode)
    _need(shape is not None, f"out_mode: one of the OUT_* forms is needed, got {out_mode}")
    if to_mx:
        y_type, kind = 0, torch.uint8
        if out_scales is None:
            out_scales = torch.empty((R, N // 64), dtype=torch.uint8, device=dev)
        else:
            _dense(out_scales, "out_scales", torch.uint8, (R, N // 64), dev)
    else:
        _need(out_scales is None, "out_scales: with OUT_SWIGLU_MXFP4 only")
        kind = out_dtype if out_dtype is not None else out.dtype if out is not None else (
            torch.bfloat16 if out_mode == OUT_SWIGLU_BF16 else torch.float32)
        _need(kind in _TYPES, f"out_dtype: {' or '.join(map(str, _TYPES))}, got {kind}")
        y_type = _TYPES[kind]
    if out is None:
        out = torch.empty(shape, dtype=kind, device=dev)
    else:
        _dense(out, "out", kind, shape, dev)
    if workspace is None:
        workspace = torch.empty(mxfp4_grouped_workspace_size(T, top_k, N, K, E, out_mode), dtype=torch.uint8, device=dev)
    else:
        _need(workspace.is_cuda and workspace.device == dev and workspace.is_contiguous(), f"workspace: contiguous, on {dev}, is needed")
    nbytes = ctypes.c_size_t(workspace.numel() * workspace.element_size())
    _run(dev, "mxfp4_grouped_linear", act, xp, xsp, ldx, 1 if rows_per_route else 0, T, top_k, N, K, E,
         w_codes.data_ptr(), w_scales.data_ptr(), topk_ids.data_ptr(), None if topk_w is None else topk_w.data_ptr(),
         out_mode | (OUT_REUSE_GROUPING if reuse_grouping else 0), y_type, out.data_ptr(),
         out_scales.data_ptr() if to_mx else None, workspace.data_ptr(), ctypes.byref(nbytes),
         F_CHECK if check else 0, _word(faults, dev))
    return (out, out_scales) if to_mx else out
