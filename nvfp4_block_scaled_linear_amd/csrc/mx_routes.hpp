// What the grouped MXFP4 kernels share about routes.
#pragma once

#include "mx_device.hpp"
#include "mx_kernels.hpp"

namespace nvfp4 {

// SwiGLU to MXFP4, after the grouping, which clears the codes of the routes it drops: their
// scales, shared out over the launch.
__device__ __forceinline__ void clear_dropped_scales(const MxArgs& a) {
  const int64_t bytes = a.N >> 6, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < a.R; r += step)
    if (a.route_expert[r] < 0)
      for (int64_t b = 0; b < bytes; b++) a.y_scales[r * bytes + b] = 0;
}

// whether topk_ids[r] is an expert that its token has not named before
__device__ __forceinline__ bool keeps_route(const int32_t* ids, int64_t r, int top_k, int E) {
  const int32_t e = ids[r];
  bool ok = e >= 0 && e < E;
  for (int64_t q = r - r % top_k; q < r; q++) ok = ok && ids[q] != e;
  return ok;
}

// Without a grouping: reports the dropped routes and clears their rows (one workgroup; the
// rows of a combine are only read where a route is kept).
template <int SWIGLU>
__device__ __forceinline__ void drop_routes(const MxArgs& a) {
  const int64_t bytes = SWIGLU == 0 ? a.N * (a.y_type == MXFP4_F32 ? 4 : 2)
                        : SWIGLU == MXFP4_OUT_SWIGLU_BF16 ? a.N : a.N >> 2;
  for (int64_t r = threadIdx.x; r < a.R; r += blockDim.x) {
    if (keeps_route(a.ids, r, a.top_k, a.num_experts)) continue;
    if (a.faults) atomicOr(a.faults, (uint32_t)NVFP4_FAULT_BAD_ROUTE);
    uint16_t* row = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a.y) + r * bytes);
    for (int64_t b = 0; b < bytes >> 1; b++) row[b] = 0;
    if (SWIGLU == MXFP4_OUT_SWIGLU_MXFP4)
      for (int64_t b = 0; b < a.N >> 6; b++) a.y_scales[r * (a.N >> 6) + b] = 0;
  }
}

}  // namespace nvfp4
