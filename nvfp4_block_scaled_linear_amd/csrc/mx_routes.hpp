// What the grouped MXFP4 kernels share about routes.
#pragma once

#include "mx_device.hpp"
#include "mx_kernels.hpp"

namespace nvfp4 {

// whether topk_ids[r] is an expert that its token has not named before
__device__ __forceinline__ bool keeps_route(const int32_t* ids, int64_t r, int top_k, int E) {
  const int32_t e = ids[r];
  bool ok = e >= 0 && e < E;
  for (int64_t q = r - r % top_k; q < r; q++) ok = ok && ids[q] != e;
  return ok;
}

// A call that reuses a grouping is given a workspace, and one that holds no grouping, or that of
// other sizes, must not make it leave its buffers: what is read there is an expert, a place or a
// route only as far as the call has them. Rows of x need no such care, their loads have a range: a
// route is looked at where its row is stored, not on the way to the first loads.
__device__ __forceinline__ int32_t in_experts(const MxArgs& a, int32_t e) {
  const uint32_t last = (uint32_t)a.num_experts - 1;
  return (int32_t)((uint32_t)e < last ? (uint32_t)e : last);
}

// how many of the places [first, end) of `sorted`, `most` at most, there are
__device__ __forceinline__ int run_length(const MxArgs& a, int32_t first, int32_t end, int most) {
  const int32_t R = (int32_t)a.R;
  end = end < R ? end : R;
  if (first < 0 || first >= end) return 0;
  return end - first < most ? end - first : most;
}

__device__ __forceinline__ int32_t in_routes(const MxArgs& a, int32_t route) {
  const uint32_t last = (uint32_t)a.R - 1;
  return (int32_t)((uint32_t)route < last ? (uint32_t)route : last);
}

__device__ __forceinline__ int32_t route_at(const MxArgs& a, int32_t place) {
  return in_routes(a, a.sorted[place]);
}

// One wave writes zeros over the output row of a dropped route.
template <int SWIGLU>
__device__ __forceinline__ void clear_route(const MxArgs& a, int64_t r) {
  const int lane = threadIdx.x & 63;
  const int64_t bytes = SWIGLU == 0 ? a.N * (a.y_type == MXFP4_F32 ? 4 : 2)
                        : SWIGLU == MXFP4_OUT_SWIGLU_BF16 ? a.N : a.N >> 2;
  uint8_t* const row = static_cast<uint8_t*>(a.y) + r * bytes;
  if ((((uintptr_t)a.y | (uintptr_t)bytes) & 3) == 0)
    for (int64_t b = 4 * lane; b < bytes; b += 256) *reinterpret_cast<uint32_t*>(row + b) = 0u;
  else
    for (int64_t b = 2 * lane; b < bytes; b += 128) *reinterpret_cast<uint16_t*>(row + b) = 0;
  if (SWIGLU == MXFP4_OUT_SWIGLU_MXFP4)
    for (int64_t b = lane; b < a.N >> 6; b += 64) a.y_scales[r * (a.N >> 6) + b] = 0;
}

// The output rows of dropped routes become zeros, each by one wave, shared out over the launch:
// batches are padded with routes that no expert takes. With half of 512 x top-4 routes like
// that and 2048 columns of fp32, K = 2048 and 32 experts, the product takes 41 us with BF16
// activations and 24 with MXFP4 ones (43 and 26 where all are routed); with a lane of the
// grouping's one workgroup to a row it took 1114.
//
// After a grouping, a wave looks at as many routes as make them go round.
template <int SWIGLU>
__device__ __forceinline__ void clear_dropped(const MxArgs& a) {
  if (!a.zero_dropped) return;
  const int lane = threadIdx.x & 63, W = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t waves = (int64_t)gridDim.x * W;
  int64_t per = (a.R + waves - 1) / waves;
  per = per < 64 ? per : 64;
  for (int64_t r0 = ((int64_t)blockIdx.x * W + wave) * per; r0 < a.R; r0 += waves * per) {
    uint64_t drop = __ballot(lane < per && r0 + lane < a.R && a.route_expert[r0 + lane] < 0);
    for (; drop; drop &= drop - 1) clear_route<SWIGLU>(a, r0 + __builtin_ctzll(drop));
  }
}

// Without a grouping, a wave looks at one route and those of its token before it (top_k <= 64),
// and also reports the dropped ones.
template <int SWIGLU>
__device__ __forceinline__ void drop_routes(const MxArgs& a) {
  if (!a.zero_dropped && !a.faults) return;
  const int lane = threadIdx.x & 63, W = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int R = (int)a.R, waves = (int)gridDim.x * W;
  for (int r = (int)blockIdx.x * W + wave; r < R; r += waves) {
    const int j = r % a.top_k;
    const int32_t id = lane <= j ? a.ids[r - j + lane] : -1;
    const int32_t e = __builtin_amdgcn_readlane(id, j);
    if (e >= 0 && e < a.num_experts && __builtin_popcountll(__ballot(id == e)) == 1) continue;
    if (a.faults && lane == 0) atomicOr(a.faults, (uint32_t)NVFP4_FAULT_BAD_ROUTE);
    if (a.zero_dropped) clear_route<SWIGLU>(a, r);
  }
}

}  // namespace nvfp4
