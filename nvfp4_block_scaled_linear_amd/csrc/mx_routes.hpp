// What the grouped MXFP4 and FP8 kernels share about routes. A is the kernels' argument struct
// (MxArgs, F8Args), whose members of the grouped form have the same names.
#pragma once

#include "fp8.h"
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
template <class A>
__device__ __forceinline__ int32_t in_experts(const A& a, int32_t e) {
  const uint32_t last = (uint32_t)a.num_experts - 1;
  return (int32_t)((uint32_t)e < last ? (uint32_t)e : last);
}

// how many of the places [first, end) of `sorted`, `most` at most, there are
template <class A>
__device__ __forceinline__ int run_length(const A& a, int32_t first, int32_t end, int most) {
  const int32_t R = (int32_t)a.R;
  end = end < R ? end : R;
  if (first < 0 || first >= end) return 0;
  return end - first < most ? end - first : most;
}

template <class A>
__device__ __forceinline__ int32_t in_routes(const A& a, int32_t route) {
  const uint32_t last = (uint32_t)a.R - 1;
  return (int32_t)((uint32_t)route < last ? (uint32_t)route : last);
}

template <class A>
__device__ __forceinline__ int32_t route_at(const A& a, int32_t place) {
  return in_routes(a, a.sorted[place]);
}

// One wave writes zeros over the output row of a dropped route.
template <int SWIGLU, class A>
__device__ __forceinline__ void clear_route(const A& a, int64_t r) {
  const int lane = threadIdx.x & 63;
  const int64_t bytes = SWIGLU == 0 ? a.N * (a.y_type == MXFP4_F32 ? 4 : 2)
                        : SWIGLU == MXFP4_OUT_SWIGLU_BF16 ? a.N : SWIGLU == MXFP4_OUT_SWIGLU_MXFP4 ? a.N >> 2 : a.N >> 1;
  uint8_t* const row = static_cast<uint8_t*>(a.y) + r * bytes;
  if ((((uintptr_t)a.y | (uintptr_t)bytes) & 3) == 0)
    for (int64_t b = 4 * lane; b < bytes; b += 256) *reinterpret_cast<uint32_t*>(row + b) = 0u;
  else
    for (int64_t b = 2 * lane; b < bytes; b += 128) *reinterpret_cast<uint16_t*>(row + b) = 0;
  constexpr int shift = SWIGLU == MXFP4_OUT_SWIGLU_MXFP4 ? 6 : 8;  // columns of a block, gate and up
  if (SWIGLU == MXFP4_OUT_SWIGLU_MXFP4 || SWIGLU == FP8_OUT_SWIGLU_FP8)
    for (int64_t b = lane; b < a.N >> shift; b += 64) a.y_scales[r * (a.N >> shift) + b] = 0;
}

// The output rows of dropped routes become zeros, each by one wave, shared out over the launch:
// batches are padded with routes that no expert takes. With half of 512 x top-4 routes like
// that and 2048 columns of fp32, K = 2048 and 32 experts, the product takes 41 us with BF16
// activations and 24 with MXFP4 ones (43 and 26 where all are routed); with a lane of the
// grouping's one workgroup to a row it took 1114.
//
// After a grouping, a wave looks at as many routes as make them go round.
template <int SWIGLU, class A>
__device__ __forceinline__ void clear_dropped(const A& a) {
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
template <int SWIGLU, class A>
__device__ __forceinline__ void drop_routes(const A& a) {
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

// How a grouped workgroup finds its expert and the routes of it
enum Mode {
  kDense,
  kByExpert,  // few routes in all: the workgroup looks for its routes in topk_ids
  kBySlot     // from the grouping: a slot record's first kMxSlotRoutes routes, or a list tile
};

// kByExpert: the workgroup groups of R routes. A group takes at most kMxSlotRoutes routes of an
// expert, as a slot does, so that an expert that many tokens pick is spread over groups. With
// fewer routes than experts the groups are the routes, and those whose place among their expert's
// is a multiple of kMxSlotRoutes have work. Otherwise they are the experts' first routes, and as
// many groups behind them as there can be runs of further ones (an expert has at most a route of
// each token; past its first kMxSlotRoutes, c routes make at most c / kMxSlotRoutes runs).
// A layer of 128 experts, 2048 / 768, BF16, takes 46 us for 256 tokens that all pick one expert, 75
// for 64 tokens x top-4 that share one; in one workgroup a column block these were 276 and 119.
// Tokens that pick evenly take what they took (one token 14.9 us, 16 46.5).
__host__ __device__ inline int64_t scan_groups(int64_t R, int top_k, int E) {
  return R < E ? R : E + (R / top_k > kMxSlotRoutes ? R / kMxSlotRoutes : 0);
}

// The expert and the first place of the run-th of the runs of routes that go past the experts'
// first ones; false when there are fewer. By all of a workgroup, with R >= E and E ints of LDS.
// (Routes that repeat an id within a token are counted: a run may turn out empty.)
__device__ __forceinline__ bool further_run(const int32_t* ids, int R, int E, int run, int32_t* cnt,
                                            int* expert, int* begin) {
  const int lane = threadIdx.x & 63;
  for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  for (int r = threadIdx.x; r < R; r += blockDim.x) {
    const int32_t e = ids[r];
    if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  bool found = false;
  int before = 0;  // runs of the experts so far
#pragma unroll
  for (int i = 0; i < kScanRoutes / 64; i++) {
    const int e = 64 * i + lane, c = e < E ? cnt[e] : 0;
    const int own = c > 0 ? (c - 1) / kMxSlotRoutes : 0;
    int upto = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d, 64);
      if (lane >= d) upto += v;
    }
    const uint64_t hit = __ballot(run < before + upto && run >= before + upto - own);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      *expert = 64 * i + l;
      *begin = kMxSlotRoutes * (1 + run - (before + __builtin_amdgcn_readlane(upto - own, l)));
      found = true;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  __syncthreads();  // the counters' LDS is used again
  return found;
}

// The expert of workgroup group `group`, the bits of the routes 64 * i + lane that it keeps (those
// that hold it and are not a repeat of it within their token; top_k <= 64: the token starts in
// this group of 64 or the last), and the places [*begin, *end) among them that are the group's;
// returns whether there are any.
__device__ __forceinline__ bool scan_routes(const int32_t* ids, int R, int top_k, int E, int group,
                                            int32_t* lds, int* expert, int* begin, int* end,
                                            uint64_t (&kept)[kScanRoutes / 64]) {
  const int lane = threadIdx.x & 63;
  int e = group;
  *begin = 0;
  int32_t id[kScanRoutes / 64];
#pragma unroll
  for (int i = 0; i < kScanRoutes / 64; i++) id[i] = 64 * i + lane < R ? ids[64 * i + lane] : -1;
  if (__builtin_expect(R >= E && group >= E, 0) && !further_run(ids, R, E, group - E, lds, &e, begin)) return false;
  if (R < E) {
#pragma unroll
    for (int i = 0; i < kScanRoutes / 64; i++)
      if (i == group / 64) e = __builtin_amdgcn_readlane(id[i], group % 64);
    if (e < 0 || e >= E) return false;
  }
  *expert = e;
  uint64_t last = 0u;
  int count = 0, held = 0;  // routes kept, and with repeats
#pragma unroll
  for (int i = 0; i < kScanRoutes / 64; i++) {
    const uint64_t m = __ballot(id[i] == e);
    held += __builtin_popcountll(m);
    kept[i] = m;
    if (__builtin_popcountll(m) + (last != 0u) > 1) {  // there may be repeats
      const int before = (64 * i + lane) % top_k;      // routes of the token before this one
      // bit 63: the route before this one, bit 62 the one before that, ...
      const uint64_t window = (lane ? m << (64 - lane) : 0u) | last >> lane;
      const bool repeat = before && (window >> (64 - before)) != 0u;
      kept[i] = __ballot(id[i] == e && !repeat);
    }
    last = m;
    count += __builtin_popcountll(kept[i]);
  }
  if (R < E && held > 1) {  // this route's place, if it is kept (of one route there is no question)
    bool mine = false;
#pragma unroll
    for (int i = 0; i < kScanRoutes / 64; i++) {
      const uint64_t below = i < group / 64 ? ~0ull : i == group / 64 ? (1ull << group % 64) - 1 : 0ull;
      *begin += __builtin_popcountll(kept[i] & below);
      mine = mine || (i == group / 64 && (kept[i] >> group % 64 & 1));
    }
    if (!mine || *begin % kMxSlotRoutes != 0) return false;
  }
  *end = count - *begin < kMxSlotRoutes ? count : *begin + kMxSlotRoutes;
  return *begin < *end;
}

}  // namespace nvfp4
