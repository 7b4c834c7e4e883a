// Route grouping of the MXFP4 grouped product for up to kMxGroupRoutes routes: one workgroup,
// one pass over the routes.
//
// Each kept route takes its place among its expert's with an LDS counter (the order within an
// expert is left open: a route's row depends on its own activation row and its expert alone),
// one scan over the experts gives the offsets and where slot records and tiles go, and the
// routes are put down. The time is launch and memory latency: 999 routes over 24 experts take
// about 5 us, where ranking every route against all earlier ones takes 19.
#include "mx_device.hpp"
#include "mx_kernels.hpp"
#include "mx_routes.hpp"

namespace nvfp4 {
namespace {

constexpr int kThreads = 1024;
constexpr int kPer = kMxGroupRoutes / kThreads;  // routes of a thread

__global__ __launch_bounds__(kThreads) void mx_group(const int32_t* ids, int R, int top_k, int E,
                                                     RouteWorkspace ws, uint32_t* faults) {
  extern __shared__ int32_t sh[];
  int32_t* id = sh;          // [R]
  int32_t* cnt = sh + R;     // [E] routes, then first place in `sorted`
  int32_t* slot = cnt + E;   // [E] slot record of an active expert
  __shared__ int32_t wave_sum[3][kThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int r = tid; r < R; r += kThreads) id[r] = ids[r];
  for (int e = tid; e < E; e += kThreads) cnt[e] = 0;
  __syncthreads();
  int32_t rank[kPer];
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int r = i * kThreads + tid;
    rank[i] = -1;
    if (r >= R) continue;
    if (keeps_route(id, r, top_k, E)) {
      rank[i] = atomicAdd(&cnt[id[r]], 1);
      ws.route_expert[r] = id[r];
      continue;
    }
    ws.route_expert[r] = -1;
    if (faults) atomicOr(faults, (uint32_t)NVFP4_FAULT_BAD_ROUTE);
  }
  __syncthreads();
  int32_t run[3] = {0, 0, 0};  // routes, active experts and tiles of the experts so far
  for (int e0 = 0; e0 < E; e0 += kThreads) {
    const int e = e0 + tid;
    const int32_t c = e < E ? cnt[e] : 0;
    const int32_t rest = c > ws.main_rows ? c - ws.main_rows : 0;
    const int32_t own[3] = {c, c > 0, (rest + ws.tile_rows - 1) / ws.tile_rows};
    int32_t at[3];
#pragma unroll
    for (int k = 0; k < 3; k++) {
      int32_t x = own[k];
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int32_t y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
      }
      if (lane == 63) wave_sum[k][wave] = x;
      at[k] = x - own[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; k++) {
      at[k] += run[k];
      for (int w = 0; w < kThreads / 64; w++) {
        const int32_t s = wave_sum[k][w];
        at[k] += w < wave ? s : 0;
        run[k] += s;
      }
    }
    __syncthreads();  // the sums are used again
    if (e >= E) continue;
    ws.offsets[e] = at[0];
    cnt[e] = at[0];
    if (c > 0) {
      ws.active[at[1]] = e;
      slot[e] = at[1];
      *reinterpret_cast<int4*>(ws.slots + kSlotInts * at[1]) =
          make_int4(e, at[0], at[0] + c, c < kSlotRoutes ? c : kSlotRoutes);
    }
    for (int i = 0; i < own[2]; i++) {
      ws.tiles[2 * (at[2] + i)] = e;
      ws.tiles[2 * (at[2] + i) + 1] = at[0] + (c - rest) + i * ws.tile_rows;
    }
  }
  for (int s = run[1] + tid; s < ws.max_slots; s += kThreads) ws.slots[kSlotInts * s] = -1;
  if (tid == 0) {
    ws.offsets[E] = run[0];
    *ws.n_active = run[1];
    *ws.n_tiles = run[2];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    if (rank[i] < 0) continue;
    const int r = i * kThreads + tid, e = id[r];
    ws.sorted[cnt[e] + rank[i]] = r;
    if (rank[i] < kSlotRoutes) ws.slots[kSlotInts * slot[e] + 4 + rank[i]] = r;
  }
}

}  // namespace

hipError_t launch_mx_group(const int32_t* topk_ids, int64_t R, int top_k, int E,
                           const RouteWorkspace& ws, uint32_t* faults, hipStream_t stream) {
  hipLaunchKernelGGL(mx_group, dim3(1), dim3(kThreads), sizeof(int32_t) * (size_t)(R + 2 * E),
                     stream, topk_ids, (int)R, top_k, E, ws, faults);
  return hipGetLastError();
}

}  // namespace nvfp4
