// Host side of the grouped MXFP4 and FP8 calls: how a call goes about its routes, and the part
// of its workspace that holds their grouping.
#pragma once

#include "mx_kernels.hpp"

namespace nvfp4 {

// How a grouped call goes about R = T * top_k routes. It depends on nothing else, so that
// both calls of a layer agree on the workspace's grouping.
//  - scan: few routes; each workgroup looks for its expert in topk_ids and nothing is grouped.
//  - slots: less than `tiled_routes` routes per active expert on average; the weight is
//    streamed for up to 16 routes, experts with more have the rest in the list of tiles.
//  - tiles of up to 64 or 128 routes of an expert for more (128 from `tile128_routes` on).
struct RoutePlan {
  bool scan, slots;
  int tile_rows, main_rows;
  int64_t max_tiles;
};

inline RoutePlan plan_routes(int64_t T, int top_k, int E, int64_t tiled_routes, int64_t tile128_routes) {
  const int64_t R = T * top_k, active = R < E ? R : E;
  if (R < tiled_routes * active) {
    // an expert has at most T routes; past its first 16, c routes make at most c / 16 tiles
    if (R <= kScanRoutes) return {true, false, 0, 0, 0};
    return {false, true, kMxSlotRoutes, kMxSlotRoutes, T > kMxSlotRoutes ? R / kMxSlotRoutes : 0};
  }
  const int rows = R < tile128_routes * active ? 64 : 128;
  return {false, false, rows, 0, R / rows + active};  // one partial tile per expert
}

// Grouped-call workspace: 256-byte aligned regions, those of the grouping first and the same
// in every output form; then `row_bytes` bytes of each route's row.
struct RouteLayout {
  size_t offsets, active, n_active, route_expert, sorted, slots, tiles, n_tiles, chunks, rows, total;
};

inline RouteLayout layout_routes(const RoutePlan& p, int64_t T, int top_k, int E, size_t row_bytes) {
  RouteLayout L{};
  const int64_t R = T * top_k, active = R < E ? R : E;
  size_t o = 256;  // never empty
  const auto region = [&o](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) & ~(size_t)255;
    return at;
  };
  const auto ints = [&region](int64_t n) { return region(4 * (size_t)n); };
  if (!p.scan) {
    L.offsets = ints(E + 1);
    L.active = ints(E);
    L.n_active = ints(1);
    L.route_expert = ints(R);
    L.sorted = ints(R);
    L.slots = ints(kSlotInts * active);
    L.tiles = ints(2 * p.max_tiles);
    L.n_tiles = ints(1);
    L.chunks = ints(route_chunk_ints(T, top_k, E));
  }
  L.rows = region((size_t)R * row_bytes);
  L.total = o;
  return L;
}

// The routes' part of a grouped call's arguments (MxArgs, F8Args); the routes are grouped unless
// the plan does without or the workspace holds the grouping already.
template <class A>
hipError_t prepare_routes(A& a, const RoutePlan& plan, const RouteLayout& L, void* workspace,
                          const int32_t* topk_ids, int64_t T, bool reuse, uint32_t* faults,
                          hipStream_t s) {
  if (plan.scan) {
    a.ids = topk_ids;
    a.faults = reuse ? nullptr : faults;  // reported by the earlier call
    return hipSuccess;
  }
  char* const base = static_cast<char*>(workspace);
  const auto ints = [base](size_t at) { return reinterpret_cast<int32_t*>(base + at); };
  RouteWorkspace ws{};
  ws.offsets = ints(L.offsets);
  ws.active = ints(L.active);
  ws.n_active = ints(L.n_active);
  ws.route_expert = ints(L.route_expert);
  ws.sorted = ints(L.sorted);
  ws.slots = ints(L.slots);
  ws.max_slots = (int32_t)(a.R < a.num_experts ? a.R : a.num_experts);
  ws.tiles = ints(L.tiles);
  ws.n_tiles = ints(L.n_tiles);
  ws.chunk_counts = ints(L.chunks);
  ws.tile_rows = plan.tile_rows;
  ws.main_rows = plan.main_rows;
  a.tile_rows = plan.tile_rows; a.max_tiles = plan.max_tiles; a.max_slots = ws.max_slots;
  a.tiles = ws.tiles; a.n_tiles = ws.n_tiles; a.offsets = ws.offsets; a.sorted = ws.sorted;
  a.slots = ws.slots; a.route_expert = ws.route_expert;
  if (reuse) return hipSuccess;
  return a.R <= kMxGroupRoutes
             ? launch_mx_group(topk_ids, a.R, a.top_k, a.num_experts, ws, faults, s)
             : launch_route_sort(topk_ids, T, a.top_k, a.num_experts, ws, faults, nullptr, 0, s);
}

}  // namespace nvfp4
