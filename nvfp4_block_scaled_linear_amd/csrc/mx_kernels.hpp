// Internal launch interface of the MXFP4 operators, between their C ABI (mx_api.hip) and the
// kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.hpp"
#include "mxfp4.h"

namespace nvfp4 {

// One product x W^T, dense or grouped by expert.
struct MxArgs {
  // activations: BF16 [rows][ldx], or codes [rows][K/2] with scales [rows][K/32]
  const void* x;
  const uint8_t* x_scales;
  int64_t ldx;
  // weight (grouped: expert 0; expert e lies e * N * K/2 bytes and e * N * K/32 scales on)
  const uint8_t* w_codes;
  const uint8_t* w_scales;
  int64_t M, N, K;
  // output: rows of ldy values of y_type; SwiGLU to MXFP4 also writes y_scales
  void* y;
  uint8_t* y_scales;
  int64_t ldy;
  int32_t y_type;
  int32_t swiglu;  // 0, or MXFP4_OUT_SWIGLU_BF16 / MXFP4_OUT_SWIGLU_MXFP4
  // grouped form (NULL topk_ids and tiles for dense)
  const int32_t* ids;      // topk_ids, where the kernel finds the routes itself (else NULL)
  int32_t num_experts;
  uint32_t* faults;        // with ids
  int32_t zero_dropped;    // rows of dropped routes are written (as zeros)
  // otherwise the grouping: slot records of the experts, tiles of routes
  int32_t tile_rows;       // most routes of a list tile (16 by slots, 64 or 128)
  int64_t max_tiles;       // bounds of the lists
  int32_t max_slots;
  const int32_t* tiles;    // [n_tiles][2] (expert, first place in sorted)
  const int32_t* n_tiles;  // [1]
  const int32_t* slots;    // [max_slots] slot records (RouteWorkspace::slots)
  const int32_t* offsets;  // [E+1]
  const int32_t* sorted;   // route ids grouped by expert
  const int32_t* route_expert;  // [R] expert of a route, -1 when dropped
  int64_t R;
  int64_t x_rows;          // rows of x
  int32_t rows_per_token;  // x row of route r: r / top_k (1) or r (0)
  int32_t top_k;
};

hipError_t launch_mx_quantize(int x_type, const void* x, int64_t ldx, int64_t M, int64_t K,
                              uint8_t* codes, uint8_t* scales, uint32_t* faults,
                              hipStream_t stream);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K,
                                int y_type, void* y, int64_t ldy, hipStream_t stream);

// LDS tiles (mx_tiled.hip): dense, or the grouping's list of tiles of tile_rows routes
hipError_t launch_mx_tiled(const MxArgs& a, int act_kind, hipStream_t stream);
// the weight streamed (mx_stream.hip) for about `rows` activation rows per weight (dense: M of
// them), the grouped form by ids or by slots
hipError_t launch_mx_stream(const MxArgs& a, int act_kind, int64_t rows, hipStream_t stream);
// most routes in all that the form by ids takes (four per lane), and the routes of a slot or a
// list tile of the other
constexpr int kScanRoutes = 256;
constexpr int kMxSlotRoutes = 16;

// groups up to kMxGroupRoutes routes; what launch_route_sort writes
constexpr int kMxGroupRoutes = 4096;
hipError_t launch_mx_group(const int32_t* topk_ids, int64_t R, int top_k, int E,
                           const RouteWorkspace& ws, uint32_t* faults, hipStream_t stream);

// y[t] = sum over t's kept routes in ascending expert id of topk_w * rows[route], N columns of
// rows of `pitch` and ldy values
hipError_t launch_mx_combine(const float* rows, int64_t pitch, const int32_t* topk_ids,
                             const float* topk_w, int64_t T, int top_k, int E, int64_t N,
                             int y_type, void* y, int64_t ldy, hipStream_t stream);

// check mode: scale bytes 0xFF in [0, bytes) set NVFP4_FAULT_NAN_SCALE
hipError_t launch_mx_check_scales(const uint8_t* scales, int64_t bytes, uint32_t* faults,
                                  hipStream_t stream);

}  // namespace nvfp4
