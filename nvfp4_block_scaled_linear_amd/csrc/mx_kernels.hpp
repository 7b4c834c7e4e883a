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
  // grouped form (NULL tiles for dense): tiles of tile_rows routes of one expert
  int32_t tile_rows;
  int64_t x_rows;          // rows of x
  const int32_t* tiles;    // [n_tiles][2] (expert, first slot in sorted)
  const int32_t* n_tiles;  // [1]
  const int32_t* slots;    // [max_slots] slot records (RouteWorkspace::slots)
  const int32_t* offsets;  // [E+1]
  const int32_t* sorted;   // route ids grouped by expert
  const int32_t* route_expert;  // [R] expert of a route, -1 when dropped
  int64_t R;
  int32_t rows_per_token;  // x row of route r: r / top_k (1) or r (0)
  int32_t top_k;
};

hipError_t launch_mx_quantize(int x_type, const void* x, int64_t ldx, int64_t M, int64_t K,
                              uint8_t* codes, uint8_t* scales, uint32_t* faults,
                              hipStream_t stream);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K,
                                int y_type, void* y, int64_t ldy, hipStream_t stream);

// routes of one tile of the grouped form's tile list, for R routes over `active` experts
int mx_tile_rows(int64_t R, int64_t active);
// the kernel for LDS tiles (mx_tiled.hip), and whether its 32-bit offsets reach the operands
bool mx_tiled_takes(const MxArgs& a, int act_kind);
hipError_t launch_mx_tiled(const MxArgs& a, int act_kind, int64_t max_tiles, hipStream_t stream);
// the kernel that streams the weight (mx_stream.hip) for about `rows` activation rows per
// weight (dense: M of them, at most 64)
bool mx_stream_takes(const MxArgs& a, int act_kind);
hipError_t launch_mx_stream(const MxArgs& a, int act_kind, int64_t rows, int64_t max_slots,
                            hipStream_t stream);
// max_tiles and max_slots bound the tile list and the slot records of the grouped form (0: dense)
hipError_t launch_mx_product(const MxArgs& a, int act_kind, int64_t max_tiles, int64_t max_slots,
                             hipStream_t stream);

// y[t] = sum over t's kept routes in ascending expert id of topk_w * rows[route]
hipError_t launch_mx_combine(const float* rows, const int32_t* route_expert, const float* topk_w,
                             int64_t T, int top_k, int64_t N, int y_type, void* y,
                             hipStream_t stream);
// check mode: scale bytes 0xFF in [0, bytes) set NVFP4_FAULT_NAN_SCALE
hipError_t launch_mx_check_scales(const uint8_t* scales, int64_t bytes, uint32_t* faults,
                                  hipStream_t stream);

}  // namespace nvfp4
