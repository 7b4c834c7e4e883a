// Internal launch interface of the FP8 operators and the router, between their C ABI
// (f8_api.hip) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8.h"
#include "mx_kernels.hpp"

namespace nvfp4 {

constexpr int kF8Block = 128;  // k of a block of scales, and weight rows

// Beside FP8_ACT_*: FP8 activations whose products are summed in fp32 throughout (see mfma_f8),
// for fp32 results and SwiGLU's
constexpr int kF8Exact = 2;

// One product x W^T, dense or grouped by expert. The members of the grouped form are those of
// MxArgs.
struct F8Args {
  // activations: BF16 [rows][ldx], or codes [rows][ldx] with scales [rows][KB]
  const void* x;
  const float* x_scales;
  int64_t ldx;
  // weight (grouped: expert 0; expert e lies e * N * K codes and e * NB * KB scales on)
  const uint8_t* w_codes;
  const float* w_scales;
  int64_t M, N, K;
  // output: rows of ldy values of y_type; SwiGLU to FP8 also writes y_scales
  void* y;
  float* y_scales;
  int64_t ldy;
  int32_t y_type;
  int32_t swiglu;  // 0, or FP8_OUT_SWIGLU_BF16 / FP8_OUT_SWIGLU_FP8
  const int32_t* ids;
  int32_t num_experts;
  uint32_t* faults;
  int32_t zero_dropped;
  int32_t tile_rows;
  int64_t max_tiles;
  int32_t max_slots;
  const int32_t* tiles;
  const int32_t* n_tiles;
  const int32_t* slots;
  const int32_t* offsets;
  const int32_t* sorted;
  const int32_t* route_expert;
  int64_t R;
  int64_t x_rows;
  int32_t rows_per_token;
  int32_t top_k;
};

hipError_t launch_f8_quantize(int x_type, const void* x, int64_t ldx, int64_t M, int64_t K,
                              int block_rows, int scale_rule, uint8_t* codes, float* scales,
                              uint32_t* faults, hipStream_t stream);
hipError_t launch_f8_dequantize(const uint8_t* codes, const float* scales, int64_t M, int64_t K,
                                int block_rows, int y_type, void* y, int64_t ldy,
                                hipStream_t stream);

// LDS tiles (f8_tiled.hip): dense, or the grouping's list of tiles of tile_rows routes
hipError_t launch_f8_tiled(const F8Args& a, int act_kind, hipStream_t stream);
// the weight streamed (f8_stream.hip) for about `rows` activation rows per weight (dense: M of
// them), the grouped form by ids or by slots
hipError_t launch_f8_stream(const F8Args& a, int act_kind, int64_t rows, hipStream_t stream);

// check mode: scales that are not finite set NVFP4_FAULT_NAN_SCALE, NaN codes of rows
// [rows][ld], K each (multiples of 16), NVFP4_FAULT_NONFINITE
hipError_t launch_f8_check_scales(const float* scales, int64_t n, uint32_t* faults,
                                  hipStream_t stream);
hipError_t launch_f8_check_codes(const uint8_t* codes, int64_t ld, int64_t rows, int64_t K,
                                 uint32_t* faults, hipStream_t stream);

struct RouteArgs {
  const void* logits;
  const float* bias;  // NULL: none
  int64_t ld, T;
  int32_t logits_type, num_experts, top_k, scoring, num_groups, top_groups, group_score, renormalize;
  float scale;
  int32_t* topk_ids;
  float* topk_w;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t stream);

}  // namespace nvfp4
