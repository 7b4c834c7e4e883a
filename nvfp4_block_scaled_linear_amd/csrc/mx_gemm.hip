// MXFP4 products on the matrix cores: y = x W^T, dense or grouped by expert, with BF16 or
// MXFP4 activations.
//
// The weight's rows are the MFMA's A rows and the activation rows its columns, so a lane's
// four results are four consecutive columns of one output row. A wave takes 32 weight rows
// (SwiGLU: 32 gate rows and the 32 up rows that belong to them) and 16 activation rows, and
// walks K in steps of 128: lane l holds the 32 k of block l / 16 of the step, one 16-byte
// load of codes and one scale byte per row.
//  - MXFP4 activations: one scaled MFMA over the 128 k per 16 weight rows, both operands as
//    they are stored.
//  - BF16 activations: the codes are decoded with the block's scale to BF16 (two values per
//    conversion, exact) and the step is four BF16 MFMAs, the j-th of them over k =
//    32 * (l / 16) + 8j + [0, 8) of lane l.
#include "mx_device.hpp"
#include "mx_kernels.hpp"

namespace nvfp4 {
namespace {

constexpr int kTileRows = 16;  // activation rows of a tile
constexpr int kTileCols = 32;  // output columns of a tile

__device__ __forceinline__ u32x4 load16(const uint8_t* p, bool ok) {
  return ok ? *reinterpret_cast<const u32x4*>(p) : u32x4{0u, 0u, 0u, 0u};
}

// four consecutive columns n, n+1, .. of output row `row`
__device__ __forceinline__ void store4(const MxArgs& a, int64_t row, int64_t n, int64_t N,
                                       const float v[4]) {
#pragma unroll
  for (int r = 0; r < 4; r++) {
    if (n + r >= N) break;
    if (a.y_type == MXFP4_F32) {
      static_cast<float*>(a.y)[row * a.ldy + n + r] = v[r];
    } else {
      static_cast<uint16_t*>(a.y)[row * a.ldy + n + r] = (uint16_t)f32_to_bf16_any(v[r]);
    }
  }
}

// SwiGLU to MXFP4: the scales of the routes that the grouping dropped (it clears their codes),
// shared out over the launch's tiles: routes n * tile + [0, n), tiles past the list included
__device__ __forceinline__ void clear_dropped_scales(const MxArgs& a, int64_t tile, int n) {
  const int64_t bytes = a.N >> 6;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int64_t r = tile * n + i;
    if (r >= a.R || a.route_expert[r] >= 0) continue;
    for (int64_t b = 0; b < bytes; b++) a.y_scales[r * bytes + b] = 0;
  }
}

template <int ACT, bool GROUPED, int SWIGLU>
__global__ __launch_bounds__(64) void mx_tile(MxArgs a) {
  constexpr int NT = SWIGLU ? 4 : 2;  // 16-row weight tiles: gate 0, 1 and up 2, 3
  const int lane = threadIdx.x, c = lane & 15, g = lane >> 4;
  const int64_t N = a.N, K = a.K, half = N >> 1;
  const int64_t cols = SWIGLU ? half : N;
  const int64_t nbn = (cols + kTileCols - 1) / kTileCols;
  const int64_t tile = blockIdx.x / nbn;  // of kTileRows rows; grouped: a part of a list tile
  const int64_t n0 = (blockIdx.x % nbn) * kTileCols;
  const uint8_t* wc = a.w_codes;
  const uint8_t* ws = a.w_scales;
  int64_t xrow, yrow;
  bool row_ok;
  if (GROUPED) {
    if (SWIGLU == MXFP4_OUT_SWIGLU_MXFP4 && n0 == 0) clear_dropped_scales(a, tile, kTileRows);
    const int parts = a.tile_rows / kTileRows;
    const int64_t lt = tile / parts;
    if (lt >= *a.n_tiles) return;
    const int e = a.tiles[2 * lt];
    const int first = a.tiles[2 * lt + 1] + (int)(tile % parts) * kTileRows;
    if (first >= a.offsets[e + 1]) return;
    const int slot = first + c;
    row_ok = slot < a.offsets[e + 1];
    yrow = row_ok ? a.sorted[slot] : 0;
    xrow = a.rows_per_token ? yrow / a.top_k : yrow;
    wc += (int64_t)e * N * (K >> 1);
    ws += (int64_t)e * N * (K >> 5);
  } else {
    xrow = yrow = tile * kTileRows + c;
    row_ok = xrow < a.M;
  }
  int64_t wrow[NT];
  bool wok[NT];
#pragma unroll
  for (int t = 0; t < NT; t++) {
    const int64_t n = n0 + 16 * (t & 1) + c;
    wok[t] = n < cols;
    wrow[t] = n + (t >= 2 ? half : 0);
  }
  f32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; t++) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int64_t nb = K >> 5;
  for (int64_t b0 = 0; b0 < nb; b0 += 4) {
    const int64_t b = b0 + g;
    const bool in = b < nb;
    u32x4 xc[ACT == MXFP4_ACT_BF16 ? 4 : 1];
    uint32_t xs = 0u;
    if (ACT == MXFP4_ACT_BF16) {
      const uint8_t* p = static_cast<const uint8_t*>(a.x) + (xrow * a.ldx + 32 * b) * 2;
#pragma unroll
      for (int j = 0; j < 4; j++) xc[j] = load16(p + 16 * j, in && row_ok);
    } else {
      xc[0] = load16(static_cast<const uint8_t*>(a.x) + xrow * (K >> 1) + 16 * b, in && row_ok);
      xs = in && row_ok ? a.x_scales[xrow * nb + b] : 0u;
    }
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const bool ok = in && wok[t];
      const u32x4 w = load16(wc + wrow[t] * (K >> 1) + 16 * b, ok);
      const uint32_t s = ok ? ws[wrow[t] * nb + b] : 0u;
      if (ACT == MXFP4_ACT_BF16) {
        const float sc = e8m0_operand(s);
#pragma unroll
        for (int j = 0; j < 4; j++) acc[t] = mfma16(mx_decode8(w[j], sc), xc[j], acc[t]);
      } else {
        acc[t] = mfma_mx(w, xc[0], acc[t], s, xs);
      }
    }
  }

  if (!SWIGLU) {
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const float v[4] = {acc[t][0], acc[t][1], acc[t][2], acc[t][3]};
      if (row_ok) store4(a, yrow, n0 + 16 * t + 4 * g, N, v);
    }
    return;
  }
  uint32_t bits[2][4];  // BF16 silu(gate) * up of this lane's columns
#pragma unroll
  for (int t = 0; t < 2; t++)
#pragma unroll
    for (int r = 0; r < 4; r++) bits[t][r] = f32_to_bf16_any(silu(acc[t][r]) * acc[t + NT / 2][r]);
  if (SWIGLU == MXFP4_OUT_SWIGLU_BF16) {
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
      for (int r = 0; r < 4; r++) {
        const int64_t n = n0 + 16 * t + 4 * g + r;
        if (row_ok && n < half) static_cast<uint16_t*>(a.y)[yrow * half + n] = (uint16_t)bits[t][r];
      }
    return;
  }
  // to MXFP4: the tile's 32 columns are one block, spread over the four lanes of a row
  uint32_t amax = 0u;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint32_t m = (bits[i >> 2][i & 3] & 0x7FFFu) << 16;
    amax = amax > m ? amax : m;
  }
  uint32_t o = __shfl_xor(amax, 16, 64);
  amax = amax > o ? amax : o;
  o = __shfl_xor(amax, 32, 64);
  amax = amax > o ? amax : o;
  const uint32_t s = e8m0_of_amax(amax);
  const bool bad = amax >= 0x7F800000u;
  if (!row_ok) return;
#pragma unroll
  for (int t = 0; t < 2; t++) {
    float q[4];
#pragma unroll
    for (int r = 0; r < 4; r++)
      q[r] = __builtin_ldexpf(bf16_bits_to_f32(bits[t][r]), 127 - (int)s);
    const uint32_t code = e2m1_rne2<1>(e2m1_rne2<0>(0u, q[0], q[1]), q[2], q[3]);
    *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a.y) + yrow * (half >> 1) +
                                 ((n0 + 16 * t + 4 * g) >> 1)) = bad ? 0 : (uint16_t)code;
  }
  if (g == 0) a.y_scales[yrow * (half >> 5) + (n0 >> 5)] = (uint8_t)(bad ? kE8M0Nan : s);
}

}  // namespace

int mx_tile_rows(int64_t R, int64_t active) { return R >= 64 * active ? 128 : kTileRows; }

hipError_t launch_mx_product(const MxArgs& a, int act_kind, int64_t max_tiles, int64_t max_slots,
                             hipStream_t stream) {
  if (a.tiles ? a.tile_rows > kTileRows : a.M > 64) {
    if (mx_tiled_takes(a, act_kind)) return launch_mx_tiled(a, act_kind, max_tiles, stream);
  } else if (mx_stream_takes(a, act_kind)) {
    const int64_t rows = a.tiles ? (a.R + max_slots - 1) / max_slots : a.M;
    return launch_mx_stream(a, act_kind, rows, max_slots, stream);
  }
  const int64_t cols = a.swiglu ? a.N >> 1 : a.N;
  const int64_t gx = a.tiles ? max_tiles * (a.tile_rows / kTileRows) : (a.M + kTileRows - 1) / kTileRows;
  const int64_t groups = gx * ((cols + kTileCols - 1) / kTileCols);
  if (groups * 64 > (int64_t)UINT32_MAX) return hipErrorInvalidConfiguration;
  const bool bf = act_kind == MXFP4_ACT_BF16;
  auto k = !a.tiles ? (bf ? mx_tile<0, false, 0> : mx_tile<1, false, 0>)
           : a.swiglu == 0 ? (bf ? mx_tile<0, true, 0> : mx_tile<1, true, 0>)
           : a.swiglu == MXFP4_OUT_SWIGLU_BF16
               ? (bf ? mx_tile<0, true, MXFP4_OUT_SWIGLU_BF16> : mx_tile<1, true, MXFP4_OUT_SWIGLU_BF16>)
               : (bf ? mx_tile<0, true, MXFP4_OUT_SWIGLU_MXFP4> : mx_tile<1, true, MXFP4_OUT_SWIGLU_MXFP4>);
  hipLaunchKernelGGL(k, dim3((uint32_t)groups), dim3(64), 0, stream, a);
  return hipGetLastError();
}

}  // namespace nvfp4
