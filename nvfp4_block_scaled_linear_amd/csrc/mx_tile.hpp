// How the tiled MXFP4 and FP8 kernels bring their results out.
#pragma once

#include "mx_device.hpp"
#include "mx_routes.hpp"

namespace nvfp4 {

// LDS that store_tile takes of each wave: a row tile of fp32
template <class S>
__host__ __device__ constexpr int store_bytes() {
  return 16 * S::TW * 16 * 4;
}

// A wave's results to rows of y, ES bytes a value; cols columns are left from n on. In
// registers, 16 consecutive lanes hold 16 rows, so a store from there would touch 64 cache
// lines; each tile of 16 rows goes through LDS and out along the rows, 16 bytes a lane, or a
// value a lane where rows are not aligned or end inside (1001 columns of fp32 stored from
// registers took 10 of 20 us). Piece q of row r lies at slot q ^ f(r), as in the operands.
template <class S, bool GROUPED, int ES, class A>
__device__ __forceinline__ void store_tile(const A& a, uint8_t* lds, f32x4 (&acc)[S::TW][S::TX],
                                           int wx, int64_t m0, int slot0, int64_t rows_m, int64_t n,
                                           int64_t cols, bool vec) {
  constexpr int RB = S::TW * 16 * ES, PIECES = RB / 16, ROWS = 64 / PIECES;  // rows of a store
  static_assert(PIECES >= 8 && PIECES <= 64, "");
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const auto swizzle = [](int r) { return PIECES == 8 ? (r >> 1) & 7 : r & 15; };
  const bool whole = vec && cols >= S::TW * 16;
#pragma unroll
  for (int x = 0; x < S::TX; x++) {
    const int r0 = (wx * S::TX + x) * 16;
    if (r0 >= rows_m) break;
    const int route = GROUPED && r0 + c < rows_m ? route_at(a, slot0 + r0 + c) : 0;
#pragma unroll
    for (int w = 0; w < S::TW; w += ES == 4 ? 1 : 2) {  // one 16-byte piece
      // tiles w .. of group w / 4 hold columns 64 * (w / 4) + 16 * g + 4 * (w % 4) and on
      const int piece = (64 * (w / 4) + 16 * g + 4 * (w % 4)) * ES / 16;
      u32x4 v;
      if constexpr (ES == 4) {
        v = __builtin_bit_cast(u32x4, acc[w][x]);
      } else {
        const f32x4 p = acc[w][x], q = acc[w + 1][x];
        v = u32x4{bf16_pair(p[0], p[1]), bf16_pair(p[2], p[3]), bf16_pair(q[0], q[1]), bf16_pair(q[2], q[3])};
      }
      *reinterpret_cast<u32x4*>(lds + c * RB + ((piece ^ swizzle(c)) << 4)) = v;
    }
    if (whole) {
#pragma unroll
      for (int i = 0; i < 16 / ROWS; i++) {
        const int r = i * ROWS + lane / PIECES, q = lane % PIECES;
        const u32x4 v = *reinterpret_cast<const u32x4*>(lds + r * RB + ((q ^ swizzle(r)) << 4));
        const int64_t row = GROUPED ? __shfl(route, r, 64) : m0 + r0 + r;
        if (r0 + r < rows_m)
          *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(a.y) + (row * a.ldy + n) * ES + 16 * q) = v;
      }
      continue;
    }
    for (int r = 0; r < 16 && r0 + r < rows_m; r++) {
      const int64_t row = GROUPED ? __builtin_amdgcn_readlane(route, r) : m0 + r0 + r;
#pragma unroll
      for (int k = 0; k < S::TW / 4; k++) {
        const int e = 64 * k + lane;  // column of the wave's
        const uint8_t* p = lds + r * RB + (((e * ES >> 4) ^ swizzle(r)) << 4) + (e * ES & 15);
        if (e >= cols) continue;
        if constexpr (ES == 4)
          static_cast<uint32_t*>(a.y)[row * a.ldy + n + e] = *reinterpret_cast<const uint32_t*>(p);
        else
          static_cast<uint16_t*>(a.y)[row * a.ldy + n + e] = *reinterpret_cast<const uint16_t*>(p);
      }
    }
  }
}

}  // namespace nvfp4
