// Device helpers of the MXFP4 kernels: block scales, decode to BF16, scaled MFMA.
#pragma once

#include "device.hpp"

namespace nvfp4 {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kE8M0Nan = 0xFFu;

// floor(log2(amax)) - 2 as an E8M0 byte, clamped below at 0, for a finite amax >= 0 given by
// its bits: fp32's exponent field less two (2 = the exponent of 6, E2M1's largest value).
// Subnormal and zero amax have field 0 and clamp to 0, as their exponents do.
__device__ __forceinline__ uint32_t e8m0_of_amax(uint32_t bits) {
  const int32_t e = (int32_t)(bits >> 23) - 2;
  return e < 0 ? 0u : (uint32_t)e;
}

// E8M0 byte -> the float whose exponent field it is (the scale operand of gfx950's scaled
// conversions, which look at nothing else)
__device__ __forceinline__ float e8m0_operand(uint32_t s) { return __uint_as_float(s << 23); }

// Scaled MFMA over 128 k of MXFP4 rows: lane l holds codes of row l % 16 at k = 32 * (l / 16)
// + [0, 32) (16 bytes) and, in byte SEL of its scale register, that block's E8M0 scale;
// result C[4 * (l / 16) + r][l % 16].
template <int SA = 0, int SB = 0>
__device__ __forceinline__ f32x4 mfma_mx(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, SA, (int)sa, SB,
                                                          (int)sb);
}

// 8 codes (one dword, k ascending from the low nibble) times a power of two -> 8 BF16
__device__ __forceinline__ u32x4 mx_decode8(uint32_t codes, float scale) {
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  return r;
}

// f32 -> BF16 bits, round to nearest even; NaN stays NaN
__device__ __forceinline__ uint32_t f32_to_bf16_any(float v) {
  return v != v ? 0x7FC0u : f32_to_bf16_rne(v);
}

}  // namespace nvfp4
