// Device helpers of the FP8 kernels: E4M3 decode and encode, MFMA over a block of 128.
#pragma once

#include "fp8.h"
#include "mx_device.hpp"

namespace nvfp4 {

constexpr float kF8Top = 448.0f;  // E4M3's largest value

// MFMA over 128 k of E4M3 rows: lane l holds 32 codes of row l % 16 on either side, the same k on
// both; result C[4 * (l / 16) + r][l % 16]. (Constant zeros for the block scales make it the
// instruction without them.)
//
// The instruction sums less exactly than fp32. Of the products of eight consecutive k of a lane it
// drops what lies below 2^-13 of the largest one's power of two (measured; the sums of eights
// are added as in fp32; the older 16x16x32 form does the same), at most 7 * 2^-13 of that
// product. By the 2-norm that is 1.4e-5 of the results with unit normal activations and 2.6e-5 to
// 2.9e-5 with loud channels among them (one in 250, twenty times as large; K from 512 to 14336),
// with fp32 sums 5e-8 to 2e-7; rounding to BF16 is 1.7e-3. E4M3 activations are rounded by 2^-4. For
// results in fp32, and for SwiGLU's, codes are decoded to BF16, whose MFMA sums in fp32, at half
// the rate.
__device__ __forceinline__ f32x4 mfma_f8(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1, f32x4 c) {
  const i32x8 a = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
  const i32x8 b = {(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3], (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// 8 codes (two dwords, k ascending) -> 8 BF16, exact
__device__ __forceinline__ u32x4 f8_decode8(uint32_t lo, uint32_t hi) {
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, 0));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, 1));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, 0));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, 1));
  return r;
}

// 32 codes to BF16, eight k to a register group
__device__ __forceinline__ void f8_decode32(u32x4 a, u32x4 b, u32x4 (&f)[4]) {
  f[0] = f8_decode8(a[0], a[1]);
  f[1] = f8_decode8(a[2], a[3]);
  f[2] = f8_decode8(b[0], b[1]);
  f[3] = f8_decode8(b[2], b[3]);
}

// Four values of magnitude up to 448 -> their codes, nearest, ties to even (v_cvt_pk_fp8_f32)
__device__ __forceinline__ uint32_t f8_codes4(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}

// The scale of a block whose largest magnitude is amax (finite).
template <int RULE>
__device__ __forceinline__ float f8_scale(float amax) {
  const float s = amax / kF8Top;
  if (RULE == FP8_SCALE_F32) return s;
  const uint32_t u = __float_as_uint(s);
  if (u <= 1u) return s;
  // a subnormal s is an integer times 2^-149; 2^23 of those are the least normal number
  return __uint_as_float(u < 0x800000u ? 1u << (32 - __builtin_clz(u - 1)) : (u + 0x7FFFFFu) & 0xFF800000u);
}

// x / s for the encoder: +-0 where s is 0, and no more than 448
__device__ __forceinline__ float f8_ratio(float x, float s) {
  const float q = s == 0.0f ? __builtin_copysignf(0.0f, x) : x / s;
  return __builtin_fminf(__builtin_fmaxf(q, -kF8Top), kF8Top);
}

// Codes of n values of a block whose largest magnitude is amax and scale s. The correctly rounded
// quotients by one reciprocal: with r the rounded 1 / s, x * r is within 1.5 ulp of x / s, one
// correction by the remainder makes it a neighbour of x / s, and by Markstein's theorem the next
// rounds correctly (five operations a value, a division takes a dozen). Remainders stay
// representable wherever the quotient is more than half of E4M3's least, as long as s is not tiny.
// Such quotients are at most 448 rounded up, which the encoder rounds to 448.
template <int n>
__device__ __forceinline__ void f8_codes(const float* v, float amax, float s, uint32_t* codes) {
  float q[n];
  if (amax >= 0x1p-70f) {
    const float r = 1.0f / s;
#pragma unroll
    for (int i = 0; i < n; i++) {
      float c = v[i] * r;
      c = __builtin_fmaf(__builtin_fmaf(-c, s, v[i]), r, c);
      c = __builtin_fmaf(__builtin_fmaf(-c, s, v[i]), r, c);
      q[i] = __builtin_copysignf(c, v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < n; i++) q[i] = f8_ratio(v[i], s);
  }
#pragma unroll
  for (int i = 0; i < n / 4; i++) codes[i] = f8_codes4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
}

// n BF16 pairs as values
template <int n>
__device__ __forceinline__ void f8_values(const uint32_t* pairs, float* v) {
#pragma unroll
  for (int i = 0; i < n; i++) {
    v[2 * i] = __uint_as_float(pairs[i] << 16);
    v[2 * i + 1] = __uint_as_float(pairs[i] & 0xFFFF0000u);
  }
}

}  // namespace nvfp4
