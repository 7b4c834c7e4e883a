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

// two f32 -> BF16 pair, round to nearest even, NaN stays NaN
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// largest magnitude (f32 bits) of n BF16 pairs
template <int n>
__device__ __forceinline__ uint32_t amax_pairs(const uint32_t* h) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < n; i++) {
    const uint32_t lo = (h[i] & 0x7FFFu) << 16, hi = h[i] & 0x7FFF0000u;
    m = m > lo ? m : lo;
    m = m > hi ? m : hi;
  }
  return m;
}

// two BF16 pairs -> their four codes (16 bits) at scale byte s
__device__ __forceinline__ uint32_t codes_of_pairs(uint32_t a, uint32_t b, uint32_t s) {
  const int up = 127 - (int)s;
  const float q0 = __builtin_ldexpf(__uint_as_float(a << 16), up);
  const float q1 = __builtin_ldexpf(__uint_as_float(a & 0xFFFF0000u), up);
  const float q2 = __builtin_ldexpf(__uint_as_float(b << 16), up);
  const float q3 = __builtin_ldexpf(__uint_as_float(b & 0xFFFF0000u), up);
  return e2m1_rne2<1>(e2m1_rne2<0>(0u, q0, q1), q2, q3);
}

// ---------------------------------------------------------------------------------------
// Loads from memory straight into LDS, through a buffer descriptor: lanes out of its range
// write zeros and touch no memory. They are instructions without outputs, so the compiler
// neither tracks nor waits for them: a counted wait (wait_loads) stands before the reads.
// ---------------------------------------------------------------------------------------
constexpr uint32_t kOutOfRange = 0x80000000u;  // an offset past every descriptor's range

__device__ __forceinline__ u32x4 lds_load_rsrc(const void* base, int64_t bytes) {
  const uint64_t p = (uint64_t)(uintptr_t)base;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)p);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32) & 0xFFFFu);
  const uint32_t n = __builtin_amdgcn_readfirstlane((uint32_t)(bytes > 0x7FFFFFFF ? 0x7FFFFFFF : bytes));
  return u32x4{lo, hi, n, 0x00020000u};
}

// BYTES (16, 4 or 1) bytes per lane from offset `off`; lane l's go to lds + l * max(BYTES, 4)
// (a byte as a dword). lds is the same in all lanes.
template <int BYTES>
__device__ __forceinline__ void lds_load(u32x4 rsrc, uint32_t off, uint32_t lds) {
  static_assert(BYTES == 16 || BYTES == 4 || BYTES == 1, "");
  lds = __builtin_amdgcn_readfirstlane(lds);
  if (BYTES == 16)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :: "v"(off), "s"(rsrc), "s"(lds) : "memory", "m0");
  else if (BYTES == 4)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 :: "v"(off), "s"(rsrc), "s"(lds) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_ubyte %0, %1, 0 offen lds"
                 :: "v"(off), "s"(rsrc), "s"(lds) : "memory", "m0");
}

// all but this wave's latest N loads are done, and its LDS reads
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// this wave's LDS reads are done (what they read may be overwritten)
__device__ __forceinline__ void wait_lds_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// all but the latest N loads and the LDS reads are done, and the workgroup's other waves have come as far
template <int N>
__device__ __forceinline__ void wait_loads_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds_address(void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)p;
}

}  // namespace nvfp4
