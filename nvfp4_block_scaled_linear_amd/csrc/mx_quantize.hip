// MXFP4 quantizer and its way back (rules in mxfp4.h). Both are bound by memory: 2 or 4 bytes
// of a value on one side, 17/32 on the other, and a few VALU operations in between.
//
// A quad of lanes takes a block of 32 values, eight per lane (16 bytes of BF16), so that the
// block's largest value is two exchanges inside the quad and a lane's eight codes are one
// dword; a wave reads 1 KiB of BF16 and writes 256 bytes of codes and 16 scale bytes in order.
// 2048 x 14336 in BF16, 59 and 16 MB, take 16.4 us one way and 12.6 the other (4.5 and 5.9 TB/s,
// partly out of the caches), in fp32, 117 and 16 MB, 27.9 and 30.3; 16 x 4096, 2.2 and 2.0 us in
// either type, are launch latency.
#include "mx_device.hpp"
#include "mx_kernels.hpp"

#pragma clang fp contract(off)

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

template <int T>
__device__ __forceinline__ void load8(const void* x, int64_t off, float v[8]) {
  if (T == MXFP4_BF16) {
    const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + off);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  } else {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(x) + off);
    const u32x4 a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  }
}

// Eight values of a block and the quad's largest magnitude (bits) -> codes and scale byte.
// A NaN or Inf anywhere in the block makes the largest magnitude's exponent field 255.
__device__ __forceinline__ uint32_t quantize8(const float v[8], uint32_t amax, uint32_t* scale) {
  const uint32_t s = e8m0_of_amax(amax);
  const int up = 127 - (int)s;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; i++) q[i] = __builtin_ldexpf(v[i], up);
  uint32_t c = e2m1_rne2<0>(0u, q[0], q[1]);
  c = e2m1_rne2<1>(c, q[2], q[3]);
  c = e2m1_rne2<2>(c, q[4], q[5]);
  c = e2m1_rne2<3>(c, q[6], q[7]);
  const bool bad = amax >= 0x7F800000u;
  *scale = bad ? kE8M0Nan : s;
  return bad ? 0u : c;
}

// Threads of a workgroup: 2^shift side by side along a row, the rest down the rows.
template <int T>
__global__ __launch_bounds__(kThreads) void mx_quantize_rows(const void* x, int64_t ldx, int64_t M,
                                                             int64_t K, int shift, uint8_t* codes,
                                                             uint8_t* scales, uint32_t* faults) {
  const int64_t row = (int64_t)blockIdx.x * (kThreads >> shift) + (threadIdx.x >> shift);
  if (row >= M) return;
  const int64_t pieces = K >> 3;  // of eight values; a multiple of 4, so quads stay whole
  bool bad = false;
  for (int64_t p = ((int64_t)blockIdx.y << shift) + (threadIdx.x & ((1 << shift) - 1)); p < pieces;
       p += (int64_t)gridDim.y << shift) {
    float v[8];
    load8<T>(x, row * ldx + 8 * p, v);
    uint32_t amax = 0u;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint32_t m = __float_as_uint(v[i]) & 0x7FFFFFFFu;
      amax = amax > m ? amax : m;
    }
    uint32_t o = __shfl_xor(amax, 1, 4);
    amax = amax > o ? amax : o;
    o = __shfl_xor(amax, 2, 4);
    amax = amax > o ? amax : o;
    uint32_t s;
    const uint32_t c = quantize8(v, amax, &s);
    bad = bad || s == kE8M0Nan;
    *reinterpret_cast<uint32_t*>(codes + row * (K >> 1) + 4 * p) = c;
    if ((p & 3) == 0) scales[row * (K >> 5) + (p >> 2)] = (uint8_t)s;
  }
  if (bad && faults) atomicOr(faults, (uint32_t)NVFP4_FAULT_NONFINITE);
}

// value of a code (as f32) times 2^(s - 127); exact unless it overflows
__device__ __forceinline__ float value_of(float e2m1, uint32_t s) {
  return s == kE8M0Nan ? __uint_as_float(0x7FC00000u) : __builtin_ldexpf(e2m1, (int)s - 127);
}

template <int T>
__global__ __launch_bounds__(kThreads) void mx_dequantize_rows(const uint8_t* codes,
                                                               const uint8_t* scales, int64_t M,
                                                               int64_t K, int shift, void* y,
                                                               int64_t ldy) {
  const int64_t row = (int64_t)blockIdx.x * (kThreads >> shift) + (threadIdx.x >> shift);
  if (row >= M) return;
  const int64_t pieces = K >> 3;
  for (int64_t p = ((int64_t)blockIdx.y << shift) + (threadIdx.x & ((1 << shift) - 1)); p < pieces;
       p += (int64_t)gridDim.y << shift) {
    const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + row * (K >> 1) + 4 * p);
    const uint32_t s = scales[row * (K >> 5) + (p >> 2)];
    f32x2 w[4];
    w[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
    w[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    w[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
    w[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = __float_as_uint(value_of(w[i >> 1][i & 1], s));
    if (T == MXFP4_BF16) {
      u32x4 o;  // at most two significant bits: the high halves are exact
#pragma unroll
      for (int i = 0; i < 4; i++) o[i] = (v[2 * i] >> 16) | (v[2 * i + 1] & 0xFFFF0000u);
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(y) + row * ldy + 8 * p) = o;
    } else {
      u32x4* d = reinterpret_cast<u32x4*>(static_cast<float*>(y) + row * ldy + 8 * p);
      d[0] = u32x4{v[0], v[1], v[2], v[3]};
      d[1] = u32x4{v[4], v[5], v[6], v[7]};
    }
  }
}

// threads along a row (a power of two, at least a quad) and the launch grid
struct RowShape {
  int shift;
  dim3 grid;
};

RowShape row_shape(int64_t M, int64_t K) {
  const int64_t pieces = K >> 3;
  int shift = 2;
  while (shift < 8 && ((int64_t)1 << shift) < pieces) shift++;
  const int64_t gx = (M + (kThreads >> shift) - 1) / (kThreads >> shift);
  int64_t gy = (pieces + ((int64_t)1 << shift) - 1) >> shift;
  if (gy > 1024) gy = 1024;
  return {shift, dim3((uint32_t)gx, (uint32_t)gy)};
}

__global__ __launch_bounds__(kThreads) void mx_scan_scales(const uint8_t* p, int64_t n,
                                                           uint32_t* faults) {
  const int64_t nthr = (int64_t)gridDim.x * kThreads;
  bool hit = false;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += nthr)
    hit = hit || p[i] == kE8M0Nan;
  if (hit) atomicOr(faults, (uint32_t)NVFP4_FAULT_NAN_SCALE);
}

}  // namespace

hipError_t launch_mx_quantize(int x_type, const void* x, int64_t ldx, int64_t M, int64_t K,
                              uint8_t* codes, uint8_t* scales, uint32_t* faults,
                              hipStream_t stream) {
  const RowShape r = row_shape(M, K);
  auto k = x_type == MXFP4_BF16 ? mx_quantize_rows<MXFP4_BF16> : mx_quantize_rows<MXFP4_F32>;
  hipLaunchKernelGGL(k, r.grid, dim3(kThreads), 0, stream, x, ldx, M, K, r.shift, codes, scales,
                     faults);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K,
                                int y_type, void* y, int64_t ldy, hipStream_t stream) {
  const RowShape r = row_shape(M, K);
  auto k = y_type == MXFP4_BF16 ? mx_dequantize_rows<MXFP4_BF16> : mx_dequantize_rows<MXFP4_F32>;
  hipLaunchKernelGGL(k, r.grid, dim3(kThreads), 0, stream, codes, scales, M, K, r.shift, y, ldy);
  return hipGetLastError();
}

hipError_t launch_mx_check_scales(const uint8_t* scales, int64_t bytes, uint32_t* faults,
                                  hipStream_t stream) {
  int64_t g = (bytes + kThreads * 16 - 1) / (kThreads * 16);
  if (g > 2048) g = 2048;
  hipLaunchKernelGGL(mx_scan_scales, dim3((uint32_t)g), dim3(kThreads), 0, stream, scales, bytes,
                     faults);
  return hipGetLastError();
}

}  // namespace nvfp4
