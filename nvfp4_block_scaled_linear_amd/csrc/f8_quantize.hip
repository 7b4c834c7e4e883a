// FP8 quantizer and its way back (rules in fp8.h), and the scans of check mode. Bound by memory:
// 2 or 4 bytes of a value on one side, 1 + 4/128 on the other. Measured, 2048 x 14336 BF16: 16 to 18
// us (89 MB, 5.1 TB/s), from fp32 28 (149 MB), the way back 17; a weight of 14336 x 4096 36 (176 MB,
// 4.9 TB/s), from fp32 55 (294 MB); 16 x 4096 3.1 and 2.5, the latency of a launch.
//
// Eight lanes take a block of 128 k of a row, 16 values per lane, so that the block's largest
// value is three exchanges inside the eight and a lane's codes are one 16-byte store. A weight's
// block is a workgroup's: 32 rows at a time, four times, held in registers between the
// largest value and the codes, which are joined in LDS.
#include "f8_kernels.hpp"

#include "f8_device.hpp"

#pragma clang fp contract(off)

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 8;  // of a row's block, 16 values each

template <int T>
__device__ __forceinline__ void load16(const void* x, int64_t off, float v[16]) {
  constexpr int E = T == FP8_BF16 ? 2 : 4;
  const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(x) + off * E);
  u32x4 a[E];
#pragma unroll
  for (int i = 0; i < E; i++) a[i] = p[i];
#pragma unroll
  for (int i = 0; i < 16; i++) {
    if (T == FP8_F32)
      v[i] = __uint_as_float(a[i >> 2][i & 3]);
    else
      v[i] = __uint_as_float(i & 1 ? a[i >> 3][(i & 7) >> 1] & 0xFFFF0000u : a[i >> 3][(i & 7) >> 1] << 16);
  }
}

__device__ __forceinline__ uint32_t largest16(const float v[16]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 16; i++) {
    const uint32_t u = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    m = m > u ? m : u;
  }
  return m;
}

__device__ __forceinline__ uint32_t largest_of_lanes(uint32_t m) {
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) {
    const uint32_t o = __shfl_xor(m, d, 64);
    m = m > o ? m : o;
  }
  return m;
}

// 16 codes of a block with largest magnitude amax (bits) and scale s; of one that is not finite, 0
__device__ __forceinline__ void store_codes(uint8_t* to, const float v[16], uint32_t amax, float s) {
  u32x4 c = {0u, 0u, 0u, 0u};
  if (amax < 0x7F800000u) f8_codes<16>(v, __uint_as_float(amax), s, reinterpret_cast<uint32_t*>(&c));
  *reinterpret_cast<u32x4*>(to) = c;
}

// Threads of a workgroup: 2^shift side by side along a row, eight to a block, the rest down the
// rows.
template <int T, int RULE>
__global__ __launch_bounds__(kThreads) void f8_quantize_rows(const void* x, int64_t ldx, int64_t M,
                                                             int64_t K, int32_t kb, int shift,
                                                             uint8_t* codes, float* scales,
                                                             uint32_t* faults) {
  const int64_t row = (int64_t)blockIdx.x * (kThreads >> shift) + (threadIdx.x >> shift);
  if (row >= M) return;
  const int pieces = kb * kLanes;  // of 16 values, of whole blocks
  bool bad = false;
  // whole groups of lanes leave together
  for (int p = ((int)blockIdx.y << shift) + (threadIdx.x & ((1 << shift) - 1)); p < pieces; p += gridDim.y << shift) {
    const int64_t k = 16 * (int64_t)p;
    const bool in = k < K;  // K % 16 == 0
    float v[16];
    if (in) {
      load16<T>(x, row * ldx + k, v);
    } else {
#pragma unroll
      for (int i = 0; i < 16; i++) v[i] = 0.0f;
    }
    const uint32_t amax = largest_of_lanes(largest16(v));
    const bool odd = amax >= 0x7F800000u;  // a NaN or Inf is the largest as bits
    bad = bad || odd;
    const float s = f8_scale<RULE>(__uint_as_float(amax));
    if (in) store_codes(codes + row * K + k, v, amax, s);
    if (p % kLanes == 0) scales[row * kb + p / kLanes] = odd ? __uint_as_float(0x7FC00000u) : s;
  }
  if (bad && faults) atomicOr(faults, (uint32_t)NVFP4_FAULT_NONFINITE);
}

template <int T, int RULE>
__global__ __launch_bounds__(kThreads) void f8_quantize_blocks(const void* x, int64_t ldx, int64_t M,
                                                               int64_t K, int32_t kb, uint8_t* codes,
                                                               float* scales, uint32_t* faults) {
  constexpr int kRows = kThreads / kLanes, kPer = kF8Block / kRows;
  __shared__ uint32_t top[kThreads / 64];
  const int64_t b = blockIdx.x, down = b / kb, k = (b - down * kb) * kF8Block + 16 * (threadIdx.x % kLanes);
  const int64_t row0 = down * kF8Block + threadIdx.x / kLanes;
  float v[kPer][16];
  uint32_t amax = 0u;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    if (k < K && row0 + i * kRows < M) {
      load16<T>(x, (row0 + i * kRows) * ldx + k, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 16; j++) v[i][j] = 0.0f;
    }
    const uint32_t m = largest16(v[i]);
    amax = amax > m ? amax : m;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_xor(amax, d, 64);
    amax = amax > o ? amax : o;
  }
  if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; w++) amax = amax > top[w] ? amax : top[w];
  const bool odd = amax >= 0x7F800000u;
  const float s = f8_scale<RULE>(__uint_as_float(amax));
#pragma unroll
  for (int i = 0; i < kPer; i++)
    if (k < K && row0 + i * kRows < M)
      store_codes(codes + (row0 + i * kRows) * K + k, v[i], amax, s);
  if (threadIdx.x == 0) {
    scales[b] = odd ? __uint_as_float(0x7FC00000u) : s;
    if (odd && faults) atomicOr(faults, (uint32_t)NVFP4_FAULT_NONFINITE);
  }
}

template <int T>
__global__ __launch_bounds__(kThreads) void f8_dequantize_rows(const uint8_t* codes, const float* scales,
                                                               int64_t M, int64_t K, int32_t kb,
                                                               int row_shift, int shift, void* y, int64_t ldy) {
  const int64_t row = (int64_t)blockIdx.x * (kThreads >> shift) + (threadIdx.x >> shift);
  if (row >= M) return;
  const int pieces = (int)(K >> 4);
  for (int p = ((int)blockIdx.y << shift) + (threadIdx.x & ((1 << shift) - 1)); p < pieces; p += gridDim.y << shift) {
    const int64_t k = 16 * (int64_t)p;
    const u32x4 c = *reinterpret_cast<const u32x4*>(codes + row * K + k);
    const float s = scales[(row >> row_shift) * kb + (k >> 7)];
    float v[16];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[4 * i] = e4m3_to_f32<0>(c[i]) * s;
      v[4 * i + 1] = e4m3_to_f32<1>(c[i]) * s;
      v[4 * i + 2] = e4m3_to_f32<2>(c[i]) * s;
      v[4 * i + 3] = e4m3_to_f32<3>(c[i]) * s;
    }
    if (T == FP8_BF16) {
      u32x4* d = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(y) + row * ldy + k);
#pragma unroll
      for (int i = 0; i < 2; i++)
        d[i] = u32x4{bf16_pair(v[8 * i], v[8 * i + 1]), bf16_pair(v[8 * i + 2], v[8 * i + 3]),
                     bf16_pair(v[8 * i + 4], v[8 * i + 5]), bf16_pair(v[8 * i + 6], v[8 * i + 7])};
    } else {
      f32x4* d = reinterpret_cast<f32x4*>(static_cast<float*>(y) + row * ldy + k);
#pragma unroll
      for (int i = 0; i < 4; i++) d[i] = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    }
  }
}

__global__ __launch_bounds__(kThreads) void f8_scan_scales(const float* p, int64_t n, uint32_t* faults) {
  bool hit = false;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads)
    hit = hit || !is_finite(p[i]);
  if (hit) atomicOr(faults, (uint32_t)NVFP4_FAULT_NAN_SCALE);
}

// A byte's low seven bits plus one reach 0x80 only from 0x7F, the NaN, and no byte carries.
__global__ __launch_bounds__(kThreads) void f8_scan_codes(const uint8_t* p, int64_t ld, int64_t rows,
                                                          int64_t K, uint32_t* faults) {
  const int64_t pieces = K >> 4, all = rows * pieces;
  uint32_t hit = 0u;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = i / pieces;
    const u32x4 v = *reinterpret_cast<const u32x4*>(p + row * ld + ((i - row * pieces) << 4));
#pragma unroll
    for (int j = 0; j < 4; j++) hit |= ((v[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  }
  if (hit) atomicOr(faults, (uint32_t)NVFP4_FAULT_NONFINITE);
}

// threads along a row of `pieces` (a power of two, at least 2^least) and the launch grid
struct RowShape {
  int shift;
  dim3 grid;
};

RowShape row_shape(int64_t M, int64_t pieces, int least) {
  int shift = least;
  while (shift < 8 && ((int64_t)1 << shift) < pieces) shift++;
  const int64_t gx = (M + (kThreads >> shift) - 1) / (kThreads >> shift);
  const int64_t gy = (pieces + ((int64_t)1 << shift) - 1) >> shift;
  return {shift, dim3((uint32_t)gx, (uint32_t)(gy < 1024 ? gy : 1024))};
}

// workgroups for n items of a thread each, at most `most`
dim3 grid_of(int64_t n, int64_t most) {
  const int64_t g = (n + kThreads - 1) / kThreads;
  return dim3((uint32_t)(g < most ? g : most));
}

}  // namespace

hipError_t launch_f8_quantize(int x_type, const void* x, int64_t ldx, int64_t M, int64_t K,
                              int block_rows, int scale_rule, uint8_t* codes, float* scales,
                              uint32_t* faults, hipStream_t stream) {
  const int32_t kb = (int32_t)((K + kF8Block - 1) / kF8Block);
  const bool bf16 = x_type == FP8_BF16, pow2 = scale_rule == FP8_SCALE_POW2;
  if (block_rows == 1) {
    const RowShape r = row_shape(M, kb * (int64_t)kLanes, 3);
    auto k = bf16 ? pow2 ? f8_quantize_rows<FP8_BF16, FP8_SCALE_POW2> : f8_quantize_rows<FP8_BF16, FP8_SCALE_F32>
                  : pow2 ? f8_quantize_rows<FP8_F32, FP8_SCALE_POW2> : f8_quantize_rows<FP8_F32, FP8_SCALE_F32>;
    hipLaunchKernelGGL(k, r.grid, dim3(kThreads), 0, stream, x, ldx, M, K, kb, r.shift, codes, scales, faults);
    return hipGetLastError();
  }
  const int64_t blocks = (M + kF8Block - 1) / kF8Block * kb;
  if (blocks * kThreads > (int64_t)UINT32_MAX) return hipErrorInvalidConfiguration;
  auto k = bf16 ? pow2 ? f8_quantize_blocks<FP8_BF16, FP8_SCALE_POW2> : f8_quantize_blocks<FP8_BF16, FP8_SCALE_F32>
                : pow2 ? f8_quantize_blocks<FP8_F32, FP8_SCALE_POW2> : f8_quantize_blocks<FP8_F32, FP8_SCALE_F32>;
  hipLaunchKernelGGL(k, dim3((uint32_t)blocks), dim3(kThreads), 0, stream, x, ldx, M, K, kb, codes, scales, faults);
  return hipGetLastError();
}

hipError_t launch_f8_dequantize(const uint8_t* codes, const float* scales, int64_t M, int64_t K,
                                int block_rows, int y_type, void* y, int64_t ldy,
                                hipStream_t stream) {
  const int32_t kb = (int32_t)((K + kF8Block - 1) / kF8Block);
  const RowShape r = row_shape(M, K >> 4, 0);
  auto k = y_type == FP8_BF16 ? f8_dequantize_rows<FP8_BF16> : f8_dequantize_rows<FP8_F32>;
  hipLaunchKernelGGL(k, r.grid, dim3(kThreads), 0, stream, codes, scales, M, K, kb, block_rows == 1 ? 0 : 7, r.shift,
                     y, ldy);
  return hipGetLastError();
}

hipError_t launch_f8_check_scales(const float* scales, int64_t n, uint32_t* faults,
                                  hipStream_t stream) {
  hipLaunchKernelGGL(f8_scan_scales, grid_of(n, 2048), dim3(kThreads), 0, stream, scales, n, faults);
  return hipGetLastError();
}

hipError_t launch_f8_check_codes(const uint8_t* codes, int64_t ld, int64_t rows, int64_t K,
                                 uint32_t* faults, hipStream_t stream) {
  hipLaunchKernelGGL(f8_scan_codes, grid_of(rows * (K >> 4), 2048), dim3(kThreads), 0, stream, codes, ld, rows,
                     K, faults);
  return hipGetLastError();
}

}  // namespace nvfp4
