// The ordered combine of the MXFP4 grouped product.
#include "mx_device.hpp"
#include "mx_kernels.hpp"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTopK = 64;

// One workgroup per (token, 1024 columns). The first top_k threads rank their routes by
// expert among the token's kept ones (in range, the first of their id) and stage row and
// weight in that order; each thread then adds its four columns of the rows with fmaf, in
// that order, from zero.
__global__ __launch_bounds__(kThreads) void mx_combine(const float* rows,
                                                       const int32_t* topk_ids,
                                                       const float* topk_w, int top_k, int E,
                                                       int64_t N, int y_type, void* y) {
  __shared__ int32_t ex[kMaxTopK];
  __shared__ int64_t rr[kMaxTopK];
  __shared__ float wr[kMaxTopK];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  int32_t e = -1;
  float w = 0.f;
  if (tid < top_k) {
    ex[tid] = e = topk_ids[t * top_k + tid];
    w = topk_w[t * top_k + tid];
  }
  __syncthreads();
  int kept = 0, slot = 0;
  bool mine = e >= 0 && e < E;
  for (int j = 0; j < top_k; j++) {
    const int32_t f = ex[j];
    bool ok = f >= 0 && f < E;
    for (int i = 0; i < j; i++) ok = ok && ex[i] != f;
    kept += ok;
    slot += ok && f < e;
    if (j < tid && f == e) mine = false;
  }
  if (mine) {
    rr[slot] = t * top_k + tid;
    wr[slot] = w;
  }
  __syncthreads();
  const int64_t n0 = (int64_t)blockIdx.y * (4 * kThreads) + 4 * tid;
  if (n0 >= N) return;
  const bool vec = (N & 3) == 0;  // then n0 + 4 <= N and every row is 16-byte aligned
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  constexpr int kBatch = 8;  // rows in flight per thread
  for (int q0 = 0; q0 < kept; q0 += kBatch) {
    float v[kBatch][4];
#pragma unroll
    for (int q = 0; q < kBatch; q++) {
      if (q0 + q >= kept) break;
      const float* src = rows + rr[q0 + q] * N + n0;
      if (vec) {
        const float4 f = *reinterpret_cast<const float4*>(src);
        v[q][0] = f.x, v[q][1] = f.y, v[q][2] = f.z, v[q][3] = f.w;
      } else {
#pragma unroll
        for (int c = 0; c < 4; c++) v[q][c] = n0 + c < N ? src[c] : 0.f;
      }
    }
#pragma unroll
    for (int q = 0; q < kBatch; q++) {
      if (q0 + q >= kept) break;
#pragma unroll
      for (int c = 0; c < 4; c++) acc[c] = __builtin_fmaf(wr[q0 + q], v[q][c], acc[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < 4; c++) {
    if (n0 + c >= N) break;
    if (y_type == MXFP4_F32) {
      static_cast<float*>(y)[t * N + n0 + c] = acc[c];
    } else {
      static_cast<uint16_t*>(y)[t * N + n0 + c] = (uint16_t)f32_to_bf16_any(acc[c]);
    }
  }
}

}  // namespace

hipError_t launch_mx_combine(const float* rows, const int32_t* topk_ids, const float* topk_w,
                             int64_t T, int top_k, int E, int64_t N, int y_type, void* y,
                             hipStream_t stream) {
  hipLaunchKernelGGL(mx_combine, dim3((uint32_t)T, (uint32_t)((N + 4 * kThreads - 1) / (4 * kThreads))),
                     dim3(kThreads), 0, stream, rows, topk_ids, topk_w, top_k, E, N, y_type, y);
  return hipGetLastError();
}

}  // namespace nvfp4
