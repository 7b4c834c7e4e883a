// The ordered combine of the MXFP4 grouped product.
#include "mx_device.hpp"
#include "mx_kernels.hpp"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

// One wave per (token, 256 columns), four columns per lane. Lane j holds the token's j-th
// route: kept when its id is in range and the first of its kind, ranked by id among the kept
// ones, and moved to the lane of its rank (top_k <= 64), with no barrier; then the rows are
// added with fmaf in that order, from zero. Bound by the rows' bytes at prompt sizes (268 MB
// of them for 4096 tokens x top-8 x 2048 columns, read at 5.2 TB/s) and by two dependent reads
// at decode sizes.
__global__ __launch_bounds__(kThreads) void mx_combine(const float* rows, int64_t pitch,
                                                       const int32_t* topk_ids,
                                                       const float* topk_w, int top_k, int E,
                                                       int64_t N, int y_type, void* y,
                                                       int64_t ldy) {
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63;
  const bool have = lane < top_k;
  const int32_t id = have ? topk_ids[t * top_k + lane] : -1;
  const float w = have ? topk_w[t * top_k + lane] : 0.f;
  bool mine = id >= 0 && id < E;
  for (int i = 0; i < top_k; i++) mine = mine && !(i < lane && __builtin_amdgcn_readlane(id, i) == id);
  const uint64_t kept_mask = __ballot(mine);
  const int kept = __builtin_popcountll(kept_mask);
  int rank = 0, behind = kept;  // lanes that keep nothing go behind, to lanes of their own
  for (int i = 0; i < top_k; i++)
    rank += (kept_mask >> i & 1) && __builtin_amdgcn_readlane(id, i) < id;
  behind += __builtin_popcountll(~kept_mask & ((1ull << lane) - 1));
  const int to = 4 * (mine ? rank : behind);
  const int route = __builtin_amdgcn_ds_permute(to, lane);
  const int weight = __builtin_amdgcn_ds_permute(to, __float_as_int(w));

  const int64_t n0 = (int64_t)blockIdx.y * (4 * kThreads) + 4 * threadIdx.x;
  const bool vec = ((N | pitch) & 3) == 0;  // then n0 + 4 <= N and rows are 16-byte aligned
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  constexpr int kBatch = 8;  // rows in flight per thread
  for (int q0 = 0; q0 < kept; q0 += kBatch) {
    float v[kBatch][4];
#pragma unroll
    for (int q = 0; q < kBatch; q++) {
      if (q0 + q >= kept) break;
      const float* src = rows + (t * top_k + __builtin_amdgcn_readlane(route, q0 + q)) * pitch + n0;
      if (vec) {
        const float4 f = n0 < N ? *reinterpret_cast<const float4*>(src) : float4{0.f, 0.f, 0.f, 0.f};
        v[q][0] = f.x, v[q][1] = f.y, v[q][2] = f.z, v[q][3] = f.w;
      } else {
#pragma unroll
        for (int c = 0; c < 4; c++) v[q][c] = n0 + c < N ? src[c] : 0.f;
      }
    }
#pragma unroll
    for (int q = 0; q < kBatch; q++) {
      if (q0 + q >= kept) break;
      const float wq = __int_as_float(__builtin_amdgcn_readlane(weight, q0 + q));
#pragma unroll
      for (int c = 0; c < 4; c++) acc[c] = __builtin_fmaf(wq, v[q][c], acc[c]);
    }
  }
  if (n0 >= N) return;
  const bool whole = n0 + 4 <= N;
  if (y_type == MXFP4_F32) {
    float* d = static_cast<float*>(y) + t * ldy + n0;
    if (whole && ((uintptr_t)d & 15) == 0) {
      *reinterpret_cast<float4*>(d) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; c++)
        if (n0 + c < N) d[c] = acc[c];
    }
  } else {
    uint16_t* d = static_cast<uint16_t*>(y) + t * ldy + n0;
    const uint2 b = make_uint2(bf16_pair(acc[0], acc[1]), bf16_pair(acc[2], acc[3]));
    if (whole && ((uintptr_t)d & 7) == 0) {
      *reinterpret_cast<uint2*>(d) = b;
    } else {
#pragma unroll
      for (int c = 0; c < 4; c++)
        if (n0 + c < N) d[c] = (uint16_t)((c < 2 ? b.x : b.y) >> (16 * (c & 1)));
    }
  }
}

}  // namespace

hipError_t launch_mx_combine(const float* rows, int64_t pitch, const int32_t* topk_ids,
                             const float* topk_w, int64_t T, int top_k, int E, int64_t N,
                             int y_type, void* y, int64_t ldy, hipStream_t stream) {
  hipLaunchKernelGGL(mx_combine, dim3((uint32_t)T, (uint32_t)((N + 4 * kThreads - 1) / (4 * kThreads))),
                     dim3(kThreads), 0, stream, rows, pitch, topk_ids, topk_w, top_k, E, N, y_type,
                     y, ldy);
  return hipGetLastError();
}

}  // namespace nvfp4
