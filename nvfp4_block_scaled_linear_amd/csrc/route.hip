// Routing to experts (moe_route in fp8.h).
//
// One wave per token. Lane l holds the experts l * V + [0, V) in registers: their logits and the
// keys that they are picked by. Without a bias the keys are the logits themselves (scores grow
// with them), otherwise the scores in 64 bits: experts lie close together, and in 32 bits which
// of two is the larger would depend on how the sums were ordered. The picks are top_k rounds of a
// largest key over the wave, ties to the lower lane and index; lane j keeps pick j and computes
// its weight. Groups are scored by a lane each, from the keys in LDS.
#include <type_traits>

#include "f8_kernels.hpp"

#include "device.hpp"

namespace nvfp4 {
namespace {

constexpr float kLargest = 3.402823466e+38f;

__device__ __forceinline__ float minus_inf() { return __uint_as_float(0xFF800000u); }

// this wave's LDS writes stand before its reads that follow
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <class T>
__device__ __forceinline__ T wave_max(T v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const T o = __shfl_xor(v, d, 64);
    v = o > v ? o : v;
  }
  return v;
}

template <class T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// V experts a lane; SCORES: keys are scores (with a bias, or for the sum of a group's two best)
template <int V, bool SCORES>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs a) {
  typedef typename std::conditional<SCORES, double, float>::type Key;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * waves + wave;
  if (t >= a.T) return;
  const int E = a.num_experts, G = a.num_groups;
  const Key none = (Key)minus_inf();
  float l[V];
  Key key[V];
#pragma unroll
  for (int i = 0; i < V; i++) {
    const int e = lane * V + i;
    float v = minus_inf();
    if (e < E) {
      if (a.logits_type == FP8_BF16)
        v = bf16_bits_to_f32(static_cast<const uint16_t*>(a.logits)[t * a.ld + e]);
      else
        v = static_cast<const float*>(a.logits)[t * a.ld + e];
      v = v > minus_inf() ? (v < kLargest ? v : kLargest) : minus_inf();
    }
    l[i] = v;
  }
  float top = l[0];
#pragma unroll
  for (int i = 1; i < V; i++) top = l[i] > top ? l[i] : top;
  top = wave_max(top);
  double total = 1.0;  // softmax's sum, where it is needed
  if (a.scoring == ROUTE_SOFTMAX && (SCORES || !a.renormalize)) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; i++) {
      const double p = l[i] > minus_inf() ? exp((double)l[i] - (double)top) : 0.0;
      if (SCORES) key[i] = (Key)p;
      sum += p;
    }
    total = wave_sum(sum);
  }
#pragma unroll
  for (int i = 0; i < V; i++) {
    if (!SCORES) {
      key[i] = l[i];
      continue;
    }
    const double s = a.scoring == ROUTE_SOFTMAX ? (double)key[i] / total : 1.0 / (1.0 + exp(-(double)l[i]));
    const int e = lane * V + i;
    const float b = a.bias && e < E ? a.bias[e] : 0.0f;
    key[i] = l[i] > minus_inf() && b > minus_inf() ? (Key)(s + (double)b) : none;
  }

  if (G > 1) {
    Key* const keys = reinterpret_cast<Key*>(smem) + (int64_t)wave * (E + G);
    Key* const best = keys + E;
#pragma unroll
    for (int i = 0; i < V; i++)
      if (lane * V + i < E) keys[lane * V + i] = key[i];
    wave_lds_fence();
    const int size = E / G;
    for (int g = lane; g < G; g += 64) {
      Key first = none, second = none;
      for (int i = 0; i < size; i++) {
        const Key k = keys[g * size + i];
        second = k > first ? first : k > second ? k : second;
        first = k > first ? k : first;
      }
      best[g] = a.group_score == ROUTE_GROUP_TOP2 && second > none ? first + second : first;
    }
    wave_lds_fence();
    // a group's place among all: those with a larger score, and equal ones before it
    for (int g = lane; g < G; g += 64) {
      const Key mine = best[g];
      int place = 0;
      for (int o = 0; o < G; o++) place += best[o] > mine || (best[o] == mine && o < g);
      if (place >= a.top_groups)
        for (int i = 0; i < size; i++) keys[g * size + i] = none;
    }
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < V; i++)
      if (lane * V + i < E) key[i] = keys[lane * V + i];
  }

  int32_t id = -1;
  float mine = 0.0f;  // lane j: the logit of pick j
  for (int j = 0; j < a.top_k; j++) {
    Key k = key[0];
    int at = 0;
    float lg = l[0];
#pragma unroll
    for (int i = 1; i < V; i++)
      if (key[i] > k) k = key[i], at = i, lg = l[i];
    const Key m = wave_max(k);
    if (!(m > none)) break;
    const int from = __builtin_ctzll(__ballot(k == m));
    const int where = __builtin_amdgcn_readlane(at, from);
    const float logit = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(lg), from));
    if (lane == j) id = from * V + where, mine = logit;
#pragma unroll
    for (int i = 0; i < V; i++)
      if (lane == from && i == where) key[i] = none;
  }
  double s = 0.0;
  if (id >= 0) s = a.scoring == ROUTE_SOFTMAX ? exp((double)mine - (double)top) / total : 1.0 / (1.0 + exp(-(double)mine));
  if (a.renormalize) {
    const double sum = wave_sum(s);
    s = sum > 0.0 ? s / sum : 0.0;
  }
  if (lane < a.top_k) {
    a.topk_ids[t * a.top_k + lane] = id;
    a.topk_w[t * a.top_k + lane] = (float)(s * (double)a.scale);
  }
}

template <int V, bool SCORES>
hipError_t launch(const RouteArgs& a, hipStream_t stream) {
  const size_t bytes = a.num_groups > 1 ? (SCORES ? 8 : 4) * (size_t)(a.num_experts + a.num_groups) : 0;
  const int waves = bytes * 4 <= 65536 ? 4 : 1;
  hipLaunchKernelGGL((moe_route_kernel<V, SCORES>), dim3((uint32_t)((a.T + waves - 1) / waves)), dim3(64 * waves),
                     bytes * waves, stream, a);
  return hipGetLastError();
}

template <bool SCORES>
hipError_t launch_experts(const RouteArgs& a, hipStream_t stream) {
  const int E = a.num_experts;
  if (E <= 64) return launch<1, SCORES>(a, stream);
  if (E <= 128) return launch<2, SCORES>(a, stream);
  if (E <= 256) return launch<4, SCORES>(a, stream);
  if (E <= 512) return launch<8, SCORES>(a, stream);
  if (E <= 1024) return launch<16, SCORES>(a, stream);
  return launch<64, SCORES>(a, stream);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
  const bool scores = a.bias || (a.num_groups > 1 && a.group_score == ROUTE_GROUP_TOP2);
  return scores ? launch_experts<true>(a, stream) : launch_experts<false>(a, stream);
}

}  // namespace nvfp4
