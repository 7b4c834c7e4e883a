// Routing to experts (moe_route in fp8.h).
//
// One wave per token (many tokens: moe_route_many, below). Lane l holds the experts l * V + [0, V):
// the keys that they are picked by, as 32-bit integers in the order of the floats that they stand
// for. The picks are top_k rounds of a largest key over the wave (lane exchanges inside the vector
// unit, no LDS), ties to the lower lane and index; lane j keeps pick j, and computes its weight in
// 64 bits at the end.
// Measured: one token of 128 experts 2.9 us, 16 4.8, which is latency; 16384 of 256, groups and a
// bias, 20 us (17 MB: 3.6 us to read): 1640 vector instructions a wave and four waves on a SIMD keep
// the vector units busy for 27000 cycles of it, more than half. About a fifth of them are the
// picks; the others sort the lists, score the groups and compute the weights in 64 bits.
//  - Without a bias, and unless groups are scored by their two best, the keys are the logits
//    themselves: scores grow with them, so the order is exact.
//  - Otherwise the keys are fp32 scores, good to near_of / 2. Where two picks in a row, the last pick
//    and the next best, or a kept group and one that is not lie closer than that allows to tell
//    apart (picks that are equal in logit and bias aside), the token is decided again by scores in
//    64 bits (decide64), a few tokens in a thousand where logits are spread like a router's.
// Groups are scored by lane exchanges where a group is a power of two of lanes, up to 16, and by a
// lane each, from keys in LDS, otherwise (scores: in decide64).
#include "f8_kernels.hpp"

#include "device.hpp"

namespace nvfp4 {
namespace {

constexpr float kLargest = 3.402823466e+38f;
// Twice the error of an fp32 score plus bias, relative to 1 + its magnitude. A score is at most 1. A
// sigmoid's exponential (its argument's rounding included), sum and reciprocal and the addition of
// the bias are off by less than 6 * 2^-24. An exponential of softmax is off by the rounding of its
// argument x, 2^-23 |x| of itself, which is at most 2^-24 of the largest score; its sum of `terms`
// steps by as many times 2^-24 of itself, and product and reciprocal by a few more.
__device__ __forceinline__ float near_of(int scoring, int terms) {
  return 2.0f / 16777216.0f * (scoring == ROUTE_SOFTMAX ? (float)(terms + 16) : 6.0f);
}

__device__ __forceinline__ float minus_inf() { return __uint_as_float(0xFF800000u); }

// floats (no NaN; -0 must have been made +0) as integers of the same order, and back
__device__ __forceinline__ int32_t ordered(float v) {
  const int32_t b = __float_as_int(v);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float unordered(int32_t k) { return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF)); }
constexpr int32_t kNone = (int32_t)0x807FFFFF;  // ordered(-infinity)

// v from another lane of the same 16 (in a form that the compiler folds into the operation on it)
template <int CTRL>
__device__ __forceinline__ int32_t from_lane(int32_t v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float from_lane(float v) {
  return __int_as_float(from_lane<CTRL>(__float_as_int(v)));
}
// lane l ^ 1, l ^ 2; the mirrored lane of 8, of 16; l - n round the 16
enum { kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140, kRotate = 0x120 };

__device__ __forceinline__ int32_t larger(int32_t a, int32_t b) { return a > b ? a : b; }

// the largest of 16 lanes, in each of them; of the wave's
__device__ __forceinline__ int32_t row_max(int32_t v) {
  v = larger(v, from_lane<kXor1>(v));
  v = larger(v, from_lane<kXor2>(v));
  v = larger(v, from_lane<kMirror8>(v));
  return larger(v, from_lane<kMirror16>(v));
}
__device__ __forceinline__ int32_t wave_max(int32_t v) {
  v = row_max(v);
  return larger(larger(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
                larger(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}

template <int CTRL>
__device__ __forceinline__ double from_lane(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = (uint32_t)from_lane<CTRL>((int32_t)b), hi = (uint32_t)from_lane<CTRL>((int32_t)(b >> 32));
  return __builtin_bit_cast(double, hi << 32 | lo);
}
__device__ __forceinline__ float lane_of(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
__device__ __forceinline__ double lane_of(double v, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = (uint32_t)__builtin_amdgcn_readlane((int32_t)b, l);
  const uint64_t hi = (uint32_t)__builtin_amdgcn_readlane((int32_t)(b >> 32), l);
  return __builtin_bit_cast(double, hi << 32 | lo);
}

// the sum over the wave, in every lane
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
  v += from_lane<kXor1>(v);
  v += from_lane<kXor2>(v);
  v += from_lane<kMirror8>(v);
  v += from_lane<kMirror16>(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}
// the largest of the wave's, in every lane
template <int CTRL>
__device__ __forceinline__ double larger_of_lane(double v) {
  const double o = from_lane<CTRL>(v);
  return o > v ? o : v;
}
__device__ __forceinline__ double wave_max(double v) {
  v = larger_of_lane<kXor1>(v);
  v = larger_of_lane<kXor2>(v);
  v = larger_of_lane<kMirror8>(v);
  v = larger_of_lane<kMirror16>(v);
  const double p = lane_of(v, 0), q = lane_of(v, 16), r = lane_of(v, 32), u = lane_of(v, 48);
  const double x = p > q ? p : q, y = r > u ? r : u;
  return x > y ? x : y;
}

// this wave's LDS writes stand before its reads that follow
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// a logit as it counts: -infinity for a closed expert's, +0 for -0
__device__ __forceinline__ float counted(float v) {
  return v > minus_inf() ? (v < kLargest ? v : kLargest) + 0.0f : minus_inf();
}

__device__ __forceinline__ float logit_of(const RouteArgs& a, int64_t t, int e) {
  return counted(a.logits_type == FP8_BF16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(a.logits)[t * a.ld + e])
                                           : static_cast<const float*>(a.logits)[t * a.ld + e]);
}

// The logits of experts first + i * step, i < V, of token t; all loads at once, past the last expert
// of the last one.
template <int V>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t t, int first, int step, float (&l)[V]) {
  const int last = a.num_experts - 1;
  const auto place = [&](int i) { return first + i * step < last ? first + i * step : last; };
  if (a.logits_type == FP8_BF16) {
    const uint16_t* const p = static_cast<const uint16_t*>(a.logits) + t * a.ld;
#pragma unroll
    for (int i = 0; i < V; i++) l[i] = bf16_bits_to_f32(p[place(i)]);
  } else {
    const float* const p = static_cast<const float*>(a.logits) + t * a.ld;
#pragma unroll
    for (int i = 0; i < V; i++) l[i] = p[place(i)];
  }
#pragma unroll
  for (int i = 0; i < V; i++) l[i] = first + i * step <= last ? counted(l[i]) : minus_inf();
}

// the biases of the same experts (0 without)
template <int V>
__device__ __forceinline__ void load_bias(const RouteArgs& a, int first, int step, float (&b)[V]) {
  const int last = a.num_experts - 1;
  if (!a.bias) {
#pragma unroll
    for (int i = 0; i < V; i++) b[i] = 0.0f;
    return;
  }
#pragma unroll
  for (int i = 0; i < V; i++) b[i] = a.bias[first + i * step < last ? first + i * step : last];
}

// The picks of token t by a whole wave, by keys of 64 bits: scores, or without SCORES the logits
// themselves, which scores of 64 bits do not tell apart everywhere (sigmoids above 37 are 1, so is
// exp of 1e-20, and exp of -800 is 0). Returns the id of pick `lane`, or -1. Lane l has experts
// l * V + [0, V); LDS (E + G doubles) serves groups that are no power of two of lanes.
template <int V, bool SCORES>
__device__ __forceinline__ int32_t decide64(const RouteArgs& a, int64_t t, double* lds) {
  const int lane = threadIdx.x & 63, E = a.num_experts, G = a.num_groups;
  const double none = (double)minus_inf();
  float l[V], bias[V];
  if (SCORES) load_bias<V>(a, lane * V, 1, bias);
  load_logits<V>(a, t, lane * V, 1, l);
  double key[V];
  if (!SCORES) {
#pragma unroll
    for (int i = 0; i < V; i++) key[i] = (double)l[i];
  } else if (a.scoring == ROUTE_SOFTMAX) {
    int32_t m = ordered(l[0]);
#pragma unroll
    for (int i = 1; i < V; i++) m = larger(m, ordered(l[i]));
    const double top = (double)unordered(wave_max(m));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; i++) {
      key[i] = l[i] > minus_inf() ? exp((double)l[i] - top) : 0.0;
      sum += key[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < V; i++) key[i] /= sum;
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) key[i] = 1.0 / (1.0 + exp(-(double)l[i]));
  }
  if (SCORES) {
#pragma unroll
    for (int i = 0; i < V; i++) key[i] = l[i] > minus_inf() && bias[i] > minus_inf() ? key[i] + (double)bias[i] : none;
  }
  if (G > 1) {
    double* const best = lds + E;
#pragma unroll
    for (int i = 0; i < V; i++)
      if (lane * V + i < E) lds[lane * V + i] = key[i];
    wave_lds_fence();
    const int size = E / G;
    for (int g = lane; g < G; g += 64) {
      double first = none, second = none;
#pragma unroll 4
      for (int i = 0; i < size; i++) {
        const double k = lds[g * size + i];
        second = k > first ? first : k > second ? k : second;
        first = k > first ? k : first;
      }
      best[g] = a.group_score == ROUTE_GROUP_TOP2 && second > none ? first + second : first;
    }
    wave_lds_fence();
    // a group's place among all: those with a larger score, and equal ones before it
    for (int g = lane; g < G; g += 64) {
      const double mine = best[g];
      int place = 0;
#pragma unroll 4
      for (int o = 0; o < G; o++) place += best[o] > mine || (best[o] == mine && o < g);
      if (place >= a.top_groups)
        for (int i = 0; i < size; i++) lds[g * size + i] = none;
    }
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < V; i++)
      if (lane * V + i < E) key[i] = lds[lane * V + i];
  }
  int32_t id = -1;
  for (int j = 0; j < a.top_k; j++) {
    double k = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < V; i++) {
      at = key[i] > k ? i : at;
      k = key[i] > k ? key[i] : k;
    }
    const double m = wave_max(k);
    if (!(m > none)) break;
    const int from = __builtin_ctzll(__ballot(k == m));
    const int e = from * V + __builtin_amdgcn_readlane(at, from);
    if (lane == j) id = e;
#pragma unroll
    for (int i = 0; i < V; i++) key[i] = lane * V + i == e ? none : key[i];
  }
  return id;
}

// One key more to the two largest.
__device__ __forceinline__ void put(int32_t& first, int32_t& second, int32_t k) {
  const int32_t low = first < k ? first : k;
  second = larger(second, low);
  first = larger(first, k);
}

// The two largest keys of a group of 2^shift lanes, in all its lanes, from each lane's own two.
__device__ __forceinline__ void group_best2(int shift, int32_t& first, int32_t& second) {
  const auto merge = [&](int32_t f, int32_t s) {
    put(first, second, f);
    second = larger(second, s);
  };
  if (shift >= 1) merge(from_lane<kXor1>(first), from_lane<kXor1>(second));
  if (shift >= 2) merge(from_lane<kXor2>(first), from_lane<kXor2>(second));
  if (shift >= 3) merge(from_lane<kMirror8>(first), from_lane<kMirror8>(second));
  if (shift >= 4) merge(from_lane<kMirror16>(first), from_lane<kMirror16>(second));
}

// A group's score as a key, and how large (as a positive float's bits) what it is made of is. Two low
// biases may add up to less than fp32 holds: the group is open all the same and must not look like a
// closed one (and infinitely large, it is close to every other).
__device__ __forceinline__ int32_t group_score(const RouteArgs& a, int32_t first, int32_t second, int32_t* size) {
  const bool two = a.group_score == ROUTE_GROUP_TOP2 && second > kNone;
  const float f = unordered(first), s = two ? unordered(second) : 0.0f;
  *size = first > kNone ? __float_as_int(2.0f + fabsf(f) + fabsf(s)) : 0;
  return first > kNone ? ordered(fmaxf(f + s, -kLargest) + 0.0f) : kNone;
}

// V experts a lane; SCORES: keys are scores. group_shift: lanes of a group as a power of two, or
// -1: groups are scored from LDS. lds_bytes: of a wave.
template <int V, bool SCORES>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs a, int group_shift, int lds_bytes) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * waves + wave;
  if (t >= a.T) return;
  uint8_t* const lds = smem + wave * lds_bytes;
  const int E = a.num_experts, G = a.num_groups;
  float l[V], bias[V];
  if (SCORES) load_bias<V>(a, lane * V, 1, bias);
  load_logits<V>(a, t, lane * V, 1, l);
  int32_t key[V];
  // softmax's largest logit and sum, where scores are needed (fp32), or weights that keep the sum
  float top = l[0];
#pragma unroll
  for (int i = 1; i < V; i++) top = fmaxf(top, l[i]);
  top = unordered(wave_max(ordered(top)));
  if (SCORES) {
    float s[V];
    if (a.scoring == ROUTE_SOFTMAX) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; i++) {
        s[i] = l[i] > minus_inf() ? __expf(l[i] - top) : 0.0f;
        sum += s[i];
      }
      const float inverse = 1.0f / wave_sum(sum);
#pragma unroll
      for (int i = 0; i < V; i++) s[i] *= inverse;
    } else {
#pragma unroll
      for (int i = 0; i < V; i++) s[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[i]));
    }
#pragma unroll
    for (int i = 0; i < V; i++)
      key[i] = l[i] > minus_inf() && bias[i] > minus_inf() ? ordered(s[i] + bias[i] + 0.0f) : kNone;
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) key[i] = ordered(l[i]);
  }

  // (the same in all lanes) fp32 scores do not decide; where groups are scored from LDS, they are not asked
  bool near = SCORES && G > 1 && group_shift < 0;
  // whether keys m >= n of experts may be the other way round
  const auto close = [&](int32_t m, int32_t n) {
    const float x = unordered(m), y = unordered(n);
    return !(x - y > near_of(a.scoring, V + 6) * (1.0f + fabsf(x)));
  };
  if (G > 1 && group_shift >= 0) {
    int32_t first = kNone, second = kNone, size;
#pragma unroll
    for (int i = 0; i < V; i++) put(first, second, key[i]);
    group_best2(group_shift, first, second);
    const int32_t mine = group_score(a, first, second, &size);
    const int g = lane >> group_shift;
    int place = 0;
    for (int o = 0; o < G; o++) {
      const int32_t other = __builtin_amdgcn_readlane(mine, o << group_shift);
      place += other > mine || (other == mine && o < g);
    }
    const bool kept = place < a.top_groups;
    if (SCORES && a.top_groups < G) {
      // the least of the kept and the best of the others, and how far scores may be off
      const int32_t least = -wave_max(kept && g < G ? -mine : INT32_MIN);
      const int32_t best = wave_max(!kept && g < G ? mine : INT32_MIN);
      const float off = near_of(a.scoring, V + 6) * __int_as_float(wave_max(size));
      near = best > kNone && !(unordered(least) - unordered(best) > off);
    }
#pragma unroll
    for (int i = 0; i < V; i++) key[i] = kept ? key[i] : kNone;
  } else if (G > 1 && !SCORES) {
    int32_t* const keys = reinterpret_cast<int32_t*>(lds);
    int32_t* const best = keys + E;
#pragma unroll
    for (int i = 0; i < V; i++)
      if (lane * V + i < E) keys[lane * V + i] = key[i];
    wave_lds_fence();
    const int size = E / G;
    for (int g = lane; g < G; g += 64) {
      int32_t first = kNone;
      for (int i = 0; i < size; i++) first = larger(first, keys[g * size + i]);
      best[g] = first;
    }
    wave_lds_fence();
    for (int g = lane; g < G; g += 64) {
      const int32_t mine = best[g];
      int place = 0;
      for (int o = 0; o < G; o++) place += best[o] > mine || (best[o] == mine && o < g);
      if (place >= a.top_groups)
        for (int i = 0; i < size; i++) keys[g * size + i] = kNone;
    }
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < V; i++)
      if (lane * V + i < E) key[i] = keys[lane * V + i];
  }

  int32_t id = -1;
  int32_t last = kNone, last_id = -1;  // the pick before
  // (the one after the last pick is asked for only to see how close it is)
  for (int j = 0; j < a.top_k + (SCORES ? 1 : 0) && !near; j++) {
    int32_t k = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < V; i++) {
      at = key[i] > k ? i : at;
      k = larger(k, key[i]);
    }
    const int32_t m = wave_max(k);
    if (m <= kNone) break;
    const int from = __builtin_ctzll(__ballot(k == m));
    const int e = from * V + __builtin_amdgcn_readlane(at, from);
    if (SCORES) {
      // picks that are equal in logit and bias are in order; behind the next best one, others may be close
      if (j > 0 && close(last, m))
        near = j == a.top_k || logit_of(a, t, e) != logit_of(a, t, last_id) || (a.bias && a.bias[e] != a.bias[last_id]);
      last = m;
      last_id = e;
    }
    if (lane == j && j < a.top_k) id = e;
#pragma unroll
    for (int i = 0; i < V; i++)
      if (lane * V + i == e) key[i] = kNone;
  }
  if (SCORES && near) {
    wave_lds_fence();
    id = decide64<V, true>(a, t, reinterpret_cast<double*>(lds));
  }
  // weights: s of the picks, in 64 bits
  const float mine = id >= 0 ? logit_of(a, t, id) : minus_inf();
  double s = 0.0;
  if (id >= 0) s = a.scoring == ROUTE_SOFTMAX ? exp((double)mine - (double)top) : 1.0 / (1.0 + exp(-(double)mine));
  if (a.renormalize) {
    const double sum = wave_sum(s);
    s = sum > 0.0 ? s / sum : 0.0;
  } else if (a.scoring == ROUTE_SOFTMAX) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; i++) sum += l[i] > minus_inf() ? exp((double)l[i] - (double)top) : 0.0;
    s /= wave_sum(sum);
  }
  if (lane < a.top_k) {
    a.topk_ids[t * a.top_k + lane] = id;
    a.topk_w[t * a.top_k + lane] = id >= 0 ? (float)(s * (double)a.scale) : 0.0f;
  }
}

// Many tokens: 16 lanes to a token, four tokens to a wave. A round's work is then shared by four
// tokens, and so are group scores and the weights, whose 64-bit arithmetic takes the whole wave
// either way. Lane l of a token holds experts i * 16 + l, i < V, sorted by key, so that a round looks
// at one key a lane and the winner's lane moves its list up.
//
// The low bits of a key hold V - 1 - i in place of its own (sorting goes by minimum and maximum of
// one register, and of equal keys the lower i, then the lower lane, is the lower expert). So keys are
// good to 2^-19 of themselves (V = 16): exact for BF16 logits, otherwise `near` counts that in, and
// fp32 logits that are closer are decided by decide64 too, in their own order.
template <int V, bool SCORES>
__global__ __launch_bounds__(256) void moe_route_many(RouteArgs a, int lds_bytes) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, row = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4;
  if (t0 >= a.T) return;
  const bool have = t0 + row < a.T;
  const int64_t t = have ? t0 + row : a.T - 1;
  const int E = a.num_experts, G = a.num_groups;
  const auto row_sum = [](auto v) {
    v += from_lane<kXor1>(v);
    v += from_lane<kXor2>(v);
    v += from_lane<kMirror8>(v);
    return v + from_lane<kMirror16>(v);
  };
  // this token's 16 bits of a ballot
  const auto row_bits = [row](uint64_t m) {
    const uint32_t half = row & 2 ? (uint32_t)(m >> 32) : (uint32_t)m;
    return (row & 1 ? half >> 16 : half) & 0xFFFFu;
  };

  int32_t key[V];
  float l[V], bias[V];
  if (SCORES) load_bias<V>(a, l16, 16, bias);
  load_logits<V>(a, t, l16, 16, l);
  float top = minus_inf();
  if (a.scoring == ROUTE_SOFTMAX) {
    int32_t m = ordered(l[0]);
#pragma unroll
    for (int i = 1; i < V; i++) m = larger(m, ordered(l[i]));
    top = unordered(row_max(m));
  }
  float inverse = 1.0f;  // of softmax's sum
  if (SCORES) {
    float s[V];
    if (a.scoring == ROUTE_SOFTMAX) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; i++) {
        s[i] = l[i] > minus_inf() ? __expf(l[i] - top) : 0.0f;
        sum += s[i];
      }
      inverse = 1.0f / row_sum(sum);
#pragma unroll
      for (int i = 0; i < V; i++) s[i] *= inverse;
    } else {
#pragma unroll
      for (int i = 0; i < V; i++) s[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[i]));
    }
#pragma unroll
    for (int i = 0; i < V; i++)
      key[i] = l[i] > minus_inf() && bias[i] > minus_inf() ? ordered(s[i] + bias[i] + 0.0f) : kNone;
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) key[i] = ordered(l[i]);
  }

  const float off = SCORES ? near_of(a.scoring, V + 4) + 2.0f / 1048576.0f : 0.0f;  // of 1 + magnitudes
  bool near = false;  // (the same in a token's lanes) the keys do not decide
  if (G > 1) {  // 16 divides a group: it is `per` of the lists' places
    const int per = E / G >> 4;
    int32_t mine = INT32_MIN, size = 0;  // lane g: the score of group g
    int32_t first = kNone, second = kNone;
    int g = 0, left = per;
#pragma unroll
    for (int i = 0; i < V; i++) {
      put(first, second, key[i]);
      if (--left == 0 && g < G) {
        group_best2(4, first, second);
        if (l16 == g) mine = first, size = second;
        first = second = kNone;
        g++;
        left = per;
      }
    }
    if (l16 < G) mine = group_score(a, mine, size, &size);
    int place = 0;
    const auto against = [&](int32_t other, int n) {  // that of lane l16 - n (round the 16)
      place += other > mine || (other == mine && l16 >= n);
    };
#define AGAINST(n) against(from_lane<kRotate + n>(mine), n)
    AGAINST(1); AGAINST(2); AGAINST(3); AGAINST(4); AGAINST(5); AGAINST(6); AGAINST(7); AGAINST(8);
    AGAINST(9); AGAINST(10); AGAINST(11); AGAINST(12); AGAINST(13); AGAINST(14); AGAINST(15);
#undef AGAINST
    const bool kept = l16 < G && place < a.top_groups;
    if (SCORES && a.top_groups < G) {
      const int32_t least = -row_max(kept ? -mine : INT32_MIN);
      const int32_t best = row_max(!kept && l16 < G ? mine : INT32_MIN);
      const float most = __int_as_float(row_max(size));
      near = best > kNone && !(unordered(least) - unordered(best) > off * most);
    }
    const uint32_t groups = row_bits(__ballot(kept));
    g = 0, left = per;
#pragma unroll
    for (int i = 0; i < V; i++) {
      key[i] = groups >> g & 1 ? key[i] : kNone;
      if (--left == 0) g++, left = per;
    }
  }
  // keys with their places in the low bits (open ones stay above kNone)
  constexpr int32_t kPlace = V - 1;
#pragma unroll
  for (int i = 0; i < V; i++) key[i] = key[i] > kNone ? (key[i] & ~kPlace) | (V - 1 - i) : kNone;
  // odd-even merge sort, descending
#pragma unroll
  for (int p = 1; p < V; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; i++)
          if (j + i + q < V && (j + i) / (2 * p) == (j + i + q) / (2 * p)) {
            const int32_t x = key[j + i], y = key[j + i + q];
            key[j + i] = larger(x, y);
            key[j + i + q] = x < y ? x : y;
          }

  int32_t id = -1, got = kNone;  // lane j: pick j and its key
  for (int j = 0; j <= a.top_k; j++) {  // the one after the last pick shows how close it is
    const int32_t m = row_max(key[0]);
    const uint32_t bits = row_bits(__ballot(key[0] == m));
    const int from = __builtin_ctz(bits);
    const int e = (V - 1 - (m & kPlace)) * 16 + from;
    if (l16 == j) {
      got = m;
      id = e;
    }
    if (l16 == from) {
#pragma unroll
      for (int i = 0; i + 1 < V; i++) key[i] = key[i + 1];
      key[V - 1] = kNone;
    }
  }
  if (got <= kNone) id = -1;
  // s of the picks (softmax: before its sum) in 64 bits, for the weights and to see whether the picks
  // are in order
  float logit = id >= 0 ? logit_of(a, t, id) : minus_inf();
  const auto score_of = [&](float l) {
    return a.scoring == ROUTE_SOFTMAX ? exp((double)l - (double)top) : 1.0 / (1.0 + exp(-(double)l));
  };
  double s = id >= 0 ? score_of(logit) : 0.0;
  {
    const int32_t before = from_lane<kRotate + 1>(got);
    const float logit_before = from_lane<kRotate + 1>(logit);
    const bool next = l16 == a.top_k;  // behind it there may be others as close: the keys alone count
    bool doubt;
    if (SCORES) {
      const float b = a.bias && id >= 0 ? a.bias[id] : 0.0f, b_before = from_lane<kRotate + 1>(b);
      const float x = unordered(before & ~kPlace), y = unordered(got & ~kPlace);
      const double p = s * (double)inverse, c = p + (double)b;
      const double p_before = from_lane<kRotate + 1>(p), c_before = from_lane<kRotate + 1>(c);
      // `inverse` is an fp32 one
      const double room = (a.scoring == ROUTE_SOFTMAX ? (double)off * fabs(p_before - p) : 0.0) + 1e-14 * (1.0 + fabs(c));
      doubt = next ? !(x - y > off * (1.0f + fabsf(x)))
                   : !(c_before - c > room) && (logit != logit_before || b != b_before);
    } else {
      doubt = next ? a.logits_type != FP8_BF16 && (before & ~kPlace) == (got & ~kPlace) : logit_before < logit;
    }
    near = row_bits(__ballot(near || (l16 > 0 && l16 <= a.top_k && id >= 0 && doubt))) != 0u;
  }
  if (uint64_t undecided = __ballot(near && have && l16 == 0)) {
    for (; undecided; undecided &= undecided - 1) {
      const int r = __builtin_ctzll(undecided) >> 4;
      const int32_t ids = decide64<V / 4, SCORES>(a, t0 + r, reinterpret_cast<double*>(smem + wave * lds_bytes));
      const int32_t other = __shfl(ids, l16, 64);
      if (row == r) id = other;
      wave_lds_fence();
    }
    logit = id >= 0 ? logit_of(a, t, id) : minus_inf();
    s = id >= 0 ? score_of(logit) : 0.0;
  }
  if (l16 >= a.top_k) id = -1;
  s = id >= 0 ? s : 0.0;
  if (a.renormalize) {
    const double sum = row_sum(s);
    s = sum > 0.0 ? s / sum : 0.0;
  } else if (a.scoring == ROUTE_SOFTMAX) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; i++) sum += l[i] > minus_inf() ? exp((double)l[i] - (double)top) : 0.0;
    s /= row_sum(sum);
  }
  if (have && l16 < a.top_k) {
    a.topk_ids[t * a.top_k + l16] = id;
    a.topk_w[t * a.top_k + l16] = id >= 0 ? (float)(s * (double)a.scale) : 0.0f;
  }
}

// From this many tokens on four go to a wave (a wave on each SIMD then). 256 experts, groups and a
// bias, a wave per token against four to a wave: 1024 tokens 9.9 and 11.3 us, 4096 12.6 and 12.7,
// 16384 25.6 and 19.4; 128 experts by softmax, 16384 tokens, 11.6 and 6.2.
constexpr int64_t kManyTokens = 4096;

template <int V, bool SCORES>
hipError_t launch_many(const RouteArgs& a, hipStream_t stream) {
  const int bytes = 8 * (a.num_experts + a.num_groups);
  hipLaunchKernelGGL((moe_route_many<V, SCORES>), dim3((uint32_t)((a.T + 15) / 16)), dim3(256), (size_t)bytes * 4,
                     stream, a, bytes);
  return hipGetLastError();
}

template <int V, bool SCORES>
hipError_t launch(const RouteArgs& a, hipStream_t stream) {
  int shift = -1;
  const int size = a.num_experts / a.num_groups;
  for (int s = 0; s <= 4; s++)
    if (size == V << s) shift = s;
  const int bytes = SCORES ? 8 * (a.num_experts + a.num_groups)
                           : a.num_groups > 1 && shift < 0 ? 4 * (a.num_experts + a.num_groups) : 0;
  const int waves = bytes * 4 <= 32768 ? 4 : 1;
  hipLaunchKernelGGL((moe_route_kernel<V, SCORES>), dim3((uint32_t)((a.T + waves - 1) / waves)), dim3(64 * waves),
                     (size_t)bytes * waves, stream, a, shift, bytes);
  return hipGetLastError();
}

template <bool SCORES>
hipError_t launch_experts(const RouteArgs& a, hipStream_t stream) {
  const int E = a.num_experts;
  if (a.T >= kManyTokens && E <= 256 && a.top_k < 16 && (a.num_groups == 1 || E / a.num_groups % 16 == 0)) {
    if (E <= 64) return launch_many<4, SCORES>(a, stream);
    return E <= 128 ? launch_many<8, SCORES>(a, stream) : launch_many<16, SCORES>(a, stream);
  }
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
