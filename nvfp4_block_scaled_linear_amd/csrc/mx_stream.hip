// MXFP4 products for few activation rows: the weight is streamed once for all of them.
//
// Decode-sized products are bound by the weight's bytes, and a launch that lasts a few
// microseconds by how soon all its loads are in flight. So a workgroup takes 16 * NT weight
// rows (SwiGLU: gate rows and the up rows that belong to them) and its W waves split K into
// runs of 128-k steps; a wave keeps a ring of U steps of loads in registers, and the waves'
// partial sums meet in LDS and are added in wave order, so results do not depend on timing.
//
// A step of a 16-row tile is one 16-byte load of codes per lane: lane l = c + 16g holds block
// g (32 k) of row c, so that a row's 64 bytes are read by neighbouring lanes.
//  - MXFP4 activations: the activation rows are loaded alike and one scaled MFMA does the step.
//  - BF16 activations: MFMA j covers block j, lane (c, g) holding k = 8g + [0, 8) of it, so that
//    the activations' loads run along their rows (64 bytes of a row per instruction); the
//    codes are brought into that order by a 4 x 4 transpose of dwords between the lanes of a
//    row, four lane swaps a step.
// Loads are buffer loads, out of range (zeros, no memory touched) past the rows, past K and
// past a wave's run, so no branch stands around them.
#include "mx_device.hpp"
#include "mx_kernels.hpp"

namespace nvfp4 {
namespace {

constexpr uint32_t kOOB = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0,
                                           (int)(bytes > 0x7FFFFFFF ? 0x7FFFFFFF : bytes), 0x00020000);
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// scale bytes of a step and row: one dword when DW (K % 128 == 0 and dword-aligned scales),
// otherwise one byte load per block that the lane needs
template <int ACT, int TM, int NT>
struct Step {
  u32x4 w[NT], x[TM][ACT == MXFP4_ACT_BF16 ? 4 : 1];
  uint32_t ws[NT], xs[TM];
};

template <int ACT_, int TM_, int NT_, int W_, int U_, bool DW_>
struct Cfg {
  static constexpr int ACT = ACT_, TM = TM_, NT = NT_, W = W_, U = U_;
  static constexpr bool DW = DW_, MX = ACT_ == MXFP4_ACT_MXFP4;
};

template <class C, bool GROUPED, int SWIGLU>
__global__ __launch_bounds__(64 * C::W) void mx_stream(MxArgs a) {
  constexpr int NO = SWIGLU ? C::NT / 2 : C::NT;  // 16-column tiles of output
  static_assert(SWIGLU != MXFP4_OUT_SWIGLU_MXFP4 || NO % 2 == 0, "whole blocks of 32 columns");
  extern __shared__ __attribute__((aligned(16))) f32x4 part[];  // [W][NT][TM][64]
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t N = a.N, K = a.K, half = N >> 1;
  const int64_t cols = SWIGLU ? half : N;
  const int nb = (int)(K >> 5);
  const int64_t nbn = (cols + 16 * NO - 1) / (16 * NO);
  const int64_t n0 = (blockIdx.x % nbn) * (16 * NO);
  const uint8_t* wc = a.w_codes;
  const uint8_t* wsc = a.w_scales;
  int beg = 0, end = (int)a.M;
  const int32_t* rec = nullptr;
  if (SWIGLU == MXFP4_OUT_SWIGLU_MXFP4) {
    // scales of dropped routes, shared out over the launch (the grouping clears their codes)
    const int64_t bytes = N >> 6;
    for (int64_t r = (int64_t)blockIdx.x * blockDim.x + tid; r < a.R; r += (int64_t)gridDim.x * blockDim.x)
      if (a.route_expert[r] < 0)
        for (int64_t b = 0; b < bytes; b++) a.y_scales[r * bytes + b] = 0;
  }
  if (GROUPED) {
    rec = a.slots + kSlotInts * (blockIdx.x / nbn);
    const int e = rec[0];
    if (e < 0) return;
    beg = rec[1];
    end = rec[2];
    wc += (int64_t)e * N * (K >> 1);
    wsc += (int64_t)e * N * nb;
  }
  // weight rows of this lane, from the tile's first row (SwiGLU: from the weight's)
  const int64_t r0 = SWIGLU ? 0 : n0;
  const auto wr = rsrc_of(wc + r0 * (K >> 1), (N - r0) * (K >> 1));
  const auto wsr = rsrc_of(wsc + r0 * nb, (N - r0) * nb);
  uint32_t wo[C::NT], wso[C::NT];
#pragma unroll
  for (int t = 0; t < C::NT; t++) {
    const int64_t n = n0 + 16 * (t % NO) + c;
    const int64_t row = n - r0 + (t >= NO ? half : 0);
    wo[t] = n < cols ? (uint32_t)(row * (K >> 1)) + 16 * g : kOOB;
    wso[t] = n < cols ? (uint32_t)(row * nb) : kOOB;
  }
  // this wave's steps, a run of an even number (two steps are one 128-byte line of codes)
  const int steps = (nb + 3) >> 2;
  const int per = ((steps + 2 * C::W - 1) / (2 * C::W)) * 2;
  const int s0 = wave * per, s1 = s0 + per < steps ? s0 + per : steps;
  const int64_t xpitch = C::MX ? K >> 1 : a.ldx * 2;
  const auto xr = rsrc_of(a.x, (a.x_rows - 1) * xpitch + (C::MX ? K >> 1 : 2 * K));
  const auto xsr = C::MX ? rsrc_of(a.x_scales, a.x_rows * nb) : xr;

  for (int p0 = beg; p0 < end; p0 += 16 * C::TM) {
    uint32_t xo[C::TM], xso[C::TM];
#pragma unroll
    for (int x = 0; x < C::TM; x++) {
      const int p = p0 + 16 * x + c;
      int64_t row = p;
      if (GROUPED && p < end) {
        const int32_t route = p - beg < rec[3] ? rec[4 + p - beg] : a.sorted[p];
        row = a.rows_per_token ? route / a.top_k : route;
      }
      xo[x] = p < end ? (uint32_t)(row * xpitch) + 16 * g : kOOB;
      xso[x] = p < end ? (uint32_t)(row * nb) : kOOB;
    }
    const auto load = [&](Step<C::ACT, C::TM, C::NT>& b, int s) {
      const bool in = s < s1;
      const bool mine = in && 4 * s + g < nb;  // this lane's block of codes
#pragma unroll
      for (int t = 0; t < C::NT; t++) {
        b.w[t] = __builtin_amdgcn_raw_buffer_load_b128(wr, mine ? wo[t] + 64 * s : kOOB, 0, 0);
        if (C::DW) {
          b.ws[t] = __builtin_amdgcn_raw_buffer_load_b32(wsr, in ? wso[t] + 4 * s : kOOB, 0, 0);
        } else if (C::MX) {
          b.ws[t] = __builtin_amdgcn_raw_buffer_load_b8(wsr, mine ? wso[t] + 4 * s + g : kOOB, 0, 0);
        } else {
          uint32_t v = 0u;
#pragma unroll
          for (int j = 0; j < 4; j++)
            v |= (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
                     wsr, in && 4 * s + j < nb ? wso[t] + 4 * s + j : kOOB, 0, 0) << (8 * j);
          b.ws[t] = v;
        }
      }
#pragma unroll
      for (int x = 0; x < C::TM; x++) {
        if (C::MX) {
          b.x[x][0] = __builtin_amdgcn_raw_buffer_load_b128(xr, mine ? xo[x] + 64 * s : kOOB, 0, 0);
          if (C::DW)
            b.xs[x] = __builtin_amdgcn_raw_buffer_load_b32(xsr, in ? xso[x] + 4 * s : kOOB, 0, 0);
          else
            b.xs[x] = __builtin_amdgcn_raw_buffer_load_b8(xsr, mine ? xso[x] + 4 * s + g : kOOB, 0, 0);
        } else {
#pragma unroll
          for (int j = 0; j < 4; j++)
            b.x[x][j] = __builtin_amdgcn_raw_buffer_load_b128(
                xr, in && 4 * s + j < nb ? xo[x] + 256 * s + 64 * j : kOOB, 0, 0);
        }
      }
    };

    f32x4 acc[C::NT][C::TM];
#pragma unroll
    for (int t = 0; t < C::NT; t++)
#pragma unroll
      for (int x = 0; x < C::TM; x++) acc[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
    const auto compute = [&](Step<C::ACT, C::TM, C::NT>& b) {
      if (C::MX) {
        const int sh = C::DW ? 8 * g : 0;
#pragma unroll
        for (int t = 0; t < C::NT; t++)
#pragma unroll
          for (int x = 0; x < C::TM; x++)
            acc[t][x] = mfma_mx(b.w[t], b.x[x][0], acc[t][x], b.ws[t] >> sh, b.xs[x] >> sh);
      } else {
#pragma unroll
        for (int t = 0; t < C::NT; t++) {
          transpose4(b.w[t]);
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const u32x4 w = mx_decode8(b.w[t][j], e8m0_operand((b.ws[t] >> (8 * j)) & 0xFFu));
#pragma unroll
            for (int x = 0; x < C::TM; x++) acc[t][x] = mfma16(w, b.x[x][j], acc[t][x]);
          }
        }
      }
    };

    if (s0 < s1) {
      Step<C::ACT, C::TM, C::NT> ring[C::U];
#pragma unroll
      for (int u = 0; u < C::U; u++) load(ring[u], s0 + u);
      int s = s0;
      for (; s + C::U < s1; s += C::U) {
#pragma unroll
        for (int u = 0; u < C::U; u++) {
          compute(ring[u]);
          load(ring[u], s + C::U + u);
        }
      }
#pragma unroll
      for (int u = 0; u < C::U; u++) compute(ring[u]);
    }

    if (GROUPED && p0 != beg) __syncthreads();  // the last pass's partial sums have been read
#pragma unroll
    for (int t = 0; t < C::NT; t++)
#pragma unroll
      for (int x = 0; x < C::TM; x++) part[((wave * C::NT + t) * C::TM + x) * 64 + lane] = acc[t][x];
    __syncthreads();
    const auto total = [&](int t, int x, int l) {
      f32x4 v = part[(t * C::TM + x) * 64 + l];
#pragma unroll
      for (int w = 1; w < C::W; w++) v += part[((w * C::NT + t) * C::TM + x) * 64 + l];
      return v;
    };
    // an item: four columns per lane of a 16 x 16 tile (MXFP4: of two, which make a block)
    constexpr int TS = SWIGLU == MXFP4_OUT_SWIGLU_MXFP4 ? 2 : 1;
    for (int i = wave; i < NO / TS * C::TM; i += C::W) {
      const int t = i % (NO / TS) * TS, x = i / (NO / TS);
      const int p = p0 + 16 * x + c;
      const bool ok = p < end;
      int64_t row = p;
      if (GROUPED) row = !ok ? 0 : p - beg < rec[3] ? rec[4 + p - beg] : a.sorted[p];
      const int64_t n = n0 + 16 * t + 4 * g;
      const f32x4 v = total(t, x, lane);
      if (!SWIGLU) {
        if (!ok) continue;
#pragma unroll
        for (int q = 0; q < 4; q++) {
          if (n + q >= N) continue;
          if (a.y_type == MXFP4_F32)
            static_cast<float*>(a.y)[row * a.ldy + n + q] = v[q];
          else
            static_cast<uint16_t*>(a.y)[row * a.ldy + n + q] = (uint16_t)bf16_pair(v[q], 0.f);
        }
        continue;
      }
      const f32x4 u = total(NO + t, x, lane);
      const uint32_t h[2] = {bf16_pair(silu(v[0]) * u[0], silu(v[1]) * u[1]),
                             bf16_pair(silu(v[2]) * u[2], silu(v[3]) * u[3])};
      if (SWIGLU == MXFP4_OUT_SWIGLU_BF16) {
#pragma unroll
        for (int q = 0; q < 4; q++)
          if (ok && n + q < half)
            static_cast<uint16_t*>(a.y)[row * half + n + q] = (uint16_t)(h[q >> 1] >> (16 * (q & 1)));
        continue;
      }
      const f32x4 v1 = total(t + 1, x, lane), u1 = total(NO + t + 1, x, lane);
      const uint32_t k[4] = {h[0], h[1], bf16_pair(silu(v1[0]) * u1[0], silu(v1[1]) * u1[1]),
                             bf16_pair(silu(v1[2]) * u1[2], silu(v1[3]) * u1[3])};
      uint32_t amax = 0u;
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const uint32_t lo = (k[q] & 0x7FFFu) << 16, hi = k[q] & 0x7FFF0000u;
        amax = amax > lo ? amax : lo;
        amax = amax > hi ? amax : hi;
      }
      uint32_t o = __shfl_xor(amax, 16, 64);
      amax = amax > o ? amax : o;
      o = __shfl_xor(amax, 32, 64);
      amax = amax > o ? amax : o;
      const uint32_t sc = e8m0_of_amax(amax);
      const bool bad = amax >= 0x7F800000u;
      if (!ok || n >= half) continue;  // blocks end where the columns do
#pragma unroll
      for (int q = 0; q < 2; q++) {
        float f[4];
#pragma unroll
        for (int j = 0; j < 2; j++) {
          f[2 * j] = __builtin_ldexpf(__uint_as_float(k[2 * q + j] << 16), 127 - (int)sc);
          f[2 * j + 1] = __builtin_ldexpf(__uint_as_float(k[2 * q + j] & 0xFFFF0000u), 127 - (int)sc);
        }
        const uint32_t code = e2m1_rne2<1>(e2m1_rne2<0>(0u, f[0], f[1]), f[2], f[3]);
        *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a.y) + row * (half >> 1) + ((n + 16 * q) >> 1)) =
            bad ? 0 : (uint16_t)code;
      }
      if (g == 0) a.y_scales[row * (half >> 5) + (n >> 5)] = (uint8_t)(bad ? kE8M0Nan : sc);
    }
    if (!GROUPED) return;  // dense: M <= 16 * TM
  }
}

template <class C>
hipError_t launch_cfg(const MxArgs& a, int64_t max_slots, hipStream_t stream) {
  const int64_t no = a.swiglu ? C::NT / 2 : C::NT;
  const int64_t cols = a.swiglu ? a.N >> 1 : a.N;
  const int64_t groups = (cols + 16 * no - 1) / (16 * no) * (a.slots ? max_slots : 1);
  if (groups * 64 * C::W > (int64_t)UINT32_MAX) return hipErrorInvalidConfiguration;
  const size_t lds = sizeof(f32x4) * 64 * C::W * C::NT * C::TM;
  auto k = !a.slots ? mx_stream<C, false, 0> : mx_stream<C, true, 0>;
  if constexpr (C::NT == 4) {
    if (a.swiglu)
      k = a.swiglu == MXFP4_OUT_SWIGLU_BF16 ? mx_stream<C, true, MXFP4_OUT_SWIGLU_BF16>
                                            : mx_stream<C, true, MXFP4_OUT_SWIGLU_MXFP4>;
  }
  hipLaunchKernelGGL(k, dim3((uint32_t)groups), dim3(64 * C::W), lds, stream, a);
  return hipGetLastError();
}

template <int ACT, int TM, int NT, int U>
hipError_t launch_rows(const MxArgs& a, bool dw, int64_t max_slots, hipStream_t stream) {
  if (a.K >= 2048) {
    return dw ? launch_cfg<Cfg<ACT, TM, NT, 8, U, true>>(a, max_slots, stream)
              : launch_cfg<Cfg<ACT, TM, NT, 8, U, false>>(a, max_slots, stream);
  }
  return dw ? launch_cfg<Cfg<ACT, TM, NT, 4, U, true>>(a, max_slots, stream)
            : launch_cfg<Cfg<ACT, TM, NT, 4, U, false>>(a, max_slots, stream);
}

template <int ACT>
hipError_t launch_act(const MxArgs& a, int64_t rows, int64_t max_slots, hipStream_t stream) {
  const bool dw = a.K % 128 == 0 && ((uintptr_t)a.w_scales | (uintptr_t)a.x_scales) % 4 == 0;
  if (a.swiglu) return launch_rows<ACT, 1, 4, 2>(a, dw, max_slots, stream);
  if (rows <= 16) return launch_rows<ACT, 1, 2, 4>(a, dw, max_slots, stream);
  if (rows <= 32) return launch_rows<ACT, 2, 2, 2>(a, dw, max_slots, stream);
  return launch_rows<ACT, 4, 2, 2>(a, dw, max_slots, stream);
}

}  // namespace

bool mx_stream_takes(const MxArgs& a, int act_kind) {
  // 32-bit offsets into the activations and one weight
  const int64_t pitch = act_kind == MXFP4_ACT_MXFP4 ? a.K >> 1 : a.ldx * 2;
  return a.x_rows * pitch < (int64_t)kOOB && a.N * (a.K >> 1) < (int64_t)kOOB;
}

hipError_t launch_mx_stream(const MxArgs& a, int act_kind, int64_t rows, int64_t max_slots,
                            hipStream_t stream) {
  return act_kind == MXFP4_ACT_BF16 ? launch_act<MXFP4_ACT_BF16>(a, rows, max_slots, stream)
                                    : launch_act<MXFP4_ACT_MXFP4>(a, rows, max_slots, stream);
}

}  // namespace nvfp4
