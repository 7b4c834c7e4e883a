// MXFP4 products for few activation rows: the weight is streamed once for all of them.
//
// Decode-sized products are bound by the weight's bytes, and a launch of a few microseconds by
// how soon its loads are in flight and how few cache lines they look up. A workgroup takes
// 16 * NT weight rows (SwiGLU: gate rows and the up rows that belong to them); its W waves
// split K into runs of 128-k steps, each through an LDS ring of its own that holds U steps of
// both operands, so no wave waits for another before the end, when their partial sums are
// added in wave order (results do not depend on timing).
//
// The MFMA wants 16 consecutive lanes on 16 different rows. Loaded into registers like that, a
// load looks up a cache line per lane; loads into LDS (lds_load) take the rows as they lie,
// four lanes to a row's 64 bytes of codes, 16 lanes to its 256 bytes of BF16, and the LDS reads
// bring the operands into order. Row r's 16-byte piece q lies at slot q ^ f(r), so that the 16
// rows that lanes read together fall into different banks.
//  - MXFP4 activations: one scaled MFMA over the step per 16 weight rows.
//  - BF16 activations: lane (c, g) = c + 16g decodes the 32 codes of block g of its row with the
//    block's scale, and MFMA j is over k = 32g + 8j + [0, 8).
// Loads past the rows, past K and past a wave's run are out of range: every step issues the
// same number, which is what the counted waits go by.
//
// With weights from HBM, 16 x 12288 x 4096 with BF16 activations takes 10.5 us (27 MB, 2.5 TB/s; a
// plain read of the codes 5.6), 1 x 2048 x 2048 3.9, 4 x 4096 x 4096 with MXFP4 ones 4.7 (a plain
// read 3.0); with weights that the last-level cache holds 8.8, 3.2 and 3.9. Of a layer of 128
// experts, top-8, for 16 tokens, gate_up (2048 -> 2 x 768) takes 36.4 us and down (768 -> 2048)
// 19.7: 3.7 and 3.4 TB/s of the routed experts' weights, in thousands of workgroups that live a
// few microseconds each, much of that the time to their first load. Rings of several column blocks
// per workgroup and prefetches into L2 were slower.
#include "mx_device.hpp"
#include "mx_kernels.hpp"
#include "mx_routes.hpp"

namespace nvfp4 {
namespace {

// XR activation rows (4, or TM tiles of 16), NT tiles of 16 weight rows, W waves, U steps in
// the ring; DW: a row's four scale bytes of a step are loaded as one dword (K % 128 == 0 and
// dword-aligned scales), otherwise a byte per lane
template <int ACT_, int XR_, int NT_, int W_, int U_, bool DW_>
struct Cfg {
  static constexpr int ACT = ACT_, XR = XR_, TM = (XR_ + 15) / 16, NT = NT_, W = W_, U = U_;
  static constexpr bool DW = DW_, MX = ACT_ == MXFP4_ACT_MXFP4;
  static constexpr int XMAX = MX ? TM : XR / 4;  // 1 KiB loads of activations a step
  static constexpr int SW = DW ? 1 : NT, SX = MX ? (DW ? 1 : TM) : 0;  // loads of scales
  static constexpr int W0 = 0, X0 = 1024 * NT, S0 = X0 + 1024 * XMAX, STEP = S0 + 256 * (SW + SX);
  static constexpr int RING = STEP * U;                // of a wave
  static constexpr int PART = 1024 * NT * TM;          // partial sums of a wave
  static constexpr int LDS = W * (RING > PART ? RING : PART);
  static_assert(NT <= 4 && TM <= 4 && LDS <= 160 * 1024, "");
};

// slot of piece q of a 64-byte row is q ^ code_swizzle(row), of a 256-byte one piece_slot(q) ^
// row % 16: a 16-byte LDS read takes rows 0..3 and 12..15 of lanes with one g and rows 4..11 of
// those with the next one together
__device__ __forceinline__ int code_swizzle(int row) {
  const int a = (row >> 2) & 3;
  return ((a & 1) << 1) ^ ((a >> 1) * 3);
}
__device__ __forceinline__ int piece_slot(int q) { return (q & 3) << 2 | q >> 2; }  // its own inverse

struct Operands {
  u32x4 w, ws, x, xs;  // descriptors
};

// One wave's run [s0, s1) of K steps over the rows whose lanes' offsets are xo / xso.
template <class C>
__device__ __forceinline__ void run_steps(const Operands& d, uint32_t ring, const uint8_t* ring_p,
                                          int s0, int s1, int nb, const uint32_t* wo,
                                          const uint32_t* wso, const uint32_t* xo,
                                          const uint32_t* xso, f32x4 (&acc)[C::NT][C::TM]) {
  constexpr int XI = C::XMAX, LOADS = C::NT + XI + C::SW + C::SX;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  // this lane's block of a load of codes, and its 16-byte piece of a load of BF16 rows
  const int wq = (lane & 3) ^ code_swizzle(lane >> 2);
  const auto issue = [&](int s, int u) {
    const uint32_t base = ring + u * C::STEP;
    const bool in = s < s1;
    const uint32_t w_at = in && 4 * s + wq < nb ? 64 * s : kOutOfRange;
#pragma unroll
    for (int t = 0; t < C::NT; t++)
      lds_load<16>(d.w, w_at == kOutOfRange ? kOutOfRange : wo[t] + w_at, base + C::W0 + 1024 * t);
#pragma unroll
    for (int i = 0; i < XI; i++) {
      uint32_t off;
      if (C::MX) {
        off = w_at == kOutOfRange ? kOutOfRange : xo[i] + w_at;
      } else {
        const int q = piece_slot((lane & 15) ^ ((4 * i + (lane >> 4)) & 15));  // of the row's 16
        off = in && 4 * s + (q >> 2) < nb ? xo[i] + 256 * s : kOutOfRange;
      }
      lds_load<16>(d.x, off, base + C::X0 + 1024 * i);
    }
    if (C::DW) {
      lds_load<4>(d.ws, in ? wso[0] + 4 * s : kOutOfRange, base + C::S0);
      if (C::MX) lds_load<4>(d.xs, in ? xso[0] + 4 * s : kOutOfRange, base + C::S0 + 256);
    } else {
      const bool sin = in && 4 * s + (lane & 3) < nb;
#pragma unroll
      for (int t = 0; t < C::NT; t++)
        lds_load<1>(d.ws, sin ? wso[t] + 4 * s : kOutOfRange, base + C::S0 + 256 * t);
#pragma unroll
      for (int x = 0; x < C::SX; x++)
        lds_load<1>(d.xs, sin ? xso[x] + 4 * s : kOutOfRange, base + C::S0 + 256 * (C::SW + x));
    }
  };
#pragma unroll
  for (int u = 0; u < C::U - 1; u++) issue(s0 + u, u);
  int u = 0;
  for (int s = s0; s < s1; s++) {
    wait_lds_reads();  // of the step whose bytes the next loads overwrite
    issue(s + C::U - 1, u == 0 ? C::U - 1 : u - 1);
    wait_loads<(C::U - 1) * LOADS>();
    const uint8_t* b = ring_p + u * C::STEP;
    // scale byte of block g of row `row` (of the weight, or behind SW loads of the activations)
    const auto scale = [&](int side, int row) -> uint32_t {
      const uint8_t* p = b + C::S0 + 256 * side;
      return C::DW ? p[4 * row + g] : p[16 * row + 4 * g];
    };
    if (C::MX) {
      u32x4 xf[C::TM];
      uint32_t xs[C::TM];
#pragma unroll
      for (int x = 0; x < C::TM; x++) {
        xf[x] = *reinterpret_cast<const u32x4*>(b + C::X0 + 1024 * x + 64 * c + ((g ^ code_swizzle(c)) << 4));
        xs[x] = scale(C::SW, 16 * x + c);
      }
#pragma unroll
      for (int t = 0; t < C::NT; t++) {
        const u32x4 wf = *reinterpret_cast<const u32x4*>(b + C::W0 + 1024 * t + 64 * c + ((g ^ code_swizzle(c)) << 4));
        const uint32_t ws = scale(0, 16 * t + c);
#pragma unroll
        for (int x = 0; x < C::TM; x++) acc[t][x] = mfma_mx(wf, xf[x], acc[t][x], ws, xs[x]);
      }
    } else {
      u32x4 xf[C::TM][4];
#pragma unroll
      for (int x = 0; x < C::TM; x++) {
        // rows past the loaded ones read others' values, into columns that nobody stores
        const int r = (16 * x + c) % (4 * XI);
#pragma unroll
        for (int j = 0; j < 4; j++)
          xf[x][j] = *reinterpret_cast<const u32x4*>(b + C::X0 + 256 * r + (((g + 4 * j) ^ (r & 15)) << 4));
      }
#pragma unroll
      for (int t = 0; t < C::NT; t++) {
        const u32x4 wf = *reinterpret_cast<const u32x4*>(b + C::W0 + 1024 * t + 64 * c + ((g ^ code_swizzle(c)) << 4));
        const float ws = e8m0_operand(scale(0, 16 * t + c));
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const u32x4 w = mx_decode8(wf[j], ws);
#pragma unroll
          for (int x = 0; x < C::TM; x++) acc[t][x] = mfma16(w, xf[x][j], acc[t][x]);
        }
      }
    }
    u = u + 1 == C::U ? 0 : u + 1;
  }
  wait_loads<0>();
}

template <class C, int MODE, int SWIGLU>
__global__ __launch_bounds__(64 * C::W) void mx_stream(MxArgs a) {
  constexpr bool GROUPED = MODE != kDense;
  constexpr int NO = SWIGLU ? C::NT / 2 : C::NT;  // 16-column tiles of output
  static_assert(SWIGLU != MXFP4_OUT_SWIGLU_MXFP4 || NO % 2 == 0, "whole blocks of 32 columns");
  static_assert(!GROUPED || C::TM == 1, "a grouped pass has at most 16 rows");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  __shared__ int32_t route_list[C::W][16];  // the pass's routes, a copy for each wave
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // sizes below 2^31 (a weight's bytes too): 32-bit arithmetic
  const int N = (int)a.N, half = N >> 1, cols = SWIGLU ? half : N;
  const int nb = (int)(a.K >> 5), wpitch = 16 * nb;
  const uint32_t nbn = (cols + 16 * NO - 1) / (16 * NO);
  const int group = (int)(blockIdx.x / nbn);
  const int n0 = (int)(blockIdx.x - group * nbn) * (16 * NO);
  const uint8_t* wc = a.w_codes;
  const uint8_t* wsc = a.w_scales;
  // dense: groups are runs of XR rows; byExpert: the kept routes in places [begin, count); bySlot:
  // count routes, `first` on in `sorted`
  int count = 0, begin = 0, first = 0, e = 0;
  int32_t my_route = 0;                    // bySlot: routes of the first pass
  uint64_t kept[kScanRoutes / 64];
  const int row0 = MODE == kDense ? group * C::XR : 0;
  if (MODE == kDense) count = (int)a.M - row0 < C::XR ? (int)a.M - row0 : C::XR;
  if (MODE == kByExpert) {
    drop_routes<SWIGLU>(a);
    if (!scan_routes(a.ids, (int)a.R, a.top_k, a.num_experts, group, reinterpret_cast<int32_t*>(smem), &e,
                     &begin, &count, kept))
      return;
  }
  if (MODE == kBySlot) {
    clear_dropped<SWIGLU>(a);
    if (group < a.max_slots) {
      const int32_t v = lane < kSlotInts ? a.slots[(int64_t)kSlotInts * group + lane] : 0;
      e = __builtin_amdgcn_readlane(v, 0);
      if (e < 0) return;
      e = in_experts(a, e);
      first = __builtin_amdgcn_readlane(v, 1);
      count = run_length(a, first, __builtin_amdgcn_readlane(v, 2), kMxSlotRoutes);
      const int n = __builtin_amdgcn_readlane(v, 3);
      my_route = __shfl(v, 4 + c, 64);
      if (n < count && c >= n && c < count) my_route = a.sorted[first + c];
    } else {
      const int tile = group - a.max_slots;
      if (tile >= *a.n_tiles) return;
      e = in_experts(a, a.tiles[2 * tile]);
      first = a.tiles[2 * tile + 1];
      count = run_length(a, first, a.offsets[e + 1], kMxSlotRoutes);
      my_route = c < count ? a.sorted[first + c] : 0;
    }
  }
  if (GROUPED) {
    wc += (int64_t)e * N * wpitch;
    wsc += (int64_t)e * N * nb;
  }
  Operands d;
  const int r0 = SWIGLU ? 0 : n0;  // weight row that the offsets count from
  d.w = lds_load_rsrc(wc + (int64_t)r0 * wpitch, (int64_t)(N - r0) * wpitch);
  d.ws = lds_load_rsrc(wsc + (int64_t)r0 * nb, (int64_t)(N - r0) * nb);
  const uint32_t xpitch = C::MX ? wpitch : (uint32_t)a.ldx * 2;
  const int64_t x_rows = GROUPED ? a.x_rows : count;
  d.x = lds_load_rsrc(static_cast<const uint8_t*>(a.x) + (int64_t)row0 * xpitch,
                      (x_rows - 1) * xpitch + (C::MX ? wpitch : 4 * wpitch));
  d.xs = C::MX ? lds_load_rsrc(a.x_scales + (int64_t)row0 * nb, x_rows * nb) : d.x;
  // row i of weight tile t, from r0, or -1
  const auto w_row = [&](int t, int i) {
    const int n = n0 + 16 * (t % NO) + i;
    return n < cols ? n - r0 + (t >= NO ? half : 0) : -1;
  };
  const int wq = (lane & 3) ^ code_swizzle(lane >> 2);
  uint32_t wo[C::NT], wso[C::SW];
#pragma unroll
  for (int t = 0; t < C::NT; t++) {
    const int row = w_row(t, lane >> 2);
    wo[t] = row >= 0 ? (uint32_t)row * wpitch + 16 * wq : kOutOfRange;
    if (!C::DW) wso[t] = row >= 0 ? (uint32_t)row * nb + (lane & 3) : kOutOfRange;
  }
  if (C::DW) {
    const int row = (lane >> 4) < C::NT ? w_row(lane >> 4, c) : -1;
    wso[0] = row >= 0 ? (uint32_t)row * nb : kOutOfRange;
  }
  // this wave's steps: a run of an even number (two steps are one 128-byte line of codes)
  const int steps = (nb + 3) >> 2;
  const int per = ((steps + 2 * C::W - 1) / (2 * C::W)) * 2;
  const int s0 = wave * per, s1 = s0 + per < steps ? s0 + per : steps;
  constexpr int WAVE = C::LDS / C::W;
  const uint8_t* ring_p = smem + wave * WAVE;
  const uint32_t ring = lds_address(smem) + wave * WAVE;

  for (int p0 = begin; p0 < count; p0 += C::XR) {
    const int rows = count - p0 < C::XR ? count - p0 : C::XR;
    int32_t* const list = route_list[wave];
    if (MODE == kBySlot) {
      if (lane < 16 && lane >= p0 && lane - p0 < rows) list[lane - p0] = my_route;
    }
    if (MODE == kByExpert) {
      int before = 0;
#pragma unroll
      for (int i = 0; i < kScanRoutes / 64; i++) {
        const int at = before + __builtin_popcountll(kept[i] & ((1ull << lane) - 1)) - p0;
        if ((kept[i] >> lane & 1) && at >= 0 && at < rows) list[at] = 64 * i + lane;
        before += __builtin_popcountll(kept[i]);
      }
    }
    if (GROUPED) __builtin_amdgcn_wave_barrier();
    // output row of the pass's i-th row (from row0), and its x row or -1
    const auto y_row = [&](int i) { return GROUPED ? list[i] : p0 + i; };
    const auto x_row = [&](int i) {
      if (i >= rows) return -1;
      const int r = y_row(i);
      return GROUPED && a.rows_per_token ? (int)((uint32_t)r / (uint32_t)a.top_k) : r;
    };
    uint32_t xo[C::XMAX], xso[C::SX > 0 ? C::SX : 1];
#pragma unroll
    for (int i = 0; i < C::XMAX; i++) {
      const int row = x_row(C::MX ? 16 * i + (lane >> 2) : 4 * i + (lane >> 4));
      const int q = C::MX ? wq : piece_slot((lane & 15) ^ ((4 * i + (lane >> 4)) & 15));
      xo[i] = row >= 0 ? (uint32_t)row * xpitch + 16 * q : kOutOfRange;
      if (C::MX && !C::DW) xso[i] = row >= 0 ? (uint32_t)row * nb + (lane & 3) : kOutOfRange;
    }
    if (C::MX && C::DW) {
      const int row = (lane >> 4) < C::TM ? x_row(lane) : -1;
      xso[0] = row >= 0 ? (uint32_t)row * nb : kOutOfRange;
    }
    f32x4 acc[C::NT][C::TM];
#pragma unroll
    for (int t = 0; t < C::NT; t++)
#pragma unroll
      for (int x = 0; x < C::TM; x++) acc[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (s0 < s1) run_steps<C>(d, ring, ring_p, s0, s1, nb, wo, wso, xo, xso, acc);
    // partial sums of this wave [NT][TM][64], in the bytes of its ring
    const auto part = [&](int w) { return reinterpret_cast<f32x4*>(smem + w * WAVE); };
#pragma unroll
    for (int t = 0; t < C::NT; t++)
#pragma unroll
      for (int x = 0; x < C::TM; x++) part(wave)[(t * C::TM + x) * 64 + lane] = acc[t][x];
    __syncthreads();
    const auto total = [&](int t, int x) {
      f32x4 v = part(0)[(t * C::TM + x) * 64 + lane];
#pragma unroll
      for (int w = 1; w < C::W; w++) v += part(w)[(t * C::TM + x) * 64 + lane];
      return v;
    };
    // an item: four columns per lane of a 16 x 16 tile (MXFP4: of two, which make a block)
    constexpr int TS = SWIGLU == MXFP4_OUT_SWIGLU_MXFP4 ? 2 : 1;
    for (int i = wave; i < NO / TS * C::TM; i += C::W) {
      const int t = i % (NO / TS) * TS, x = i / (NO / TS);
      const bool ok = 16 * x + c < rows;
      int64_t row = 0;
      if (ok) row = MODE == kBySlot ? in_routes(a, y_row(16 * x + c)) : row0 + y_row(16 * x + c);
      const int n = n0 + 16 * t + 4 * g;
      const f32x4 v = total(t, x);
      if (!SWIGLU) {
        if (!ok) continue;
        const int64_t at = row * a.ldy + n;
        if (a.y_type == MXFP4_F32) {
          float* y = static_cast<float*>(a.y) + at;
          if (n + 4 <= N && ((uintptr_t)y & 15) == 0) {
            *reinterpret_cast<f32x4*>(y) = v;
          } else {
#pragma unroll
            for (int q = 0; q < 4; q++)
              if (n + q < N) y[q] = v[q];
          }
        } else {
          uint16_t* y = static_cast<uint16_t*>(a.y) + at;
          const uint2 b = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
          if (n + 4 <= N && ((uintptr_t)y & 7) == 0) {
            *reinterpret_cast<uint2*>(y) = b;
          } else {
#pragma unroll
            for (int q = 0; q < 4; q++)
              if (n + q < N) y[q] = (uint16_t)((q < 2 ? b.x : b.y) >> (16 * (q & 1)));
          }
        }
        continue;
      }
      uint32_t h[2 * TS];
#pragma unroll
      for (int k = 0; k < TS; k++) {
        const f32x4 gt = k ? total(t + k, x) : v, u = total(NO + t + k, x);
        h[2 * k] = bf16_pair(silu(gt[0]) * u[0], silu(gt[1]) * u[1]);
        h[2 * k + 1] = bf16_pair(silu(gt[2]) * u[2], silu(gt[3]) * u[3]);
      }
      if (SWIGLU == MXFP4_OUT_SWIGLU_BF16) {
#pragma unroll
        for (int q = 0; q < 4; q++)
          if (ok && n + q < half)
            static_cast<uint16_t*>(a.y)[row * half + n + q] = (uint16_t)(h[q >> 1] >> (16 * (q & 1)));
        continue;
      }
      uint32_t amax = amax_pairs<2 * TS>(h);
      uint32_t o = __shfl_xor(amax, 16, 64);
      amax = amax > o ? amax : o;
      o = __shfl_xor(amax, 32, 64);
      amax = amax > o ? amax : o;
      const uint32_t sc = e8m0_of_amax(amax);
      const bool bad = amax >= 0x7F800000u;
      if (!ok || n >= half) continue;  // blocks end where the columns do
#pragma unroll
      for (int k = 0; k < TS; k++)
        *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a.y) + row * (half >> 1) + ((n + 16 * k) >> 1)) =
            bad ? 0 : (uint16_t)codes_of_pairs(h[2 * k], h[2 * k + 1], sc);
      if (g == 0) a.y_scales[row * (half >> 5) + (n >> 5)] = (uint8_t)(bad ? kE8M0Nan : sc);
    }
    if (!GROUPED) return;  // dense: one pass
    __syncthreads();       // the partial sums have been read
  }
}

// A launch names the kernels that it may take and no others: dense forms have no SwiGLU, and among
// the grouped ones those of four weight tiles have nothing else.
template <class C, int MODE>
hipError_t launch_mode(const MxArgs& a, int64_t groups, hipStream_t stream) {
  constexpr bool SWIGLU = MODE != kDense && C::NT == 4;
  constexpr int64_t no = SWIGLU ? C::NT / 2 : C::NT;
  const int64_t cols = SWIGLU ? a.N >> 1 : a.N;
  const int64_t blocks = (cols + 16 * no - 1) / (16 * no) * groups;
  if (blocks * 64 * C::W > (int64_t)UINT32_MAX) return hipErrorInvalidConfiguration;
  const auto launch = [&](auto k) {
    hipLaunchKernelGGL(k, dim3((uint32_t)blocks), dim3(64 * C::W), C::LDS, stream, a);
    return hipGetLastError();
  };
  if constexpr (SWIGLU)
    return launch(a.swiglu == MXFP4_OUT_SWIGLU_BF16 ? mx_stream<C, MODE, MXFP4_OUT_SWIGLU_BF16>
                                                    : mx_stream<C, MODE, MXFP4_OUT_SWIGLU_MXFP4>);
  else
    return launch(mx_stream<C, MODE, 0>);
}

template <class C, bool GROUPED>
hipError_t launch_cfg(const MxArgs& a, hipStream_t stream) {
  if constexpr (GROUPED) {
    static_assert(C::LDS >= 4 * kScanRoutes, "further_run");
    return a.ids ? launch_mode<C, kByExpert>(a, scan_groups(a.R, a.top_k, a.num_experts), stream)
                 : launch_mode<C, kBySlot>(a, a.max_slots + a.max_tiles, stream);
  } else {
    return launch_mode<C, kDense>(a, (a.M + C::XR - 1) / C::XR, stream);
  }
}

template <int ACT, int XR, int NT, int W, int U, bool GROUPED = false>
hipError_t launch_rows(const MxArgs& a, hipStream_t stream) {
  const bool dw = a.K % 128 == 0 && ((uintptr_t)a.w_scales | (uintptr_t)a.x_scales) % 4 == 0;
  return dw ? launch_cfg<Cfg<ACT, XR, NT, W, U, true>, GROUPED>(a, stream)
            : launch_cfg<Cfg<ACT, XR, NT, W, U, false>, GROUPED>(a, stream);
}

template <int ACT, int XR, int U>
hipError_t launch_dense(const MxArgs& a, hipStream_t stream) {
  // So that a CU has about one workgroup: 16 x 12288 x 4096 takes 8.9 us with 48 weight rows
  // (256 workgroups), 11.2 with 16 (768, each loading the activations for itself).
  const int64_t nt = (a.N + 16 * 256 - 1) / (16 * 256);
  //
  // Steps in the ring (U), weights from HBM: BF16, 16 x 12288 x 4096 takes 10.7 us with 2, 10.8
  // with 3, 11.4 with 4, K = 14336 and N = 4096 15.8, 16.8, 17.0. MXFP4, 4 x 4096 x 4096 takes
  // 5.6, 4.8 and 4.7; where there are more rows of weight the fewer win again (12288: 9.4, 9.8,
  // 10.0).
  if (nt <= 1) return launch_rows<ACT, XR, 1, 4, U>(a, stream);
  if (nt <= 2) return launch_rows<ACT, XR, 2, 4, U>(a, stream);
  return launch_rows<ACT, XR, 3, 4, U>(a, stream);
}

template <int ACT>
hipError_t launch_act(const MxArgs& a, int64_t rows, hipStream_t stream) {
  constexpr bool MX = ACT == MXFP4_ACT_MXFP4;
  // A BF16 form of four rows loads no activations for the 12 others of the MFMA: 16 tokens x top-8
  // of 128 experts take 62 us a layer with it, 72 in the form of 16 rows, one token 17.3 and 18.1;
  // an expert with more routes takes several passes.
  if (a.ids || a.slots) {
    constexpr int FEW = MX ? 16 : 4;
    if (a.swiglu) return rows <= 2 ? launch_rows<ACT, FEW, 4, 4, 2, true>(a, stream) : launch_rows<ACT, 16, 4, 4, 2, true>(a, stream);
    return rows <= 2 ? launch_rows<ACT, FEW, 2, 2, 2, true>(a, stream) : launch_rows<ACT, 16, 2, 2, 2, true>(a, stream);
  }
  if (rows <= 4) return launch_dense<ACT, MX ? 16 : 4, MX ? 4 : 2>(a, stream);
  if (rows <= 16) return launch_dense<ACT, 16, MX ? 4 : 2>(a, stream);
  // Longer runs of rows read the weight less often, shorter ones spread it over more CUs. K =
  // 4096, BF16 activations: 64 x 4096 (256 runs of 32) 8.4 us against 12.4 in runs of 64, 256 x
  // 4096 (1024) 28.4 against 24.7.
  if (rows <= 32 || (rows + 31) / 32 * ((a.N + 31) / 32) <= 256) return launch_rows<ACT, 32, 2, 4, 2>(a, stream);
  return launch_rows<ACT, 64, 2, 4, 2>(a, stream);
}

}  // namespace

hipError_t launch_mx_stream(const MxArgs& a, int act_kind, int64_t rows, hipStream_t stream) {
  return act_kind == MXFP4_ACT_BF16 ? launch_act<MXFP4_ACT_BF16>(a, rows, stream)
                                    : launch_act<MXFP4_ACT_MXFP4>(a, rows, stream);
}

}  // namespace nvfp4
