// FP8 products for few activation rows: the weight is streamed once for all of them.
//
// Decode-sized products are bound by the weight's bytes, and a launch of a few microseconds by
// how soon its loads are in flight. A workgroup takes 16 * NT weight rows (SwiGLU: gate rows and
// the up rows that belong to them); its W waves split K into runs of steps, a block of 128 k
// each, through an LDS ring of their own that holds U steps of both operands, so no wave waits
// for another before the end, when their partial sums are added in wave order (results do not
// depend on timing). Loads go straight into LDS, eight lanes to a weight row's 128 bytes, and the
// LDS reads bring the operands into the MFMA's order; row r's 16-byte piece q lies at slot
// q ^ f(r), so that the 16 rows that lanes read together fall into different banks. Lane
// (c, g) = c + 16g takes pieces g and 4 + g of its row's eight, k = 16g and 64 + 16g on.
//  - FP8 activations, results in BF16: one MFMA over the step from zero, whose result is added
//    times both scales. (It is less exact than fp32: see mfma_f8.)
//  - otherwise the lane decodes its 32 codes to BF16 (for results in fp32 and SwiGLU those of FP8
//    activations too), four MFMAs over 32 k each from zero, whose result is added times the scales.
// The 16 weight rows of an MFMA lie in one block of 128, so its scale is the same for a wave: those
// of 64 steps are loaded at once.
// Loads past the rows, past K and past a wave's run are out of range: every step issues the
// same number, which is what the counted waits go by.
// Measured, weights from HBM: 16 x 12288 x 4096 11 to 12 us (50.5 MB, 4.2 to 4.6 TB/s; a copy of 2
// GiB reaches 4.9); one row of 4096 x 4096 4.0 us, which is the latency of a launch, one ring and the
// sum over the waves; gate_up of 16 tokens, top-8 of 128 experts of 1536 x 2048, 51 us with BF16
// activations (82 experts, 259 MB, 5.1 TB/s) and 53 in W8A8, whose sums in fp32 decode both sides.
#include "f8_device.hpp"
#include "f8_kernels.hpp"
#include "mx_routes.hpp"

namespace nvfp4 {
namespace {

// XR activation rows (4 or 8, or TM tiles of 16), NT tiles of 16 weight rows, W waves, U steps in
// the ring
template <int ACT_, int XR_, int NT_, int W_, int U_>
struct Cfg {
  static constexpr int ACT = ACT_, XR = XR_, TM = (XR_ + 15) / 16, NT = NT_, W = W_, U = U_;
  static constexpr bool F8 = ACT_ != FP8_ACT_BF16, FAST = ACT_ == FP8_ACT_FP8;
  static constexpr int XROWS = F8 ? 8 : 4, XMAX = XR / XROWS;  // 1 KiB loads of activations a step
  static constexpr int SX = F8 ? 1 : 0;  // loads of their scales
  static constexpr int LOADS = 2 * NT + XMAX + SX;
  static constexpr int W0 = 0, X0 = 2048 * NT, STEP = X0 + 1024 * XMAX;
  // of a wave: steps, scales of the weight, two windows of activation scales (16 bytes a row)
  static constexpr int WIN = 16 * XR * SX;
  static constexpr int WS0 = STEP * U, XS0 = WS0 + 256 * NT, RING = XS0 + 2 * WIN;
  static_assert(U - 1 <= 4, "a window is in use until it is overwritten");
  static constexpr int PART = 1024 * NT * TM;  // partial sums of a wave
  static constexpr int WAVES = W * (RING > PART ? RING : PART), LDS = WAVES + WIN;  // (the sink)
  static_assert(NT <= 4 && TM <= 4 && LDS <= 160 * 1024, "");
};

// 16-byte piece q of a 128-byte row lies at slot q ^ (row / 2 % 8). Of a 256-byte row of BF16,
// slot s ^ row % 16 holds this piece: those that lanes g = 0..3 read together are neighbours.
__device__ __forceinline__ int bf16_piece(int s) { return (s & 3) << 1 | ((s >> 2) & 1) | (s >> 3) << 3; }

struct Operands {
  u32x4 w, ws, x, xs;  // descriptors
};

// One wave's run [s0, s1) of steps over the rows whose lanes' offsets are wo, xo, xso; wso: where
// its weight tiles' scales begin; sink: C::WIN bytes of LDS that nobody reads.
template <class C>
__device__ __forceinline__ void run_steps(const Operands& d, uint32_t ring, const uint8_t* ring_p,
                                          int s0, int s1, int K, const uint32_t* wo,
                                          const uint32_t* xo, uint32_t xso,
                                          const uint32_t (&wso)[C::NT], uint32_t sink,
                                          f32x4 (&acc)[C::NT][C::TM]) {
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const auto issue = [&](int s, int u) {
    const uint32_t base = ring + u * C::STEP;
    const bool in = s < s1;
    // 8 rows a load; this lane's piece of its row depends on the load's parity only through the row
#pragma unroll
    for (int i = 0; i < 2 * C::NT; i++) {
      const int q = (lane & 7) ^ ((8 * i + (lane >> 3)) >> 1 & 7);
      lds_load<16>(d.w, in && 128 * s + 16 * q < K ? wo[i] + 128 * s : kOutOfRange, base + C::W0 + 1024 * i);
    }
#pragma unroll
    for (int i = 0; i < C::XMAX; i++) {
      uint32_t off;
      if (C::F8) {
        const int q = (lane & 7) ^ ((8 * i + (lane >> 3)) >> 1 & 7);
        off = in && 128 * s + 16 * q < K ? xo[i] + 128 * s : kOutOfRange;
      } else {
        const int q = bf16_piece((lane & 15) ^ ((4 * i + (lane >> 4)) & 15));
        off = in && 128 * s + 8 * q < K ? xo[i] + 256 * s : kOutOfRange;
      }
      lds_load<16>(d.x, off, base + C::X0 + 1024 * i);
    }
    if (C::F8) {
      // scales of four steps at a time: a load costs by the cache lines that it looks up (against
      // a load of 4 bytes a row and step: M 64 x 4096 x 4096 8.7 -> 8.2 us, 16 x 4096 x 14336
      // 15.0 -> 13.9 us). Past the last row they are out of range, dword by dword.
      const int n = s - s0;
      if (lane < C::XR)
        lds_load<16>(d.xs, in && n % 4 == 0 ? xso + 4 * s : kOutOfRange,
                     n % 4 == 0 ? ring + C::XS0 + n / 4 % 2 * C::WIN : sink);
    }
  };
  // the weight tiles' scales of 64 steps from s on
  const auto load_scales = [&](int s) {
#pragma unroll
    for (int t = 0; t < C::NT; t++) lds_load<4>(d.ws, s + lane < s1 ? wso[t] + 4 * (s + lane) : kOutOfRange, ring + C::WS0 + 256 * t);
  };
  load_scales(s0);
#pragma unroll
  for (int u = 0; u < C::U - 1; u++) issue(s0 + u, u);
  int u = 0;
  for (int s = s0; s < s1; s++) {
    const int sl = (s - s0) & 63;
    if (sl == 0 && s > s0) {
      wait_lds_reads();
      load_scales(s);
      wait_loads<0>();
    }
    wait_lds_reads();  // of the step whose bytes the next loads overwrite
    issue(s + C::U - 1, u == 0 ? C::U - 1 : u - 1);
    wait_loads<(C::U - 1) * C::LOADS>();
    const uint8_t* b = ring_p + u * C::STEP;
    const auto piece = [&](const uint8_t* rows, int r, int q) {
      return *reinterpret_cast<const u32x4*>(rows + 128 * r + ((q ^ (r >> 1 & 7)) << 4));
    };
    float xs[C::TM];
#pragma unroll
    for (int x = 0; x < C::TM; x++)
      xs[x] = C::F8 ? reinterpret_cast<const float*>(ring_p + C::XS0 + (s - s0) / 4 % 2 * C::WIN +
                                                     16 * ((16 * x + c) % C::XR))[(s - s0) % 4]
                    : 1.f;
    // this lane's 32 k of activation row 16x + c: two pieces of codes, or four of BF16
    u32x4 xf[C::TM][C::FAST ? 2 : 4];
#pragma unroll
    for (int x = 0; x < C::TM; x++) {
      // rows past the loaded ones read others' values, into columns that nobody stores
      const int r = (16 * x + c) % (C::XROWS * C::XMAX);
      if constexpr (C::F8) {
        const u32x4 x0 = piece(b + C::X0, r, g), x1 = piece(b + C::X0, r, 4 + g);
        if constexpr (C::FAST) {
          xf[x][0] = x0;
          xf[x][1] = x1;
        } else {
          f8_decode32(x0, x1, xf[x]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; j++)
          xf[x][j] = *reinterpret_cast<const u32x4*>(b + C::X0 + 256 * r + (((g + 4 * j) ^ (r & 15)) << 4));
      }
    }
#pragma unroll
    for (int t = 0; t < C::NT; t++) {
      const u32x4 w0 = piece(b + C::W0, 16 * t + c, g), w1 = piece(b + C::W0, 16 * t + c, 4 + g);
      const float sw = *reinterpret_cast<const float*>(ring_p + C::WS0 + 256 * t + 4 * sl);
      u32x4 wf[4];
      if constexpr (!C::FAST) f8_decode32(w0, w1, wf);
#pragma unroll
      for (int x = 0; x < C::TM; x++) {
        f32x4 p = {0.f, 0.f, 0.f, 0.f};
        if constexpr (C::FAST) {
          p = mfma_f8(w0, w1, xf[x][0], xf[x][1], p);
        } else {
#pragma unroll
          for (int j = 0; j < 4; j++) p = mfma16(wf[j], xf[x][j], p);
        }
        const float sc = C::F8 ? sw * xs[x] : sw;
#pragma unroll
        for (int i = 0; i < 4; i++) acc[t][x][i] = __builtin_fmaf(p[i], sc, acc[t][x][i]);
      }
    }
    u = u + 1 == C::U ? 0 : u + 1;
  }
  wait_loads<0>();
}

template <class C, int MODE, int SWIGLU>
__global__ __launch_bounds__(64 * C::W) void f8_stream(F8Args a) {
  constexpr bool GROUPED = MODE != kDense;
  constexpr int NO = SWIGLU ? C::NT / 2 : C::NT;  // 16-column tiles of output
  static_assert(!GROUPED || C::TM == 1, "a grouped pass has at most 16 rows");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  __shared__ int32_t route_list[C::W][16];  // the pass's routes, a copy for each wave
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // sizes below 2^31 (a weight's bytes too): 32-bit arithmetic
  const int N = (int)a.N, half = N >> 1, cols = SWIGLU ? half : N;
  const int K = (int)a.K, kb = (K + 127) >> 7;
  const uint32_t nbn = (cols + 16 * NO - 1) / (16 * NO);
  const int group = (int)(blockIdx.x / nbn);
  const int n0 = (int)(blockIdx.x - group * nbn) * (16 * NO);
  const uint8_t* wc = a.w_codes;
  const float* wsc = a.w_scales;
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
    wc += (int64_t)e * N * K;
    wsc += (int64_t)e * ((N + 127) >> 7) * kb;
  }
  Operands d;
  const int r0 = SWIGLU ? 0 : n0;  // weight row that the offsets count from
  d.w = lds_load_rsrc(wc + (int64_t)r0 * K, (int64_t)(N - r0) * K);
  d.ws = lds_load_rsrc(wsc + (int64_t)(r0 >> 7) * kb, 4 * (int64_t)(((N + 127) >> 7) - (r0 >> 7)) * kb);
  const uint32_t xpitch = (uint32_t)a.ldx * (C::F8 ? 1 : 2);
  const int64_t x_rows = GROUPED ? a.x_rows : count;
  d.x = lds_load_rsrc(static_cast<const uint8_t*>(a.x) + (int64_t)row0 * xpitch,
                      (x_rows - 1) * xpitch + (C::F8 ? 1 : 2) * (int64_t)K);
  d.xs = C::F8 ? lds_load_rsrc(a.x_scales + (int64_t)row0 * kb, 4 * x_rows * kb) : d.x;
  // row i of weight tile t, from r0, or -1; and the tile's scales
  const auto w_row = [&](int t, int i) {
    const int n = n0 + 16 * (t % NO) + i;
    return n < cols ? n - r0 + (t >= NO ? half : 0) : -1;
  };
  uint32_t wso[C::NT];
#pragma unroll
  for (int t = 0; t < C::NT; t++)  // (past the weight's rows it is out of range)
    wso[t] = 4u * (uint32_t)((n0 + 16 * (t % NO) + (t >= NO ? half : 0) - (r0 & ~127)) >> 7) * (uint32_t)kb;
  uint32_t wo[2 * C::NT];
#pragma unroll
  for (int i = 0; i < 2 * C::NT; i++) {
    const int r = 8 * (i & 1) + (lane >> 3), row = w_row(i >> 1, r);
    wo[i] = row >= 0 ? (uint32_t)row * (uint32_t)K + 16 * ((lane & 7) ^ (r >> 1 & 7)) : kOutOfRange;
  }
  // this wave's run of steps
  const int per = (kb + C::W - 1) / C::W;
  const int s0 = wave * per, s1 = s0 + per < kb ? s0 + per : kb;
  constexpr int WAVE = C::WAVES / C::W;
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
    uint32_t xo[C::XMAX], xso = kOutOfRange;
#pragma unroll
    for (int i = 0; i < C::XMAX; i++) {
      const int r = C::F8 ? 8 * i + (lane >> 3) : 4 * i + (lane >> 4), row = x_row(r);
      const int q = C::F8 ? (lane & 7) ^ (r >> 1 & 7) : bf16_piece((lane & 15) ^ (r & 15));
      xo[i] = row >= 0 ? (uint32_t)row * xpitch + 16 * q : kOutOfRange;
    }
    if (C::F8) {
      const int row = lane < C::XR ? x_row(lane) : -1;
      xso = row >= 0 ? 4u * (uint32_t)row * (uint32_t)kb : kOutOfRange;
    }
    f32x4 acc[C::NT][C::TM];
#pragma unroll
    for (int t = 0; t < C::NT; t++)
#pragma unroll
      for (int x = 0; x < C::TM; x++) acc[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (s0 < s1)
      run_steps<C>(d, ring, ring_p, s0, s1, K, wo, xo, xso, wso,
                   lds_address(smem) + C::W * WAVE, acc);
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
    // an item: four columns per lane of a 16 x 16 tile
    for (int i = wave; i < NO * C::TM; i += C::W) {
      const int t = i % NO, x = i / NO;
      if (16 * x + c >= rows) continue;
      const int64_t row = MODE == kBySlot ? in_routes(a, y_row(16 * x + c)) : row0 + y_row(16 * x + c);
      const int n = n0 + 16 * t + 4 * g;
      f32x4 v = total(t, x);
      if (SWIGLU) {
        const f32x4 u = total(NO + t, x);
#pragma unroll
        for (int q = 0; q < 4; q++) v[q] = silu(v[q]) * u[q];
      }
      const int64_t at = row * (SWIGLU ? half : a.ldy) + n;
      if (!SWIGLU && a.y_type == FP8_F32) {
        float* y = static_cast<float*>(a.y) + at;
        if (n + 4 <= cols && ((uintptr_t)y & 15) == 0) {
          *reinterpret_cast<f32x4*>(y) = v;
        } else {
#pragma unroll
          for (int q = 0; q < 4; q++)
            if (n + q < cols) y[q] = v[q];
        }
        continue;
      }
      uint16_t* y = static_cast<uint16_t*>(a.y) + at;
      const uint2 b = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
      if (n + 4 <= cols && ((uintptr_t)y & 7) == 0) {
        *reinterpret_cast<uint2*>(y) = b;
      } else {
#pragma unroll
        for (int q = 0; q < 4; q++)
          if (n + q < cols) y[q] = (uint16_t)((q < 2 ? b.x : b.y) >> (16 * (q & 1)));
      }
    }
    if (!GROUPED) return;  // dense: one pass
    __syncthreads();       // the partial sums have been read
  }
}

// Dense forms have no SwiGLU, and among the grouped ones those of four weight tiles have nothing
// else (and none of them is FAST).
template <class C, int MODE>
hipError_t launch_mode(const F8Args& a, int64_t groups, hipStream_t stream) {
  constexpr bool SWIGLU = MODE != kDense && C::NT == 4;
  constexpr int64_t no = SWIGLU ? C::NT / 2 : C::NT;
  const int64_t cols = SWIGLU ? a.N >> 1 : a.N;
  const int64_t blocks = (cols + 16 * no - 1) / (16 * no) * groups;
  if (blocks * 64 * C::W > (int64_t)UINT32_MAX) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((f8_stream<C, MODE, SWIGLU ? FP8_OUT_SWIGLU_BF16 : 0>), dim3((uint32_t)blocks),
                     dim3(64 * C::W), C::LDS, stream, a);
  return hipGetLastError();
}

template <int ACT, int XR, int NT, int W, int U, bool GROUPED = false>
hipError_t launch_rows(const F8Args& a, hipStream_t stream) {
  typedef Cfg<ACT, XR, NT, W, U> C;
  if constexpr (GROUPED) {
    static_assert(C::LDS >= 4 * kScanRoutes, "further_run");
    return a.ids ? launch_mode<C, kByExpert>(a, scan_groups(a.R, a.top_k, a.num_experts), stream)
                 : launch_mode<C, kBySlot>(a, a.max_slots + a.max_tiles, stream);
  } else {
    return launch_mode<C, kDense>(a, (a.M + C::XR - 1) / C::XR, stream);
  }
}

template <int ACT, int XR, int U>
hipError_t launch_dense(const F8Args& a, hipStream_t stream) {
  // so that a CU has about one workgroup
  const int64_t nt = (a.N + 16 * 256 - 1) / (16 * 256);
  if (nt <= 1) return launch_rows<ACT, XR, 1, 4, U>(a, stream);
  if (nt <= 2) return launch_rows<ACT, XR, 2, 4, U>(a, stream);
  return launch_rows<ACT, XR, 3, 4, U>(a, stream);
}

template <int ACT>
hipError_t launch_act(const F8Args& a, int64_t rows, hipStream_t stream) {
  constexpr bool F8 = ACT != FP8_ACT_BF16;
  // Forms of eight rows (BF16: four) load no activations for the other ones of the MFMA. By expert,
  // where two of their workgroups fit a CU and two of the larger ones do not, they also win with a
  // second turn over the weight, from L2. 128 experts, top-8, 2048 / 768: W8A8 gate_up and down of 64
  // tokens (four routes an expert) take 83 + 52 us eight rows at a time, 103 + 55 in sixteen; BF16
  // gate_up of 48 tokens 79 us with four rows, 96 with sixteen (down 50 with eight, 57), of 96
  // tokens 112 and 101 (56, 60), of 32 experts, top-4, 2048 / 1024, 32 tokens 34 and 29 (19 and 20).
  constexpr int FEW = F8 ? 8 : 4;
  if (a.ids || a.slots) {
    if constexpr (ACT != FP8_ACT_FP8) {
      if (a.swiglu)
        return F8 || rows <= 3 ? launch_rows<ACT, FEW, 4, 4, 2, true>(a, stream)
                               : launch_rows<ACT, F8 ? FEW : 16, 4, 4, 2, true>(a, stream);
    }
    return rows <= 2 ? launch_rows<ACT, FEW, 2, 2, 2, true>(a, stream)
                     : launch_rows<ACT, 8, 2, 2, 2, true>(a, stream);
  }
  if (rows <= FEW) return launch_dense<ACT, FEW, F8 ? 3 : 2>(a, stream);
  if (rows <= 16) return launch_dense<ACT, 16, F8 ? 3 : 2>(a, stream);
  if (rows <= 32) return launch_rows<ACT, 32, 2, 4, 2>(a, stream);
  return launch_rows<ACT, F8 ? 64 : 48, 2, 4, 2>(a, stream);
}

}  // namespace

hipError_t launch_f8_stream(const F8Args& a, int act_kind, int64_t rows, hipStream_t stream) {
  return act_kind == FP8_ACT_BF16  ? launch_act<FP8_ACT_BF16>(a, rows, stream)
         : act_kind == FP8_ACT_FP8 ? launch_act<FP8_ACT_FP8>(a, rows, stream)
                                   : launch_act<kF8Exact>(a, rows, stream);
}

}  // namespace nvfp4
