// FP8 products in LDS tiles, for enough activation rows to fill them.
//
// A workgroup computes BM activation rows x BN weight rows; its WX x WW waves share the tile,
// each 16 * TX rows by 16 * TW weight rows of 16x16 MFMAs with the weight rows as A, so that a
// lane's results run along an output row. K goes by in stages through a ring of D LDS buffers:
//  - Loads go from memory straight into LDS (buffer_load ... lds), D - 1 stages ahead, with no
//    registers in between. They are written as instructions without outputs, which the
//    compiler does not wait for; one counted wait and one barrier per stage stand before its
//    reads. Past the end of K (and of the rows) the loads are out of range and write zeros,
//    so every stage issues the same number and the count holds to the last one.
//  - A stage is a block of 128 k, or 64 k where the activations are BF16: 128 bytes, a cache
//    line, of an activation row.
//  - LDS rows have no padding (the loads write 1 KiB runs); 16-byte piece q of a row lies at
//    slot q ^ f(row), with f such that the 16 rows that lanes read together fall into
//    different banks. (A 16-byte read takes lanes of two neighbouring g together, whose pieces
//    have to differ in the lowest bit: piece 2g + j of BF16 rows counts as g + 4j.)
//  - Weight row 4P * a + 4s + b of a group of 16P rows is row 4a + b of the MFMA of its s-th
//    16-row tile (P tiles to a group): a lane's results are then 4P consecutive columns.
//  - An MFMA's result is that of its stage alone; it is multiplied by its scales and added to the
//    lane's sums by fp32 FMAs, which the vector units do while the matrix cores go on. The 64
//    weight rows of a group (SwiGLU: of gate, of up) lie in one block of scales, so their scale
//    is a scalar: lane l of a wave holds that of the stage that is l on. The scales of activation
//    rows come in windows of 16 bytes, four blocks at a time, through LDS.
#include <type_traits>

#include "f8_device.hpp"
#include "f8_kernels.hpp"
#include "mx_routes.hpp"
#include "mx_tile.hpp"

namespace nvfp4 {
namespace {

template <int ACT_, int BM_, int BN_, int WX_, int WW_, int D_>
struct Shape {
  static constexpr int ACT = ACT_, BM = BM_, BN = BN_, WX = WX_, WW = WW_, D = D_;
  static constexpr bool F8 = ACT != FP8_ACT_BF16, FAST = ACT == FP8_ACT_FP8;
  static constexpr int T = 64 * WX * WW;
  static constexpr int TX = BM / WX / 16, TW = BN / WW / 16;
  static constexpr int SK = F8 ? 128 : 64;  // k of a stage
  static constexpr int XB = 128, WB = SK;   // bytes of a row per stage
  static constexpr int NX = BM * XB / (16 * T), NW = BN * WB / (16 * T);
  // scales of activation rows: one load of a window in four stages, out of range in the others
  static constexpr int NS = F8 ? (BM + T - 1) / T : 0, WS = 4;
  static constexpr int LOADS = NX + NW + NS;
  static constexpr int X0 = 0, W0 = BM * XB, STAGE = W0 + BN * WB;
  static constexpr int WIN = F8 ? BM * 16 : 0;
  static constexpr int WIN0 = D * STAGE, SINK = WIN0 + 2 * WIN;  // SINK: bytes that nobody reads
  static constexpr int LDS = SINK + (F8 ? 1024 : 0);
  static_assert(D - 1 <= WS, "a window is in use until it is overwritten");
  static_assert(16 * TW * 16 * 4 * WX * WW <= LDS, "the results' way out");
  static_assert(NX * 16 * T == BM * XB && NW * 16 * T == BN * WB, "whole loads only");
  static_assert(LDS <= 160 * 1024, "LDS");
  static_assert(TW % 4 == 0, "weight rows come in groups of 64 (SwiGLU: 32 + 32)");
};

// slot of piece q of a weight row of 64 bytes is q ^ quarter_swizzle(row)
__device__ __forceinline__ int quarter_swizzle(int row) {
  const int a = (row >> 2) & 3;
  return ((a & 1) << 1) ^ ((a >> 1) * 3);
}

template <class S, bool GROUPED, int SWIGLU>
__global__ __launch_bounds__(S::T) __attribute__((amdgpu_waves_per_eu(S::T == 512 ? 2 : 1, 2)))
void f8_tiled(F8Args a, int gm, int vec) {
  constexpr int P = SWIGLU ? S::TW / 2 : 4;  // tiles of a group of weight rows
  constexpr int GROUPS = S::TW / P;          // of a wave; SwiGLU: gate, up
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int wx = wave % S::WX, ww = wave / S::WX;
  const int64_t N = a.N, half = N >> 1;
  const int K = (int)a.K, kb = (K + 127) >> 7;
  const int64_t cols = SWIGLU ? half : N;
  constexpr int BC = SWIGLU ? S::BN / 2 : S::BN;  // output columns of a tile
  const uint32_t nbn = (uint32_t)((cols + BC - 1) / BC);

  // tile of this workgroup: each XCD (blockIdx % 8) takes a run of tiles, which share
  // operands through its L2 (the parts of a list tile among them)
  int64_t mt, nt;
  int part = 0;
  {
    const uint32_t parts = GROUPED ? a.tile_rows / S::BM : 1;
    uint32_t nbm = GROUPED ? *a.n_tiles : (uint32_t)((a.M + S::BM - 1) / S::BM);
    if (GROUPED) {
      nbm = nbm < (uint32_t)a.max_tiles ? nbm : (uint32_t)a.max_tiles;
      clear_dropped<SWIGLU>(a);
    }
    const uint32_t total = nbm * nbn * parts;
    if (blockIdx.x >= total) return;
    const uint32_t q = total / 8, r = total % 8, x = blockIdx.x % 8;
    uint32_t lin = x * q + (x < r ? x : r) + blockIdx.x / 8;
    if (GROUPED) {
      part = (int)(lin % parts);
      lin /= parts;
    }
    const uint32_t first = lin / (gm * nbn) * gm, in = lin % (gm * nbn);
    const uint32_t rows = nbm - first < (uint32_t)gm ? nbm - first : gm;
    mt = first + in % rows;
    nt = in / rows;
  }
  const int64_t n0 = nt * BC;
  const uint8_t* wc = a.w_codes;
  const float* ws = a.w_scales;
  int64_t m0 = 0, rows_m;
  int32_t slot0 = 0;
  if (GROUPED) {
    const int e = in_experts(a, a.tiles[2 * mt]);
    slot0 = in_routes(a, a.tiles[2 * mt + 1]) + part * S::BM;
    rows_m = run_length(a, slot0, a.offsets[e + 1], S::BM);
    if (rows_m == 0) return;
    wc += (int64_t)e * N * K;
    ws += (int64_t)e * ((N + 127) >> 7) * kb;
  } else {
    m0 = mt * S::BM;
    rows_m = a.M - m0 < S::BM ? a.M - m0 : S::BM;
  }

  // x row of tile row r (grouped: relative to x, dense: to the tile's first row)
  const auto x_row = [&](int r) -> int64_t {
    if (!GROUPED) return r;
    const int32_t route = a.sorted[slot0 + r];
    return a.rows_per_token ? route / a.top_k : route;
  };
  constexpr int XE = S::F8 ? 1 : 2;  // bytes of an activation
  const int64_t xpitch = a.ldx * XE;
  const int64_t x_last = GROUPED ? a.x_rows : rows_m;
  const u32x4 xr = lds_load_rsrc(static_cast<const uint8_t*>(a.x) + (GROUPED ? 0 : m0 * xpitch),
                                 (x_last - 1) * xpitch + (int64_t)K * XE);
  const u32x4 wr = lds_load_rsrc(wc + (SWIGLU ? 0 : n0 * K), (N - (SWIGLU ? 0 : n0)) * K);
  // weight row of tile row t relative to that base, or -1
  const auto w_row = [&](int t) -> int64_t {
    if (!SWIGLU) return n0 + t < N ? t : -1;
    const int u = t >= BC ? t - BC : t;
    return n0 + u < half ? n0 + u + (t >= BC ? half : 0) : -1;
  };
  const auto w_swizzle = [](int t) { return ((t >> 1) & 1) | ((t / (4 * P)) & 3) << 1; };

  // this lane's loads of stage 0, and the first k of each; a stage on, offsets grow by XB / WB
  uint32_t xo[S::NX], wo[S::NW];
  int xk[S::NX], wk[S::NW];
#pragma unroll
  for (int i = 0; i < S::NX; i++) {
    const int p = i * S::T + tid, r = p >> 3;
    int q = (p & 7) ^ ((r >> 1) & 7);
    if (!S::F8) q = (q & 3) << 1 | q >> 2;
    xk[i] = q * (16 / XE);
    xo[i] = r < rows_m ? (uint32_t)(x_row(r) * xpitch) + 16 * q : kOutOfRange;
  }
#pragma unroll
  for (int i = 0; i < S::NW; i++) {
    const int p = i * S::T + tid;
    int t, q;
    if (S::F8) {
      t = p >> 3;
      q = (p & 7) ^ w_swizzle(t);
    } else {  // rows in the order of the MFMA's: row p / 4 is row p / 4 % 16 of 16-row tile p / 64
      const int u = p >> 6, i16 = (p >> 2) & 15;
      t = (u / P) * 16 * P + 4 * P * (i16 >> 2) + 4 * (u % P) + (i16 & 3);
      q = (p & 3) ^ quarter_swizzle(i16);
    }
    wk[i] = 16 * q;
    const int64_t row = w_row(t);
    wo[i] = row >= 0 ? (uint32_t)(row * K) + 16 * q : kOutOfRange;
  }
  u32x4 xsr = xr;
  uint32_t so[S::NS ? S::NS : 1];
  if (S::F8) {
    xsr = lds_load_rsrc(a.x_scales + (GROUPED ? 0 : m0 * kb), 4 * x_last * kb);
#pragma unroll
    for (int i = 0; i < S::NS; i++) {
      const int r = i * S::T + tid;
      so[i] = r < rows_m ? (uint32_t)(4 * x_row(r) * kb) : kOutOfRange;
    }
  }

  const uint32_t lds0 = lds_address(smem);
  const auto issue = [&](int st, int buf) {
    const uint32_t base = lds0 + buf * S::STAGE;
    const int k0 = st * S::SK;
#pragma unroll
    for (int i = 0; i < S::NX; i++)
      lds_load<16>(xr, k0 + xk[i] < K ? xo[i] + st * S::XB : kOutOfRange, base + S::X0 + (i * S::T + wave * 64) * 16);
#pragma unroll
    for (int i = 0; i < S::NW; i++)
      lds_load<16>(wr, k0 + wk[i] < K ? wo[i] + st * S::WB : kOutOfRange, base + S::W0 + (i * S::T + wave * 64) * 16);
#pragma unroll
    for (int i = 0; i < S::NS; i++) {
      const int r0 = i * S::T + wave * 64;
      const bool now = st % S::WS == 0 && st < kb && r0 < S::BM;
      lds_load<16>(xsr, now ? so[i] + 4 * st : kOutOfRange,
                   now ? lds0 + S::WIN0 + st / S::WS % 2 * S::WIN + r0 * 16 : lds0 + S::SINK);
    }
  };

  f32x4 acc[S::TW][S::TX];
#pragma unroll
  for (int t = 0; t < S::TW; t++)
#pragma unroll
    for (int x = 0; x < S::TX; x++) acc[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};

  // first tile row of the group of this wave's weight tile t; tile row of the tile's MFMA row
  // 4a + b
  const auto w_group = [&](int t) { return SWIGLU ? t / P * BC + ww * 16 * P : (ww * GROUPS + t / P) * 16 * P; };
  const auto w_local = [&](int t, int row) { return w_group(t) + 4 * P * (row >> 2) + 4 * (t % P) + (row & 3); };
  // scales of this wave's groups
  const float* wsp[GROUPS];
#pragma unroll
  for (int i = 0; i < GROUPS; i++) {
    const int64_t n = SWIGLU ? n0 + ww * 16 * P + i * half : n0 + w_group(i * P);
    wsp[i] = ws + (n < N ? n >> 7 : 0) * kb;
  }

  const int steps = (K + S::SK - 1) / S::SK;
#pragma unroll
  for (int i = 0; i < S::D - 1; i++) issue(i, i);
  float w_scale[GROUPS];
  const auto stage = [&](int st, int buf) {
    const int b = S::F8 ? st : st >> 1;  // block of scales
    if ((b & 63) == 0 && (S::F8 || (st & 1) == 0)) {
#pragma unroll
      for (int i = 0; i < GROUPS; i++) w_scale[i] = b + lane < kb ? wsp[i][b + lane] : 0.f;
    }
    wait_loads_barrier<(S::D - 2) * S::LOADS>();
    issue(st + S::D - 1, buf == 0 ? S::D - 1 : buf - 1);
    const uint8_t* xs = smem + buf * S::STAGE + S::X0;
    const uint8_t* wl = smem + buf * S::STAGE + S::W0;
    const uint8_t* sl = smem + S::WIN0 + st / S::WS % 2 * S::WIN + st % S::WS * 4;
    float sw[GROUPS];
#pragma unroll
    for (int i = 0; i < GROUPS; i++)
      sw[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w_scale[i]), b & 63));
    const auto add = [&](int t, int x, f32x4 p, float sc) {
#pragma unroll
      for (int i = 0; i < 4; i++) acc[t][x][i] = __builtin_fmaf(p[i], sc, acc[t][x][i]);
    };
    if constexpr (S::F8) {
      u32x4 wf[S::TW][S::FAST ? 2 : 4];
#pragma unroll
      for (int t = 0; t < S::TW; t++) {
        const int r = w_local(t, c);
        const u32x4 w0 = *reinterpret_cast<const u32x4*>(wl + r * 128 + ((g ^ w_swizzle(r)) << 4));
        const u32x4 w1 = *reinterpret_cast<const u32x4*>(wl + r * 128 + (((4 + g) ^ w_swizzle(r)) << 4));
        if constexpr (S::FAST) {
          wf[t][0] = w0;
          wf[t][1] = w1;
        } else {
          f8_decode32(w0, w1, wf[t]);
        }
      }
#pragma unroll
      for (int x = 0; x < S::TX; x++) {
        const int r = (wx * S::TX + x) * 16 + c;
        const u32x4 x0 = *reinterpret_cast<const u32x4*>(xs + r * 128 + ((g ^ ((r >> 1) & 7)) << 4));
        const u32x4 x1 = *reinterpret_cast<const u32x4*>(xs + r * 128 + (((4 + g) ^ ((r >> 1) & 7)) << 4));
        const float sx = *reinterpret_cast<const float*>(sl + r * 16);
        u32x4 xf[4];
        if constexpr (!S::FAST) f8_decode32(x0, x1, xf);
#pragma unroll
        for (int t = 0; t < S::TW; t++) {
          f32x4 p = {0.f, 0.f, 0.f, 0.f};
          if constexpr (S::FAST) {
            p = mfma_f8(wf[t][0], wf[t][1], x0, x1, p);
          } else {
#pragma unroll
            for (int j = 0; j < 4; j++) p = mfma16(wf[t][j], xf[j], p);
          }
          add(t, x, p, sw[t / P] * sx);
        }
      }
    } else {
      u32x4 xf[S::TX][2];
#pragma unroll
      for (int x = 0; x < S::TX; x++) {
        const int r = (wx * S::TX + x) * 16 + c;
#pragma unroll
        for (int j = 0; j < 2; j++)
          xf[x][j] = *reinterpret_cast<const u32x4*>(xs + r * 128 + (((g + 4 * j) ^ ((r >> 1) & 7)) << 4));
      }
#pragma unroll
      for (int t = 0; t < S::TW; t++) {
        // 16-row tile in the order of the loads
        const int u = w_group(t) / 16 + t % P;
        const u32x4 w = *reinterpret_cast<const u32x4*>(wl + u * 1024 + 64 * c + ((g ^ quarter_swizzle(c)) << 4));
        const u32x4 w0 = f8_decode8(w[0], w[1]), w1 = f8_decode8(w[2], w[3]);
#pragma unroll
        for (int x = 0; x < S::TX; x++)
          add(t, x, mfma16(w1, xf[x][1], mfma16(w0, xf[x][0], f32x4{0.f, 0.f, 0.f, 0.f})), sw[t / P]);
      }
    }
  };
  // the ring's buffers are taken in turn, by a loop that is unrolled so that they are constants
  for (int st0 = 0; st0 < steps; st0 += S::D) {
#pragma unroll
    for (int i = 0; i < S::D; i++) {
      if (i && st0 + i >= steps) break;
      stage(st0 + i, i);
    }
  }
  wait_loads<0>();  // nothing writes LDS after the workgroup

  if constexpr (!SWIGLU) {
    wait_loads_barrier<0>();  // the other waves have read their last stage
    const int64_t n = n0 + ww * S::TW * 16;
    uint8_t* const out = smem + wave * store_bytes<S>();
    if (n >= N) return;
    if (a.y_type == FP8_F32)
      store_tile<S, GROUPED, 4>(a, out, acc, wx, m0, slot0, rows_m, n, N - n, vec);
    else
      store_tile<S, GROUPED, 2>(a, out, acc, wx, m0, slot0, rows_m, n, N - n, vec);
    return;
  }
#pragma unroll
  for (int x = 0; x < S::TX; x++) {
    const int r = (wx * S::TX + x) * 16 + c;
    if (r >= rows_m) continue;
    const int64_t row = GROUPED ? route_at(a, slot0 + r) : m0 + r;
    // SwiGLU: tile t and tile P + t are gate and up of the same columns
    const int64_t n = n0 + w_local(0, 4 * g);
    uint32_t h[2 * P];  // BF16 pairs of 4P consecutive columns
#pragma unroll
    for (int s = 0; s < P; s++) {
      const f32x4 gt = acc[s][x], u = acc[P + s][x];
      h[2 * s] = bf16_pair(silu(gt[0]) * u[0], silu(gt[1]) * u[1]);
      h[2 * s + 1] = bf16_pair(silu(gt[2]) * u[2], silu(gt[3]) * u[3]);
    }
    uint16_t* d = static_cast<uint16_t*>(a.y) + row * half + n;
    if (vec && n + 4 * P <= half) {
#pragma unroll
      for (int s = 0; s < P / 2; s++)
        reinterpret_cast<u32x4*>(d)[s] = u32x4{h[4 * s], h[4 * s + 1], h[4 * s + 2], h[4 * s + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4 * P; i++)
        if (n + i < half) d[i] = (uint16_t)(h[i >> 1] >> (16 * (i & 1)));
    }
  }
}

// most rows of a tile of a grouped product
constexpr int grouped_rows(int act) { return act == FP8_ACT_FP8 ? 128 : 64; }

template <class S>
hipError_t launch_shape(const F8Args& a, hipStream_t stream) {
  const int64_t bc = a.swiglu ? S::BN / 2 : S::BN;
  const int64_t cols = a.swiglu ? a.N >> 1 : a.N;
  const int64_t nbm = a.tiles ? a.max_tiles : (a.M + S::BM - 1) / S::BM;
  const int64_t parts = a.tiles ? a.tile_rows / S::BM : 1;
  const int64_t groups = nbm * ((cols + bc - 1) / bc) * parts;
  if (groups * S::T > (int64_t)UINT32_MAX) return hipErrorInvalidConfiguration;
  // an XCD's 32 CUs work on gm x (32 / gm) tiles (grouped: on the columns of a few list tiles)
  const int gm = a.tiles ? 1 : 4;
  const int64_t ysz = a.y_type == FP8_F32 ? 4 : 2, ld = a.swiglu ? cols : a.ldy;
  const int vec = ((uintptr_t)a.y | (uintptr_t)(ld * ysz)) % 16 == 0;
  auto k = f8_tiled<S, false, 0>;
  if constexpr (S::BM <= grouped_rows(S::ACT)) {
    if (a.tiles) k = a.swiglu ? f8_tiled<S, true, FP8_OUT_SWIGLU_BF16> : f8_tiled<S, true, 0>;
  }
  hipLaunchKernelGGL(k, dim3((uint32_t)groups), dim3(S::T), S::LDS, stream, a, gm, vec);
  return hipGetLastError();
}

// The largest tile that still makes about a workgroup per CU is taken: larger ones read the
// operands less often.
constexpr int64_t kFewTiles = 200;

template <int ACT>
hipError_t launch_act(const F8Args& a, hipStream_t stream) {
  constexpr bool F8 = ACT != FP8_ACT_BF16;
  const int64_t cols = a.swiglu ? a.N >> 1 : a.N;
  const int64_t active = a.R < a.num_experts ? a.R : a.num_experts;
  // workgroups that tiles of bm rows and bn weight rows make (grouped: about)
  const auto tiles = [&](int64_t bm, int64_t bn) {
    const int64_t bc = a.swiglu ? bn / 2 : bn;
    return (a.tiles ? a.R / bm + active : (a.M + bm - 1) / bm) * ((cols + bc - 1) / bc);
  };
  const int64_t rows = !a.tiles ? a.M : a.tile_rows < grouped_rows(ACT) ? a.tile_rows : grouped_rows(ACT);
  if (rows > 128 && tiles(256, 256) >= kFewTiles) return launch_shape<Shape<ACT, 256, 256, 2, 4, F8 ? 2 : 3>>(a, stream);
  if (rows > 64 && tiles(128, 256) >= kFewTiles) return launch_shape<Shape<ACT, 128, 256, 2, 4, 3>>(a, stream);
  if (rows > 64 && (a.tiles || tiles(128, 128) >= kFewTiles)) return launch_shape<Shape<ACT, 128, 128, 2, 2, F8 ? 3 : 4>>(a, stream);
  if (tiles(64, 256) >= kFewTiles) return launch_shape<Shape<ACT, 64, 256, F8 ? 2 : 1, 4, 3>>(a, stream);
  return launch_shape<Shape<ACT, 64, 128, 2, 2, F8 ? 3 : 4>>(a, stream);
}

}  // namespace

hipError_t launch_f8_tiled(const F8Args& a, int act_kind, hipStream_t stream) {
  return act_kind == FP8_ACT_BF16  ? launch_act<FP8_ACT_BF16>(a, stream)
         : act_kind == FP8_ACT_FP8 ? launch_act<FP8_ACT_FP8>(a, stream)
                                   : launch_act<kF8Exact>(a, stream);
}

}  // namespace nvfp4
