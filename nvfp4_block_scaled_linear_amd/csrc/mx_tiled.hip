// MXFP4 products in LDS tiles, for enough activation rows to fill them.
//
// A workgroup computes BM activation rows x BN weight rows; its WX x WW waves share the tile,
// each 16 * TX rows by 16 * TW weight rows of 16x16 MFMAs with the weight rows as A, so that a
// lane's results run along an output row. K goes by in stages through a ring of D LDS buffers:
//  - Loads go from memory straight into LDS (buffer_load ... lds), D - 1 stages ahead, with no
//    registers in between. They are written as instructions without outputs, which the
//    compiler does not wait for; one counted wait and one barrier per stage stand before its
//    reads. Past the end of K (and of the rows) the loads are out of range and write zeros,
//    so every stage issues the same number and the count holds to the last one.
//  - A stage is 256 k of codes for MXFP4 activations (128 bytes, a cache line, of a row on both
//    sides), 64 k for BF16 ones (128 bytes of activations, 32 of codes).
//  - LDS rows have no padding (the loads write 1 KiB runs); 16-byte piece q of a row lies at
//    slot q ^ f(row), with f such that the 16 rows that lanes read together fall into
//    different banks. (A 16-byte read takes lanes of two neighbouring g together, whose pieces
//    have to differ in the lowest bit: piece 2g + j of BF16 rows counts as g + 4j.)
//  - Weight row 4P * a + 4s + b of a group of 16P rows is row 4a + b of the MFMA of its s-th
//    16-row tile (P tiles to a group): a lane's results are then 4P consecutive columns, so
//    it stores 16 bytes at a time and holds a block's half or quarter when SwiGLU's result is
//    quantized.
//
// 8192 x 14336 x 4096 with MXFP4 activations takes 251 to 259 us (3.7 PFLOP/s; the matrix cores are
// busy 45 % of the time, the rest is loads from beyond L2, LDS reads and the stores of 235 MB),
// 2048 x 14336 x 4096 with BF16 ones 195 to 205 (58 %; 448 tiles on 256 CUs leave an eighth of the
// launch idle, and decoding takes VALU time). 512 x 4096 x 4096 MXFP4 takes 14.0 with its weight
// from HBM, 12.7 otherwise. A prompt's layer of 128 experts, 32768 routes, spends 129 us in gate_up
// (2048 -> 2 x 768; matrix cores 23 %) and 120 in down (768 -> 2048, three stages and then 268 MB
// of fp32 rows; 12 %), with BF16 activations 234 and 216 (45 and 26 %).
#include <type_traits>

#include "mx_device.hpp"
#include "mx_kernels.hpp"
#include "mx_routes.hpp"
#include "mx_tile.hpp"

namespace nvfp4 {
namespace {

// SHIFT: scale rows that are not dword-aligned, or K that ends inside a stage.
template <int ACT_, int BM_, int BN_, int WX_, int WW_, int D_, bool SHIFT_>
struct Shape {
  static constexpr int ACT = ACT_, BM = BM_, BN = BN_, WX = WX_, WW = WW_, D = D_;
  static constexpr bool SHIFT = SHIFT_;
  static constexpr bool MX = ACT == MXFP4_ACT_MXFP4;
  static constexpr int T = 64 * WX * WW;
  static constexpr int TX = BM / WX / 16, TW = BN / WW / 16;
  static constexpr int XB = 128, WB = MX ? 128 : 32;  // bytes of a row per stage
  static constexpr int SB = MX ? 8 : 2;               // weight blocks per stage
  static constexpr int NX = BM * XB / (16 * T), NW = BN * WB / (16 * T);
  // Scales come in windows of 16 bytes a row, WS stages of them at a time (a load costs by the
  // cache lines it looks up, and every row is one), one load in WS stages and out of range in
  // the others. A SHIFT window begins up to three bytes before its first scale, at a dword.
  static constexpr int ROWS = MX ? BM + BN : BN, NS = (ROWS + T - 1) / T;
  static constexpr int WS = MX ? (SHIFT ? 1 : 2) : (SHIFT ? 6 : 8);
  static constexpr int LOADS = NX + NW + NS;
  static constexpr int X0 = 0, W0 = BM * XB, STAGE = W0 + BN * WB;
  static constexpr int WIN = NS * T * 16, WINDOWS = WS == 1 ? D : 2;
  static constexpr int WIN0 = D * STAGE, SINK = WIN0 + WINDOWS * WIN;  // SINK: bytes that nobody reads
  static constexpr int LDS = SINK + 1024;
  static_assert(SB * WS + 3 * SHIFT <= 16 && (WINDOWS - 1) * WS >= D - 1, "a window is in use until it is overwritten");
  static_assert(16 * TW * 16 * 4 * WX * WW <= LDS, "the results' way out");
  static_assert(NX * 16 * T == BM * XB && NW * 16 * T == BN * WB, "whole loads only");
  static_assert(LDS <= 160 * 1024, "LDS");
  static_assert(TW % 4 == 0, "weight rows come in groups of 64 (SwiGLU: 32 + 32)");
};

// bytes g, 4 + g, 8 + g and 12 + g of row r's 16 in a window
__device__ __forceinline__ uint32_t window_bytes(const uint8_t* win, int r, int g) {
  const u32x4 v = *reinterpret_cast<const u32x4*>(win + r * 16);
  const uint32_t lo = __builtin_amdgcn_perm(v[1], v[0], 0x0400u + 0x0101u * (uint32_t)g);
  const uint32_t hi = __builtin_amdgcn_perm(v[3], v[2], 0x0400u + 0x0101u * (uint32_t)g);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

template <class S, bool GROUPED, int SWIGLU>
__global__ __launch_bounds__(S::T) __attribute__((amdgpu_waves_per_eu(S::T == 512 ? 2 : 1, 2)))
void mx_tiled(MxArgs a, int gm, int vec) {
  constexpr int P = SWIGLU ? S::TW / 2 : 4;  // tiles of a group of weight rows
  constexpr int GROUPS = S::TW / P;          // of a wave; SwiGLU: gate, up
  static_assert(SWIGLU == 0 || P == 2, "the 32 columns of a block are 4P in each of four lanes");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int wx = wave % S::WX, ww = wave / S::WX;
  const int64_t N = a.N, K = a.K, half = N >> 1, nb = K >> 5;
  const int64_t cols = SWIGLU ? half : N;
  constexpr int BC = SWIGLU ? S::BN / 2 : S::BN;  // output columns of a tile
  const uint32_t nbn = (uint32_t)((cols + BC - 1) / BC);

  // tile of this workgroup: each XCD (blockIdx % 8) takes a run of tiles, which share
  // operands through its L2 (the parts of a list tile among them). There are at most 2^24
  // tiles; a division in 64 bits takes a hundred instructions.
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
  const uint8_t* ws = a.w_scales;
  int64_t m0 = 0, rows_m;
  int32_t slot0 = 0;
  if (GROUPED) {
    const int e = in_experts(a, a.tiles[2 * mt]);
    slot0 = in_routes(a, a.tiles[2 * mt + 1]) + part * S::BM;
    rows_m = run_length(a, slot0, a.offsets[e + 1], S::BM);
    if (rows_m == 0) return;
    wc += (int64_t)e * N * (K >> 1);
    ws += (int64_t)e * N * nb;
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
  const int64_t xpitch = S::MX ? K >> 1 : a.ldx * 2;  // bytes
  const int64_t x_last = GROUPED ? a.x_rows : rows_m;
  const u32x4 xr = lds_load_rsrc(static_cast<const uint8_t*>(a.x) + (GROUPED ? 0 : m0 * xpitch),
                             (x_last - 1) * xpitch + (S::MX ? K >> 1 : 2 * K));
  const u32x4 wr = lds_load_rsrc(wc + (SWIGLU ? 0 : n0 * (K >> 1)), (N - (SWIGLU ? 0 : n0)) * (K >> 1));
  // weight row of tile row t relative to that base, or -1
  const auto w_row = [&](int t) -> int64_t {
    if (!SWIGLU) return n0 + t < N ? t : -1;
    const int u = t >= BC ? t - BC : t;
    return n0 + u < half ? n0 + u + (t >= BC ? half : 0) : -1;
  };

  const auto w_swizzle = [](int t) { return ((t >> 1) & 1) | ((t / (4 * P)) & 3) << 1; };

  // this lane's loads of stage 0; a stage on, offsets grow by XB / WB / SB bytes
  uint32_t xo[S::NX], wo[S::NW];
  int xk[S::NX], wk[S::NW];  // first block (BF16 x: first 8-value piece) of the load
#pragma unroll
  for (int i = 0; i < S::NX; i++) {
    const int p = i * S::T + tid;
    const int r = p >> 3;
    int q = (p & 7) ^ ((r >> 1) & 7);
    if (!S::MX) q = (q & 3) << 1 | q >> 2;
    xk[i] = q;
    xo[i] = r < rows_m ? (uint32_t)(x_row(r) * xpitch) + 16 * q : kOutOfRange;
  }
#pragma unroll
  for (int i = 0; i < S::NW; i++) {
    const int p = i * S::T + tid;
    int t, q;
    if (S::MX) {
      t = p >> 3;
      q = (p & 7) ^ w_swizzle(t);
    } else {  // piece q of the row that lane p % 16 of 16-row tile p / 32 reads
      const int u = p >> 5, s = u % P;
      q = (p >> 4) & 1;
      t = (u / P) * 16 * P + 4 * P * ((p & 15) >> 2) + 4 * s + (p & 3);
    }
    wk[i] = q;
    const int64_t row = w_row(t);
    wo[i] = row >= 0 ? (uint32_t)(row * (K >> 1)) + 16 * q : kOutOfRange;
  }
  // Scales of one side: rows of nb bytes from p, counted from the dword that p lies in.
  const auto scales_of = [](const uint8_t* p, int64_t bytes) {
    const int64_t skip = (uintptr_t)p & 3;
    return lds_load_rsrc(p - skip, (skip + bytes + 3) & ~(int64_t)3);
  };
  const uint8_t* wsp = ws + (SWIGLU ? 0 : n0 * nb);
  const uint8_t* xsp = S::MX ? a.x_scales + (GROUPED ? 0 : m0 * nb) : wsp;
  const u32x4 wsr = scales_of(wsp, (N - (SWIGLU ? 0 : n0)) * nb);
  const u32x4 xsr = S::MX ? scales_of(xsp, x_last * nb) : wsr;
  // the p-th scale load is that of the p-th row, of the weight, then of the activations; the
  // weight's rows in the order in which lanes read them, 16 side by side. Whole waves read one
  // side (BN is a multiple of 64), so the descriptor is uniform.
  bool s_is_x[S::NS];
  uint32_t so[S::NS];
#pragma unroll
  for (int i = 0; i < S::NS; i++) {
    const int t = i * S::T + tid;
    s_is_x[i] = S::MX && __builtin_amdgcn_readfirstlane(t) >= S::BN;
    int64_t row = -1;
    if (t < S::BN) row = w_row(t / (16 * P) * (16 * P) + 4 * P * ((t & 15) >> 2) + 4 * ((t >> 4) % P) + (t & 3));
    else if (S::MX && t - S::BN < rows_m) row = x_row(t - S::BN);
    so[i] = row >= 0 ? ((uint32_t)(row * nb) + (uint32_t)((uintptr_t)(s_is_x[i] ? xsp : wsp) & 3)) & ~3u : kOutOfRange;
  }

  const uint32_t lds0 = lds_address(smem);
  const int nblk = (int)nb;
  const auto issue = [&](int st, int buf) {
    const uint32_t base = lds0 + buf * S::STAGE;
#pragma unroll
    for (int i = 0; i < S::NX; i++) {
      // a BF16 piece is in range when its block is: pieces 4 per block
      const int b = S::MX ? 8 * st + xk[i] : 2 * st + (xk[i] >> 2);
      lds_load<16>(xr, b < nblk ? xo[i] + st * S::XB : kOutOfRange, base + S::X0 + (i * S::T + wave * 64) * 16);
    }
#pragma unroll
    for (int i = 0; i < S::NW; i++)
      lds_load<16>(wr, S::SB * st + wk[i] < nblk ? wo[i] + st * S::WB : kOutOfRange,
                   base + S::W0 + (i * S::T + wave * 64) * 16);
#pragma unroll
    for (int i = 0; i < S::NS; i++) {
      const int w = st / S::WS;
      const bool now = st % S::WS == 0 && S::SB * st < nblk;
      lds_load<16>(s_is_x[i] ? xsr : wsr, now ? so[i] + S::SB * S::WS * w : kOutOfRange,
                   now ? lds0 + S::WIN0 + w % S::WINDOWS * S::WIN + (i * S::T + wave * 64) * 16 : lds0 + S::SINK);
    }
  };

  f32x4 acc[S::TW][S::TX];
#pragma unroll
  for (int t = 0; t < S::TW; t++)
#pragma unroll
    for (int x = 0; x < S::TX; x++) acc[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};

  // first tile row of the group of this wave's weight tile t; tile row of the tile's MFMA row
  // 4a + b; and where that row's scales are
  const auto w_group = [&](int t) { return SWIGLU ? t / P * BC + ww * 16 * P : (ww * GROUPS + t / P) * 16 * P; };
  const auto w_local = [&](int t, int row) { return w_group(t) + 4 * P * (row >> 2) + 4 * (t % P) + (row & 3); };
  const auto w_scale = [&](int t, int row) { return w_group(t) + 16 * (t % P) + row; };

  // SHIFT: where in its dword the first scale of this lane's rows lies, two bits a tile
  uint32_t w_shift = 0u, x_shift = 0u;
  if (S::SHIFT) {
#pragma unroll
    for (int t = 0; t < S::TW; t++) {
      const int64_t row = w_row(w_local(t, c));
      w_shift |= (((uint32_t)row * (uint32_t)nb + (uint32_t)(uintptr_t)wsp) & 3u) << (2 * t);
    }
    if (S::MX) {
#pragma unroll
      for (int x = 0; x < S::TX; x++) {
        const int r = (wx * S::TX + x) * 16 + c;
        const int64_t row = r < rows_m ? x_row(r) : 0;
        x_shift |= (((uint32_t)row * (uint32_t)nb + (uint32_t)(uintptr_t)xsp) & 3u) << (2 * x);
      }
    }
  }

  const int steps = (nblk + S::SB - 1) / S::SB;
#pragma unroll
  for (int i = 0; i < S::D - 1; i++) issue(i, i);
  // window scales of this lane's rows (byte 2 * phase + h: block g of half h of that stage)
  uint32_t xwin[S::TX], wwin[S::TW];
  const auto stage = [&](int st, auto phase, int buf) {
    constexpr int PH = decltype(phase)::value;
    wait_loads_barrier<(S::D - 2) * S::LOADS>();
    issue(st + S::D - 1, buf == 0 ? S::D - 1 : buf - 1);
    const uint8_t* xs = smem + buf * S::STAGE + S::X0;
    const uint8_t* wl = smem + buf * S::STAGE + S::W0;
    // scale byte of block b of the stage (g of half h: 4h + g), r-th of ROWS, shifted by sh
    const uint8_t* sl = smem + S::WIN0 + st / S::WS % S::WINDOWS * S::WIN + st % S::WS * S::SB;
    const auto scale = [&](int r, int b, uint32_t sh) -> uint32_t {
      if (!S::SHIFT) return sl[r * 16 + b];
      return S::SB * st + b < nblk ? sl[r * 16 + b + sh] : 0u;
    };
    if constexpr (S::MX) {
      if constexpr (!S::SHIFT && PH == 0) {
#pragma unroll
        for (int x = 0; x < S::TX; x++) xwin[x] = window_bytes(sl, S::BN + (wx * S::TX + x) * 16 + c, g);
#pragma unroll
        for (int t = 0; t < S::TW; t++) wwin[t] = window_bytes(sl, w_scale(t, c), g);
      }
      const auto half = [&](auto hh) {
        constexpr int H = decltype(hh)::value, SEL = !S::SHIFT ? 2 * PH + H : 0;
        u32x4 xf[S::TX];
        uint32_t xsc[S::TX];
#pragma unroll
        for (int x = 0; x < S::TX; x++) {
          const int r = (wx * S::TX + x) * 16 + c;
          xf[x] = *reinterpret_cast<const u32x4*>(xs + r * 128 + (((4 * H + g) ^ ((r >> 1) & 7)) << 4));
          xsc[x] = !S::SHIFT ? xwin[x] : scale(S::BN + r, 4 * H + g, x_shift >> (2 * x) & 3);
        }
#pragma unroll
        for (int t = 0; t < S::TW; t++) {
          const int r = w_local(t, c);
          const u32x4 wf = *reinterpret_cast<const u32x4*>(wl + r * 128 + (((4 * H + g) ^ w_swizzle(r)) << 4));
          const uint32_t s = !S::SHIFT ? wwin[t] : scale(w_scale(t, c), 4 * H + g, w_shift >> (2 * t) & 3);
#pragma unroll
          for (int x = 0; x < S::TX; x++) acc[t][x] = mfma_mx<SEL, SEL>(wf, xf[x], acc[t][x], s, xsc[x]);
        }
      };
      half(std::integral_constant<int, 0>());
      half(std::integral_constant<int, 1>());
    } else {
      u32x4 xf[S::TX][2];
      uint2 wf[S::TW];
      uint32_t ws[S::TW];
#pragma unroll
      for (int x = 0; x < S::TX; x++) {
        const int r = (wx * S::TX + x) * 16 + c;
#pragma unroll
        for (int j = 0; j < 2; j++)
          xf[x][j] = *reinterpret_cast<const u32x4*>(xs + r * 128 + (((g + 4 * j) ^ ((r >> 1) & 7)) << 4));
      }
#pragma unroll
      for (int t = 0; t < S::TW; t++) {
        const int r = w_local(t, c);
        // 16-row tile index in the order of the loads
        const int u = (r / (16 * P)) * P + (t % P);
        wf[t] = *reinterpret_cast<const uint2*>(wl + u * 512 + (((g >> 1) * 16 + c) << 4) + ((g & 1) << 3));
        ws[t] = scale(w_scale(t, c), g >> 1, w_shift >> (2 * t) & 3);
      }
#pragma unroll
      for (int t = 0; t < S::TW; t++) {
        const float s = e8m0_operand(ws[t]);
        const u32x4 w0 = mx_decode8(wf[t].x, s), w1 = mx_decode8(wf[t].y, s);
#pragma unroll
        for (int x = 0; x < S::TX; x++) acc[t][x] = mfma16(w0, xf[x][0], acc[t][x]);
#pragma unroll
        for (int x = 0; x < S::TX; x++) acc[t][x] = mfma16(w1, xf[x][1], acc[t][x]);
      }
    }
  };
  // the ring's buffers are taken in turn, by loops that are unrolled so that they are constants
  constexpr bool PAIRS = S::MX && !S::SHIFT;  // windows of two stages
  constexpr int UNROLL = PAIRS && S::D % 2 ? 2 * S::D : S::D;
  for (int st0 = 0; st0 < steps; st0 += UNROLL) {
#pragma unroll
    for (int i = 0; i < UNROLL; i++) {
      if (i && st0 + i >= steps) break;
      if (PAIRS && i % 2)
        stage(st0 + i, std::integral_constant<int, PAIRS>(), i % S::D);
      else
        stage(st0 + i, std::integral_constant<int, 0>(), i % S::D);
    }
  }
  wait_loads<0>();  // nothing writes LDS after the workgroup

  if constexpr (!SWIGLU) {
    wait_loads_barrier<0>();  // the other waves have read their last stage
    const int64_t n = n0 + ww * S::TW * 16;
    uint8_t* const out = smem + wave * store_bytes<S>();
    if (n >= N) return;
    if (a.y_type == MXFP4_F32)
      store_tile<S, GROUPED, 4>(a, out, acc, wx, m0, slot0, rows_m, n, N - n, vec);
    else
      store_tile<S, GROUPED, 2>(a, out, acc, wx, m0, slot0, rows_m, n, N - n, vec);
    return;
  }
#pragma unroll
  for (int x = 0; x < S::TX; x++) {
    const int r = (wx * S::TX + x) * 16 + c;
    const bool ok = r < rows_m;
    const int64_t row = GROUPED ? (ok ? route_at(a, slot0 + r) : 0) : m0 + r;
    // SwiGLU: tile t and tile P + t are gate and up of the same columns
    const int64_t n = n0 + w_local(0, 4 * g);
    uint32_t h[2 * P];  // BF16 pairs of 4P consecutive columns
#pragma unroll
    for (int s = 0; s < P; s++) {
      const f32x4 gt = acc[s][x], u = acc[P + s][x];
      h[2 * s] = bf16_pair(silu(gt[0]) * u[0], silu(gt[1]) * u[1]);
      h[2 * s + 1] = bf16_pair(silu(gt[2]) * u[2], silu(gt[3]) * u[3]);
    }
    if (SWIGLU == MXFP4_OUT_SWIGLU_BF16) {
      if (!ok) continue;
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
      continue;
    }
    uint32_t amax = amax_pairs<2 * P>(h);
    uint32_t o = __shfl_xor(amax, 16, 64);
    amax = amax > o ? amax : o;
    o = __shfl_xor(amax, 32, 64);
    amax = amax > o ? amax : o;
    const uint32_t sc = e8m0_of_amax(amax);
    const bool bad = amax >= 0x7F800000u;
    uint32_t code[P / 2];
#pragma unroll
    for (int i = 0; i < P / 2; i++)
      code[i] = bad ? 0u : codes_of_pairs(h[4 * i], h[4 * i + 1], sc) | codes_of_pairs(h[4 * i + 2], h[4 * i + 3], sc) << 16;
    if (!ok || n >= half) continue;  // blocks end where the columns do
    uint32_t* d = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.y) + row * (half >> 1) + (n >> 1));
#pragma unroll
    for (int i = 0; i < P / 2; i++) d[i] = code[i];
    if ((n & 31) == 0) a.y_scales[row * (half >> 5) + (n >> 5)] = (uint8_t)(bad ? kE8M0Nan : sc);
  }
}

// most rows of a tile of a grouped product
constexpr int grouped_rows(int act) { return act == MXFP4_ACT_MXFP4 ? 128 : 64; }

template <class S>
hipError_t launch_shape(const MxArgs& a, hipStream_t stream) {
  const int64_t bc = a.swiglu ? S::BN / 2 : S::BN;
  const int64_t cols = a.swiglu ? a.N >> 1 : a.N;
  const int64_t nbm = a.tiles ? a.max_tiles : (a.M + S::BM - 1) / S::BM;
  const int64_t parts = a.tiles ? a.tile_rows / S::BM : 1;
  const int64_t groups = nbm * ((cols + bc - 1) / bc) * parts;
  if (groups * S::T > (int64_t)UINT32_MAX) return hipErrorInvalidConfiguration;
  // an XCD's 32 CUs work on gm x (32 / gm) tiles (grouped: on the columns of a few list tiles)
  const int gm = a.tiles ? 1 : S::MX ? 4 : 2;
  const int64_t ysz = a.y_type == MXFP4_F32 ? 4 : 2, ld = a.swiglu ? cols : a.ldy;
  const int vec = ((uintptr_t)a.y | (uintptr_t)(ld * ysz)) % 16 == 0;
  auto k = mx_tiled<S, false, 0>;
  if constexpr (S::BM <= grouped_rows(S::ACT)) {
    if (a.tiles)
      k = a.swiglu == 0 ? mx_tiled<S, true, 0>
          : a.swiglu == MXFP4_OUT_SWIGLU_BF16 ? mx_tiled<S, true, MXFP4_OUT_SWIGLU_BF16>
                                              : mx_tiled<S, true, MXFP4_OUT_SWIGLU_MXFP4>;
  }
  hipLaunchKernelGGL(k, dim3((uint32_t)groups), dim3(S::T), S::LDS, stream, a, gm, vec);
  return hipGetLastError();
}

// The largest tile that still makes about a workgroup per CU is taken: larger ones read the
// operands less often. BF16 activations: decoding a weight (v_cvt_scalef32_pk_bf16_fp4, two
// values) takes about as long as an MFMA, and each of the WX waves that share weight rows
// decodes them for itself, so few waves stand side by side along the activations, each with
// many rows. 2048 x 14336 x 4096 takes 196 us with 2 x 4 waves, 202 with 4 x 2; 512 tokens x
// top-4 of 32 experts, 2048 x 2048, 42.6 in tiles of 64 x 256 by 1 x 4 waves, 46.7 in 64 x 128
// by 2 x 2. In a grouped product two tiles of 64 rows then stand for one of 128 on the list:
// 1024 tokens take 66 to 70 us, in tiles of 128 75. MXFP4 activations have no such cost: 512
// tokens 27.5 in tiles of 128 rows, 32.5 in tiles of 64.
constexpr int64_t kFewTiles = 200;

template <int ACT, int BM, int BN, int WX, int WW, int D>
hipError_t launch_scales(const MxArgs& a, hipStream_t stream) {
  constexpr bool MX = ACT == MXFP4_ACT_MXFP4, BIG = BM * BN == 256 * 256;
  const uintptr_t at = (uintptr_t)a.w_scales | (MX ? (uintptr_t)a.x_scales : 0);
  return a.K % (MX ? 256 : 128) == 0 && at % 4 == 0
             ? launch_shape<Shape<ACT, BM, BN, WX, WW, D, false>>(a, stream)
             // (the largest tiles have no registers left for the shifts)
             : launch_shape<Shape<ACT, (MX && BIG ? 128 : BM), BN, (!MX && BIG ? 4 : WX), (!MX && BIG ? 2 : WW), D, true>>(a, stream);
}

template <int ACT>
hipError_t launch_act(const MxArgs& a, hipStream_t stream) {
  constexpr bool MX = ACT == MXFP4_ACT_MXFP4;
  const int64_t cols = a.swiglu ? a.N >> 1 : a.N;
  const int64_t active = a.R < a.num_experts ? a.R : a.num_experts;
  // workgroups that tiles of bm rows and bn weight rows make (grouped: about)
  const auto tiles = [&](int64_t bm, int64_t bn) {
    const int64_t bc = a.swiglu ? bn / 2 : bn;
    return (a.tiles ? a.R / bm + active : (a.M + bm - 1) / bm) * ((cols + bc - 1) / bc);
  };
  const int64_t rows = !a.tiles ? a.M : a.tile_rows < grouped_rows(ACT) ? a.tile_rows : grouped_rows(ACT);
  if (rows > 128 && tiles(256, 256) >= kFewTiles) return launch_scales<ACT, 256, 256, 2, 4, MX ? 2 : 3>(a, stream);
  if (rows > 64 && tiles(128, 256) >= kFewTiles) return launch_scales<ACT, 128, 256, 2, 4, MX ? 2 : 4>(a, stream);
  if (rows > 64 && (a.tiles || tiles(128, 128) >= kFewTiles)) return launch_scales<ACT, 128, 128, 2, 2, MX ? 3 : 4>(a, stream);
  if (tiles(64, 256) >= kFewTiles) return launch_scales<ACT, 64, 256, MX ? 2 : 1, 4, 3>(a, stream);
  return launch_scales<ACT, 64, 128, 2, 2, MX ? 3 : 4>(a, stream);
}

}  // namespace

hipError_t launch_mx_tiled(const MxArgs& a, int act_kind, hipStream_t stream) {
  return act_kind == MXFP4_ACT_BF16 ? launch_act<MXFP4_ACT_BF16>(a, stream) : launch_act<MXFP4_ACT_MXFP4>(a, stream);
}

}  // namespace nvfp4
