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
// Measured: 2048 x 14336 x 4096 W8A8 129 us (1.86 PFLOP/s), 8192 rows 447 us (2.15; the library's
// product with one scale for all 403). There the matrix cores are busy 50 % of the cycles and the
// vector units, with the scales' FMAs, 41 %, at 1.97 GHz: data of zeros, which take less power, run
// 373 us; without the FMAs it would be 378, with loads from one hot line 405. BF16 activations 214
// us, fp32 results of W8A8 242: both decode in the vector units.
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
  static constexpr int RX = 16 * T / XB, RW = 16 * T / WB;  // rows of a load
  // scales of activation rows: one load of a window in four stages, out of range in the others
  static constexpr int NS = F8 ? 1 : 0, WS = 4;
  static constexpr int LOADS = NX + NW + NS;
  static constexpr int KF = F8 && !FAST ? 4 : 2;              // register groups of a row's k
  static constexpr int PER = (LOADS + TX / 2 - 1) / (TX / 2);  // loads of a step
  static constexpr int X0 = 0, W0 = BM * XB, STAGE = W0 + BN * WB;
  static constexpr int WIN = F8 ? BM * 16 : 0;
  static constexpr int WIN0 = D * STAGE, SINK = WIN0 + 2 * WIN;  // SINK: bytes that nobody reads
  static constexpr int LDS = SINK + (F8 ? 1024 : 0);
  static_assert(D - 1 <= WS, "a window is in use until it is overwritten");
  static_assert(16 * TW * 16 * 4 * WX * WW <= LDS, "the results' way out");
  static_assert(NX * 16 * T == BM * XB && NW * 16 * T == BN * WB, "whole loads only");
  static_assert(LDS <= 160 * 1024 && BM <= T, "LDS");
  static_assert(TX % 2 == 0 && TW % 4 == 0, "weight rows come in groups of 64 (SwiGLU: 32 + 32)");
};

// slot of piece q of a weight row of 64 bytes is q ^ quarter_swizzle(row)
__device__ __forceinline__ int quarter_swizzle(int row) {
  const int a = (row >> 2) & 3;
  return ((a & 1) << 1) ^ ((a >> 1) * 3);
}

// Eight values (BF16 ones) of a block, quantized. most: where the WW waves' largest magnitudes of the
// row lie, `pitch` apart; *scale is the block's.
template <int WW>
__device__ __forceinline__ uint2 quantize_block8(const float* most, int pitch, const uint32_t (&pairs)[4], float* scale) {
  float amax = most[0];
#pragma unroll
  for (int w = 1; w < WW; w++) {  // (as bits: what is not finite is largest)
    const float m = most[w * pitch];
    amax = __float_as_uint(m) > __float_as_uint(amax) ? m : amax;
  }
  if (__float_as_uint(amax) >= 0x7F800000u) {
    *scale = __uint_as_float(0x7FC00000u);
    return make_uint2(0u, 0u);
  }
  *scale = f8_scale<FP8_SCALE_F32>(amax);
  float v[8];
  uint32_t codes[2];
  f8_values<4>(pairs, v);
  f8_codes<8>(v, amax, *scale, codes);
  return make_uint2(codes[0], codes[1]);
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

  // What every workgroup does in the end: its share of dropped routes' rows, if the grouping has
  // fewer places than there are routes (looking for them took 6 of 200 us where there are none).
  const bool dropped = GROUPED && a.offsets[a.num_experts] < (int32_t)a.R;
  const auto finish = [&] {
    if constexpr (GROUPED) {
      if (dropped) clear_dropped<SWIGLU>(a);
    }
  };
  // tile of this workgroup: each XCD (blockIdx % 8) takes a run of tiles, which share
  // operands through its L2 (the parts of a list tile among them)
  int64_t mt, nt;
  int part = 0;
  {
    const uint32_t parts = GROUPED ? a.tile_rows / S::BM : 1;
    uint32_t nbm = GROUPED ? *a.n_tiles : (uint32_t)((a.M + S::BM - 1) / S::BM);
    if (GROUPED) {
      nbm = nbm < (uint32_t)a.max_tiles ? nbm : (uint32_t)a.max_tiles;
    }
    const uint32_t total = nbm * nbn * parts;
    if (blockIdx.x >= total) {
      finish();
      return;
    }
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
  int32_t slot0 = 0, route[GROUPED ? S::NX : 1], scale_route = 0;
  if (GROUPED) {
    const int e = in_experts(a, a.tiles[2 * mt]);
    slot0 = in_routes(a, a.tiles[2 * mt + 1]) + part * S::BM;
    // the routes of this lane's loads, not waiting for how many there are
#pragma unroll
    for (int i = 0; i < S::NX; i++) route[i] = a.sorted[in_routes(a, slot0 + i * S::RX + (tid >> 3))];
    scale_route = S::F8 ? a.sorted[in_routes(a, slot0 + tid)] : 0;
    rows_m = run_length(a, slot0, a.offsets[e + 1], S::BM);
    if (rows_m == 0) {
      finish();
      return;
    }
    wc += (int64_t)e * N * K;
    ws += (int64_t)e * ((N + 127) >> 7) * kb;
  } else {
    m0 = mt * S::BM;
    rows_m = a.M - m0 < S::BM ? a.M - m0 : S::BM;
  }

  // x row of a route
  const auto x_row = [&](int32_t route) -> int64_t {
    return a.rows_per_token ? (uint32_t)route / (uint32_t)a.top_k : (uint32_t)route;
  };
  constexpr int XE = S::F8 ? 1 : 2;  // bytes of an activation
  const int64_t xpitch = a.ldx * XE;
  const int64_t x_last = GROUPED ? a.x_rows : rows_m;
  const u32x4 xr = lds_load_rsrc(static_cast<const uint8_t*>(a.x) + (GROUPED ? 0 : m0 * xpitch),
                                 (x_last - 1) * xpitch + (int64_t)K * XE);
  const int64_t w0 = SWIGLU ? 0 : n0;  // weight row that the offsets count from
  const u32x4 wr = lds_load_rsrc(wc + w0 * K, (N - w0) * K);
  const auto w_swizzle = [](int t) { return ((t >> 1) & 1) | ((t / (4 * P)) & 3) << 1; };

  // This lane's loads of stage 0; a stage on, offsets grow by XB / WB. Load i is RX / RW rows
  // further down than load 0 (a group's rows are gathered), at the same piece of its row, or where
  // the swizzle goes by the load's parity at one of two. Rows past the tile's lie past the
  // descriptor; gate and up (half % 128 == 0) end with a tile.
  constexpr bool ODD = S::F8 && (S::RW / (4 * P) & 3) != 0;
  static_assert(!ODD || (S::RW / (4 * P) & 3) == 2, "two places, 4 pieces apart");
  int xk, wk[2];
  uint32_t xo[GROUPED ? S::NX : 1], wo[2];
  {
    const int r = tid >> 3;
    int q = (tid & 7) ^ ((r >> 1) & 7);
    if (!S::F8) q = (q & 3) << 1 | q >> 2;
    xk = q * (16 / XE);
#pragma unroll
    for (int i = 0; i < (GROUPED ? S::NX : 1); i++) {
      if constexpr (GROUPED)
        xo[i] = i * S::RX + r < rows_m ? (uint32_t)(x_row(route[i]) * xpitch) + 16 * q : kOutOfRange;
      else
        xo[i] = (uint32_t)(r * xpitch) + 16 * q;
    }
  }
  {
    int t, q;
    if (S::F8) {
      t = tid >> 3;
      q = (tid & 7) ^ w_swizzle(t);
    } else {  // rows in the order of the MFMA's: tid / 4 is row tid / 4 % 16 of 16-row tile `wave`
      const int r = (tid >> 2) & 15;
      t = (wave / P) * 16 * P + 4 * P * (r >> 2) + 4 * (wave % P) + (r & 3);
      q = (tid & 3) ^ quarter_swizzle(r);
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int qi = ODD && i ? q ^ 4 : q;
      wk[i] = 16 * qi;
      wo[i] = (uint32_t)((n0 - w0 + t) * K) + 16 * qi;
    }
  }
  const uint32_t x_step = (uint32_t)(S::RX * xpitch), w_step = (uint32_t)(S::RW * K);
  const uint32_t up = SWIGLU ? (uint32_t)((half - BC) * K) : 0u;  // from gate to up, past the tile's own rows
  u32x4 xsr = xr;
  uint32_t so = kOutOfRange;
  if (S::F8) {
    xsr = lds_load_rsrc(a.x_scales + (GROUPED ? 0 : m0 * kb), 4 * x_last * kb);
    if (tid < S::BM && tid < rows_m) so = (uint32_t)(4 * (GROUPED ? x_row(scale_route) : tid) * kb);
  }

  const uint32_t lds0 = lds_address(smem);
  // the i-th load of stage st
  const auto issue = [&](int st, int buf, int i) {
    const uint32_t to = lds0 + buf * S::STAGE + wave * 1024;
    const int k0 = st * S::SK;
    if (i < S::NX) {
      lds_load<16>(xr, k0 + xk < K ? xo[GROUPED ? i : 0] + (GROUPED ? 0 : i * x_step) + st * S::XB : kOutOfRange,
                   to + S::X0 + i * S::T * 16);
    } else if (i < S::NX + S::NW) {
      i -= S::NX;
      lds_load<16>(wr, (k0 + wk[ODD ? i & 1 : 0] < K ? wo[ODD ? i & 1 : 0] + st * S::WB : kOutOfRange) + i * w_step +
                           (i * S::RW >= BC ? up : 0),
                   to + S::W0 + i * S::T * 16);
    } else {
      const bool now = st % S::WS == 0 && st < kb && wave * 64 < S::BM;
      lds_load<16>(xsr, now ? so + 4 * st : kOutOfRange,
                   now ? lds0 + S::WIN0 + st / S::WS % 2 * S::WIN + wave * 1024 : lds0 + S::SINK);
    }
  };

  // scales of this wave's groups of weight rows
  const float* wsp[GROUPS];
#pragma unroll
  for (int i = 0; i < GROUPS; i++) {
    const int64_t n = SWIGLU ? n0 + ww * 32 + i * half : n0 + ww * 64;
    wsp[i] = ws + (n < N ? n >> 7 : 0) * kb;
  }
  // this lane's scale of each group, of 64 blocks from b on; waited for by themselves, because a wait
  // at their use would be for loads into LDS as well
  float w_scale[GROUPS];
  const auto load_scales = [&](int b) {
#pragma unroll
    for (int i = 0; i < GROUPS; i++) w_scale[i] = b + lane < kb ? wsp[i][b + lane] : 0.f;
  };
  const auto wait_scales = [&] {
#pragma unroll
    for (int i = 0; i < GROUPS; i++) asm volatile("" : "+v"(w_scale[i]));
  };
  load_scales(0);
  const int steps = (K + S::SK - 1) / S::SK;
  const auto piece = [](const uint8_t* p) { return *reinterpret_cast<const u32x4*>(p); };
  f32x4 acc[S::TW][S::TX];
#pragma unroll
  for (int t = 0; t < S::TW; t++)
#pragma unroll
    for (int x = 0; x < S::TX; x++) acc[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};

  // first tile row of the group of this wave's weight tile t; tile row of the tile's MFMA row
  // 4a + b
  const auto w_group = [&](int t) { return SWIGLU ? t / P * BC + ww * 16 * P : (ww * GROUPS + t / P) * 16 * P; };
  const auto w_local = [&](int t, int row) { return w_group(t) + 4 * P * (row >> 2) + 4 * (t % P) + (row & 3); };
  // where this lane reads: its pieces of an activation row and of a weight row (the second lies 64
  // bytes on or back), and the row's scale
  const int xrow = wx * S::TX * 16 + c;
  const int x_at = S::X0 + xrow * 128 + ((g ^ ((xrow >> 1) & 7)) << 4);
  const int wrow = w_local(0, c);
  const int w_at = S::F8 ? S::W0 + wrow * 128 + ((g ^ w_swizzle(wrow)) << 4)
                         : S::W0 + w_group(0) * 64 + 64 * c + ((g ^ quarter_swizzle(c)) << 4);
  // from weight tile 0 to tile t
  const auto w_off = [&](int t) {
    return SWIGLU ? t / P * BC * S::WB + t % P * (S::F8 ? 4 * 128 : 1024) : S::F8 ? t * 4 * 128 : t * 1024;
  };
  static_assert(SWIGLU || GROUPS == 1, "");

  u32x4 wf[S::TW][S::KF], xq[2][2];
  float sx[2];
  const auto read_w = [&](int buf) {
    const uint8_t* const l = smem + buf * S::STAGE;
#pragma unroll
    for (int t = 0; t < S::TW; t++) {
      const u32x4 w0 = piece(l + w_at + w_off(t));
      if constexpr (!S::F8) {
        wf[t][0] = f8_decode8(w0[0], w0[1]);
        wf[t][1] = f8_decode8(w0[2], w0[3]);
      } else {
        const u32x4 w1 = piece(l + (w_at ^ 64) + w_off(t));
        if constexpr (S::FAST) {
          wf[t][0] = w0;
          wf[t][1] = w1;
        } else {
          f8_decode32(w0, w1, wf[t]);
        }
      }
    }
  };
  const auto read_x = [&](int st, int buf, int x) {
    const uint8_t* const l = smem + buf * S::STAGE + x * 2048;
    xq[x & 1][0] = piece(l + x_at);
    xq[x & 1][1] = piece(l + (x_at ^ 64));
    if (S::F8)
      sx[x & 1] = *reinterpret_cast<const float*>(smem + S::WIN0 + st / S::WS % 2 * S::WIN + st % S::WS * 4 + xrow * 16 + x * 256);
  };
  // products of a row tile, and the scale of each group of weight rows that they are added with
  f32x4 p[2][S::TW];
  float sc[2][GROUPS];
  const auto add = [&](int x) {
#pragma unroll
    for (int t = 0; t < S::TW; t++)
#pragma unroll
      for (int i = 0; i < 4; i++) acc[t][x][i] = __builtin_fmaf(p[x & 1][t][i], sc[x & 1][t / P], acc[t][x][i]);
  };
#pragma unroll
  for (int t = 0; t < S::TW; t++) p[1][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < GROUPS; i++) sc[1][i] = 0.f;

  // stage by stage, as the waits count them; in a stage the weight first, because a group's
  // activation rows are still being looked up
#pragma unroll
  for (int s = 0; s < S::D - 1; s++) {
#pragma unroll
    for (int i = S::NX; i < S::NX + S::NW; i++) issue(s, s, i);
#pragma unroll
    for (int i = 0; i < S::NX; i++) issue(s, s, i);
    if (S::NS) issue(s, s, S::NX + S::NW);
  }
  wait_loads_barrier<(S::D - 2) * S::LOADS>();
  read_w(0);
  read_x(0, 0, 0);
  wait_scales();
  int buf = 0;
  for (int st = 0; st < steps; st++) {
    const int b = S::F8 ? st : st >> 1;  // block of scales
    if (st > 0 && st % (64 * 128 / S::SK) == 0) {
      load_scales(b);
      wait_scales();
    }
    const int next = buf + 1 == S::D ? 0 : buf + 1, free = buf == 0 ? S::D - 1 : buf - 1;
    float sw[GROUPS];
#pragma unroll
    for (int i = 0; i < GROUPS; i++)
      sw[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w_scale[i]), b & 63));
    // Step x: the MFMAs of row tile x, the reads of tile x + 1, the FMAs of tile x - 1, and in the
    // stage's first half the loads of the stage that is D - 1 on.
#pragma unroll
    for (int x = 0; x < S::TX; x++) {
#pragma unroll
      for (int i = x * S::PER; i < (x + 1) * S::PER && i < S::LOADS; i++) issue(st + S::D - 1, free, i);
      u32x4 xf[S::KF];
      if constexpr (S::F8 && !S::FAST) {
        f8_decode32(xq[x & 1][0], xq[x & 1][1], xf);
      } else {
        xf[0] = xq[x & 1][0];
        xf[1] = xq[x & 1][1];
      }
#pragma unroll
      for (int i = 0; i < GROUPS; i++) sc[x & 1][i] = S::F8 ? sw[i] * sx[x & 1] : sw[i];
      if (x + 1 < S::TX) read_x(st, buf, x + 1);
#pragma unroll
      for (int t = 0; t < S::TW; t++) {
        f32x4 q = {0.f, 0.f, 0.f, 0.f};
        if constexpr (S::FAST) {
          q = mfma_f8(wf[t][0], wf[t][1], xf[0], xf[1], q);
        } else {
#pragma unroll
          for (int j = 0; j < S::KF; j++) q = mfma16(wf[t][j], xf[j], q);
        }
        p[x & 1][t] = q;
      }
      if (x + 1 == S::TX) {
        // the stage has been read, and the next one is there when all waves have come here
        __builtin_amdgcn_sched_barrier(0);
        wait_loads_barrier<(S::D - 2) * S::LOADS>();
        read_w(next);
        read_x(st + 1, next, 0);
      }
      add(x > 0 ? x - 1 : S::TX - 1);
      if (S::FAST && x + 1 < S::TX) {
#pragma unroll
        for (int t = 0; t < S::TW; t++) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // an MFMA
          __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);  // vector operations
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    buf = next;
  }
  add(S::TX - 1);
  wait_loads_barrier<0>();  // nothing writes LDS after this, and the other waves have read their last stage

  if constexpr (SWIGLU == 0) {
    const int64_t n = n0 + ww * S::TW * 16;
    uint8_t* const out = smem + wave * store_bytes<S>();
    if (n < N) {
      if (a.y_type == FP8_F32)
        store_tile<S, GROUPED, 4>(a, out, acc, wx, m0, slot0, rows_m, n, N - n, vec);
      else
        store_tile<S, GROUPED, 2>(a, out, acc, wx, m0, slot0, rows_m, n, N - n, vec);
    }
  } else {
    // tile t and tile P + t are gate and up of the same columns
    const int64_t n = n0 + w_local(0, 4 * g);
    uint32_t pair[S::TX][2 * P];  // BF16 pairs of 4P consecutive columns
#pragma unroll
    for (int x = 0; x < S::TX; x++)
#pragma unroll
      for (int s = 0; s < P; s++) {
        const f32x4 gt = acc[s][x], u = acc[P + s][x];
        pair[x][2 * s] = bf16_pair(silu(gt[0]) * u[0], silu(gt[1]) * u[1]);
        pair[x][2 * s + 1] = bf16_pair(silu(gt[2]) * u[2], silu(gt[3]) * u[3]);
      }
    if constexpr (SWIGLU == FP8_OUT_SWIGLU_FP8) {
      // The tile's columns are a block: the waves exchange each row's largest magnitudes, and the codes
      // go out through LDS, a row's 128 bytes side by side.
      static_assert(BC == 128 && P == 2, "");
      float* const most = reinterpret_cast<float*>(smem);  // [WW][BM]
      float* const scales = most + S::WW * S::BM;          // [BM]
      uint8_t* const out = smem + 4 * (S::WW + 1) * S::BM;  // [BM][128], pieces of 16 as in the operands
      static_assert((4 * (S::WW + 1) + 128) * S::BM <= S::LDS, "");
#pragma unroll
      for (int x = 0; x < S::TX; x++) {
        uint32_t m = amax_pairs<4>(pair[x]);
        uint32_t o = __shfl_xor(m, 16, 64);
        m = m > o ? m : o;
        o = __shfl_xor(m, 32, 64);
        m = m > o ? m : o;
        if (g == 0) most[ww * S::BM + xrow + 16 * x] = __uint_as_float(m);
      }
      __syncthreads();
#pragma unroll
      for (int x = 0; x < S::TX; x++) {
        const int r = xrow + 16 * x;
        float scale;
        const uint2 codes = quantize_block8<S::WW>(most + r, S::BM, pair[x], &scale);
        *reinterpret_cast<uint2*>(out + r * 128 + (((2 * ww + (g >> 1)) ^ ((r >> 1) & 7)) << 4) + 8 * (g & 1)) = codes;
        if (ww == 0 && g == 0) scales[r] = scale;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < S::BM / (S::T / 8); i++) {
        const int r = i * (S::T / 8) + (tid >> 3), q = tid & 7;
        if (r >= rows_m) break;
        const int64_t row = GROUPED ? route_at(a, slot0 + r) : m0 + r;
        *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(a.y) + row * half + n0 + 16 * q) =
            *reinterpret_cast<const u32x4*>(out + r * 128 + ((q ^ ((r >> 1) & 7)) << 4));
        if (q == 0) a.y_scales[row * (half >> 7) + (n0 >> 7)] = scales[r];
      }
    } else {
#pragma unroll
      for (int x = 0; x < S::TX; x++) {
        const int r = xrow + 16 * x;
        if (r >= rows_m) continue;
        const int64_t row = GROUPED ? route_at(a, slot0 + r) : m0 + r;
        uint16_t* const d = static_cast<uint16_t*>(a.y) + row * half + n;
        if (vec) {
#pragma unroll
          for (int s = 0; s < P / 2; s++)
            reinterpret_cast<u32x4*>(d)[s] = u32x4{pair[x][4 * s], pair[x][4 * s + 1], pair[x][4 * s + 2], pair[x][4 * s + 3]};
        } else {
#pragma unroll
          for (int i = 0; i < 4 * P; i++) d[i] = (uint16_t)(pair[x][i >> 1] >> (16 * (i & 1)));
        }
      }
    }
  }
  finish();
}

// most rows of a tile of a grouped product
constexpr int grouped_rows(int act) { return act == FP8_ACT_BF16 ? 64 : 128; }

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
    if (a.tiles) {
      k = f8_tiled<S, true, 0>;
      if constexpr (!S::FAST) {  // (which SwiGLU's products are not)
        if (a.swiglu == FP8_OUT_SWIGLU_BF16) k = f8_tiled<S, true, FP8_OUT_SWIGLU_BF16>;
        if constexpr (S::BN == 256) {
          if (a.swiglu == FP8_OUT_SWIGLU_FP8) k = f8_tiled<S, true, FP8_OUT_SWIGLU_FP8>;
        }
      }
    }
  }
  hipLaunchKernelGGL(k, dim3((uint32_t)groups), dim3(S::T), S::LDS, stream, a, gm, vec);
  return hipGetLastError();
}

// Dense products take the tile that is done first: workgroups by the rounds that 256 CUs take them
// in, times what a stage of 128 k costs in such a tile (in 10 ns, K = 4096, rounds that are full or
// nearly so: W8A8 512 x 4096 in 256 tiles of 64 x 128 takes 19.8 us, 1024 x 4096 in 256 of 128 x 128
// 25.6, 1024 x 8192 in 256 of 128 x 256 38.2, 4096 x 4096 in 256 of 256 x 256 61). Two of the smallest
// fit a CU, and are done together sooner than one after the other (1024 tiles take 49 us; 512, which
// 1024 x 4096 goes to, 28, so the choice is 2 us off there). 1500 x
// 6000 x 2048 takes 33 us in 144 tiles of 256 x 256, 39 in 288 of 128 x 256. The fp32 results of W8A8
// decode both operands, which leaves no registers for the largest tile.
struct TileCost {
  int bm, bn;
  int alone[3], pair[3];  // by kind of activations; 0: no such tile, no two on a CU
};
constexpr TileCost kTileCosts[] = {{256, 256, {356, 191, 0}, {0, 0, 0}},   {128, 256, {205, 117, 190}, {0, 0, 0}},
                                   {128, 128, {133, 80, 127}, {0, 0, 0}},  {64, 256, {134, 82, 118}, {0, 0, 0}},
                                   {64, 128, {108, 62, 92}, {137, 77, 118}}};

// Grouped ones take the largest tile that still makes about a workgroup per CU: larger ones read the
// operands less often.
constexpr int64_t kFewTiles = 200;

template <int ACT>
hipError_t launch_act(const F8Args& a, hipStream_t stream) {
  constexpr bool F8 = ACT != FP8_ACT_BF16;
  int bm = 64, bn = 128;
  if (a.tiles) {
    const int64_t cols = a.swiglu ? a.N >> 1 : a.N;
    const int64_t active = a.R < a.num_experts ? a.R : a.num_experts;
    // workgroups that tiles of m rows and n weight rows make, about
    const auto tiles = [&](int64_t m, int64_t n) { return (a.R / m + active) * ((cols + n - 1) / n); };
    const bool block = a.swiglu == FP8_OUT_SWIGLU_FP8;  // a tile's columns have to be one
    if (a.tile_rows > 64 && grouped_rows(ACT) > 64) bm = 128;
    if (block || tiles(bm, a.swiglu ? 128 : 256) >= kFewTiles) bn = 256;
  } else {
    int64_t best = INT64_MAX;
    for (const TileCost& c : kTileCosts) {
      const int64_t alone = c.alone[ACT], pair = c.pair[ACT];
      const int64_t rounds = ((a.M + c.bm - 1) / c.bm * ((a.N + c.bn - 1) / c.bn) + 255) / 256;
      const int64_t cost = pair ? rounds / 2 * pair + rounds % 2 * alone : rounds * alone;
      if (alone == 0 || cost >= best) continue;
      best = cost;
      bm = c.bm;
      bn = c.bn;
    }
  }
  if constexpr (ACT != kF8Exact) {
    if (bm == 256) return launch_shape<Shape<ACT, 256, 256, 2, 4, F8 ? 2 : 3>>(a, stream);
  }
  if (bm == 128 && bn == 256) return launch_shape<Shape<ACT, 128, 256, 2, 4, 3>>(a, stream);
  if (bm == 128) return launch_shape<Shape<ACT, 128, 128, 2, 2, F8 ? 3 : 4>>(a, stream);
  if (bn == 256) return launch_shape<Shape<ACT, 64, 256, F8 ? 2 : 1, 4, 3>>(a, stream);
  return launch_shape<Shape<ACT, 64, 128, 2, 2, F8 ? 3 : 4>>(a, stream);
}

}  // namespace

hipError_t launch_f8_tiled(const F8Args& a, int act_kind, hipStream_t stream) {
  return act_kind == FP8_ACT_BF16  ? launch_act<FP8_ACT_BF16>(a, stream)
         : act_kind == FP8_ACT_FP8 ? launch_act<FP8_ACT_FP8>(a, stream)
                                   : launch_act<kF8Exact>(a, stream);
}

}  // namespace nvfp4
