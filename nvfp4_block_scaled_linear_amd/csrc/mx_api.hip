// C ABI of the MXFP4 operators (declared and documented in mxfp4.h): argument checks on the
// host, then kernel dispatch on the caller's stream. Nothing here allocates, synchronizes or
// keeps state.
#include <stdint.h>

#include "mx_kernels.hpp"
#include "mx_plan.hpp"

using namespace nvfp4;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxK = (int64_t)1 << 22;
constexpr int64_t kMaxRows = (int64_t)1 << 22;  // rows of a launch grid of one workgroup each
constexpr int kMaxExperts = 4096;               // route grouping keeps per-expert counters in LDS

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

nvfp4_status launch_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH; }

bool is_type(int32_t t) { return t == MXFP4_BF16 || t == MXFP4_F32; }

int64_t type_bytes(int32_t t) { return t == MXFP4_BF16 ? 2 : 4; }

nvfp4_status check_k(int64_t K) {
  return K <= 0 || K > kMaxK || K % 32 != 0 ? NVFP4_ERR_SHAPE : NVFP4_OK;
}

nvfp4_status check_act(int32_t act_kind, const void* x, const uint8_t* x_scales, int64_t ldx,
                       int64_t K) {
  if (act_kind != MXFP4_ACT_BF16 && act_kind != MXFP4_ACT_MXFP4) return NVFP4_ERR_ARG;
  if (!x) return NVFP4_ERR_NULL;
  if (!aligned(x, 16)) return NVFP4_ERR_ALIGN;
  if (act_kind == MXFP4_ACT_MXFP4) return x_scales ? NVFP4_OK : NVFP4_ERR_NULL;
  if (x_scales) return NVFP4_ERR_ARG;
  if (ldx < K || ldx > kMaxDim) return NVFP4_ERR_SHAPE;
  return ldx % 8 == 0 ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

nvfp4_status check_weight(const uint8_t* w_codes, const uint8_t* w_scales) {
  if (!w_codes || !w_scales) return NVFP4_ERR_NULL;
  return aligned(w_codes, 16) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

nvfp4_status check_flags(uint32_t flags, const uint32_t* faults) {
  if (flags & ~(uint32_t)NVFP4_F_CHECK) return NVFP4_ERR_ARG;
  if ((flags & NVFP4_F_CHECK) && !faults) return NVFP4_ERR_NULL;
  return faults && !aligned(faults, 4) ? NVFP4_ERR_ALIGN : NVFP4_OK;
}

// check mode: n_w weight scale bytes and `rows` activation rows
hipError_t check_data(int32_t act_kind, const void* x, const uint8_t* x_scales, int64_t ldx,
                      int64_t rows, int64_t K, const uint8_t* w_scales, int64_t n_w,
                      uint32_t* faults, hipStream_t s) {
  const hipError_t e = launch_mx_check_scales(w_scales, n_w, faults, s);
  if (e != hipSuccess) return e;
  return act_kind == MXFP4_ACT_MXFP4 ? launch_mx_check_scales(x_scales, rows * (K / 32), faults, s)
                                     : launch_check_bf16(x, ldx, rows, K, faults, s);
}

// The kernels address activation rows and one expert's weight with 32-bit buffer offsets.
bool fits(int64_t rows, int64_t pitch_bytes) { return rows * pitch_bytes < (int64_t)1 << 31; }

int64_t x_pitch(int32_t act_kind, int64_t ldx, int64_t K) {
  return act_kind == MXFP4_ACT_MXFP4 ? K / 2 : ldx * 2;
}

// Whether a dense product streams the weight (for runs of 64 rows, K split between the waves of
// a workgroup) or takes LDS tiles. Up to 32 rows the weight is read once. For more, what
// counts is how many runs of 64 rows x 32 columns there are for 256 CUs: with K = 4096, BF16
// activations, 256 of them (128 x 4096) take 12.4 us against 29.0 in tiles, 512 (256 x 4096)
// 23.3 against 30.1, 768 (128 x 12288) 34.2 against 30.2; with MXFP4 ones 256 take 7.1 against
// 10.7, 384 (64 x 12288) 11.4 against 11.3. Both sides grow with K, and no border in runs serves
// every K better by more than an eighth: BF16, 512 take 8.7 against 7.8 with K = 512, 15.5 against
// 17.2 with 2048, 65.5 against 92.6 with 14336, 768 take 12.2 against 7.6 with 512 and 98.6
// against 93.1 with 14336; MXFP4, 256 take 3.7 against 4.8 with 512 and 24.8 against 28.1 with
// 14336, 384 take 4.3 against 5.1 and 43.1 against 28.1.
bool streams(int32_t act_kind, int64_t M, int64_t N) {
  return M <= 32 || (M + 63) / 64 * ((N + 31) / 32) <= (act_kind == MXFP4_ACT_BF16 ? 550 : 300);
}

// Routes per active expert from which the grouped call works in tiles, and in tiles of 128
// routes (see RoutePlan). 32 experts, top-4, 2048 x 2048: 64 tokens take 21.0 us by slots and
// 28.3 in tiles, 96 26.0 and 28.4, 128 30.6 and 28.8, 256 45.0 and 31.2 (MXFP4 activations 18.1
// and 22.0, 24.5 and 22.3, 29.1 and 22.6, 40.6 and 23.8). 256 tokens take 31.3 in tiles of 64 and
// 38.1 in tiles of 128, 512 tokens 41.7 and 41.5 (MXFP4 23.7 and 24.0, 32.5 and 27.5). Without the
// scan, a layer of 128 experts, top-8, takes 21.3 us for one token and 64.3 for 16 against 17.3
// and 62.0.
constexpr int64_t kTiledRoutes = 16;
constexpr int64_t kTile128Routes = 64;

}  // namespace

extern "C" {

nvfp4_status mxfp4_quantize(int32_t x_type, const void* x, int64_t ldx, int64_t M, int64_t K,
                            uint8_t* codes, uint8_t* scales, uint32_t* faults, void* stream) {
  nvfp4_status st;
  if ((st = check_k(K)) != NVFP4_OK) return st;
  if (!is_type(x_type)) return NVFP4_ERR_ARG;
  if (M <= 0 || M > kMaxRows || ldx < K || ldx > kMaxDim) return NVFP4_ERR_SHAPE;
  if (!x || !codes || !scales) return NVFP4_ERR_NULL;
  if (!aligned(x, 16) || (ldx * type_bytes(x_type)) % 16 != 0) return NVFP4_ERR_ALIGN;
  if (!aligned(codes, 16) || (faults && !aligned(faults, 4))) return NVFP4_ERR_ALIGN;
  return launch_status(launch_mx_quantize(x_type, x, ldx, M, K, codes, scales, faults,
                                          static_cast<hipStream_t>(stream)));
}

nvfp4_status mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K,
                              int32_t y_type, void* y, int64_t ldy, void* stream) {
  nvfp4_status st;
  if ((st = check_k(K)) != NVFP4_OK) return st;
  if (!is_type(y_type)) return NVFP4_ERR_ARG;
  if (M <= 0 || M > kMaxRows || ldy < K || ldy > kMaxDim) return NVFP4_ERR_SHAPE;
  if (!y || !codes || !scales) return NVFP4_ERR_NULL;
  if (!aligned(y, 16) || (ldy * type_bytes(y_type)) % 16 != 0 || !aligned(codes, 16))
    return NVFP4_ERR_ALIGN;
  return launch_status(launch_mx_dequantize(codes, scales, M, K, y_type, y, ldy,
                                            static_cast<hipStream_t>(stream)));
}

nvfp4_status mxfp4_linear(int32_t act_kind, const void* x, const uint8_t* x_scales, int64_t ldx,
                          int64_t M, int64_t N, int64_t K, const uint8_t* w_codes,
                          const uint8_t* w_scales, int32_t y_type, void* y, int64_t ldy,
                          uint32_t flags, uint32_t* faults, void* stream) {
  nvfp4_status st;
  if ((st = check_flags(flags, faults)) != NVFP4_OK) return st;
  if ((st = check_k(K)) != NVFP4_OK) return st;
  if (!is_type(y_type)) return NVFP4_ERR_ARG;
  if (M <= 0 || N <= 0 || M > kMaxRows || N > kMaxRows) return NVFP4_ERR_SHAPE;
  if ((st = check_act(act_kind, x, x_scales, ldx, K)) != NVFP4_OK) return st;
  if ((st = check_weight(w_codes, w_scales)) != NVFP4_OK) return st;
  if (!y) return NVFP4_ERR_NULL;
  if (ldy < N || ldy > kMaxDim) return NVFP4_ERR_SHAPE;
  if (!aligned(y, (uintptr_t)type_bytes(y_type))) return NVFP4_ERR_ALIGN;
  if (!fits(M < 256 ? M : 256, x_pitch(act_kind, ldx, K))) return NVFP4_ERR_SHAPE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (flags & NVFP4_F_CHECK) {
    const hipError_t e =
        check_data(act_kind, x, x_scales, ldx, M, K, w_scales, N * (K / 32), faults, s);
    if (e != hipSuccess) return NVFP4_ERR_LAUNCH;
  }
  MxArgs a{};
  a.x = x; a.x_scales = x_scales; a.ldx = ldx;
  a.w_codes = w_codes; a.w_scales = w_scales;
  a.M = a.x_rows = M; a.N = N; a.K = K;
  a.y = y; a.ldy = ldy; a.y_type = y_type;
  return launch_status(streams(act_kind, M, N) ? launch_mx_stream(a, act_kind, M, s) : launch_mx_tiled(a, act_kind, s));
}

nvfp4_status mxfp4_grouped_linear(int32_t act_kind, const void* x, const uint8_t* x_scales,
                                  int64_t ldx, int32_t rows_mode, int64_t T, int32_t top_k,
                                  int64_t N, int64_t K, int32_t num_experts,
                                  const uint8_t* w_codes, const uint8_t* w_scales,
                                  const int32_t* topk_ids, const float* topk_w,
                                  int32_t out_mode, int32_t y_type, void* y, uint8_t* y_scales,
                                  void* workspace, size_t* workspace_bytes, uint32_t flags,
                                  uint32_t* faults, void* stream) {
  nvfp4_status st;
  if (!workspace_bytes) return NVFP4_ERR_NULL;
  if ((st = check_flags(flags, faults)) != NVFP4_OK) return st;
  const bool reuse = (out_mode & NVFP4_OUT_REUSE_GROUPING) != 0;
  out_mode &= ~(int32_t)NVFP4_OUT_REUSE_GROUPING;
  if (reuse && out_mode != MXFP4_OUT_COMBINE) return NVFP4_ERR_ARG;
  if ((st = check_k(K)) != NVFP4_OK) return st;
  if (num_experts <= 0 || num_experts > kMaxExperts) return NVFP4_ERR_ARG;
  if (top_k <= 0 || top_k > num_experts || top_k > 64) return NVFP4_ERR_ARG;
  if (rows_mode != NVFP4_ROWS_PER_TOKEN && rows_mode != NVFP4_ROWS_PER_ROUTE) return NVFP4_ERR_ARG;
  if (out_mode < MXFP4_OUT_ROUTES || out_mode > MXFP4_OUT_SWIGLU_MXFP4) return NVFP4_ERR_ARG;
  if (!is_type(y_type)) return NVFP4_ERR_ARG;
  const bool swiglu = out_mode == MXFP4_OUT_SWIGLU_BF16 || out_mode == MXFP4_OUT_SWIGLU_MXFP4;
  if (swiglu && y_type != MXFP4_BF16) return NVFP4_ERR_ARG;
  if (T <= 0 || N <= 0 || T > kMaxRows || N > kMaxRows || T * top_k > kMaxRows)
    return NVFP4_ERR_SHAPE;
  if (out_mode == MXFP4_OUT_SWIGLU_BF16 && N % 2 != 0) return NVFP4_ERR_SHAPE;
  if (out_mode == MXFP4_OUT_SWIGLU_MXFP4 && N % 64 != 0) return NVFP4_ERR_SHAPE;
  if (!fits(N, K / 2)) return NVFP4_ERR_SHAPE;
  const RoutePlan plan = plan_routes(T, top_k, num_experts, kTiledRoutes, kTile128Routes);
  const RouteLayout L = layout_routes(plan, T, top_k, num_experts, out_mode == MXFP4_OUT_COMBINE ? 4 * (size_t)N : 0);
  if (!workspace) {
    *workspace_bytes = L.total;
    return NVFP4_OK;
  }
  if (*workspace_bytes < L.total) return NVFP4_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return NVFP4_ERR_ALIGN;
  if ((st = check_act(act_kind, x, x_scales, ldx, K)) != NVFP4_OK) return st;
  if ((st = check_weight(w_codes, w_scales)) != NVFP4_OK) return st;
  if (!topk_ids || !y) return NVFP4_ERR_NULL;
  if (out_mode == MXFP4_OUT_COMBINE && !topk_w) return NVFP4_ERR_NULL;
  if (out_mode == MXFP4_OUT_SWIGLU_MXFP4 ? !y_scales : y_scales != nullptr)
    return y_scales ? NVFP4_ERR_ARG : NVFP4_ERR_NULL;
  if (!aligned(topk_ids, 4) || (topk_w && !aligned(topk_w, 4))) return NVFP4_ERR_ALIGN;
  if (!aligned(y, out_mode == MXFP4_OUT_SWIGLU_MXFP4 ? 16 : (uintptr_t)type_bytes(y_type)))
    return NVFP4_ERR_ALIGN;

  const int64_t R = T * top_k, active = R < num_experts ? R : num_experts;
  const int64_t xrows = rows_mode == NVFP4_ROWS_PER_TOKEN ? T : R;
  if (!fits(xrows, x_pitch(act_kind, ldx, K))) return NVFP4_ERR_SHAPE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (flags & NVFP4_F_CHECK) {
    const hipError_t e = check_data(act_kind, x, x_scales, ldx, xrows, K, w_scales,
                                    (int64_t)num_experts * N * (K / 32), faults, s);
    if (e != hipSuccess) return NVFP4_ERR_LAUNCH;
  }
  float* rows = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.rows);
  MxArgs a{};
  a.x = x; a.x_scales = x_scales; a.ldx = ldx;
  a.w_codes = w_codes; a.w_scales = w_scales;
  a.N = N; a.K = K;
  a.R = R; a.x_rows = xrows; a.rows_per_token = rows_mode == NVFP4_ROWS_PER_TOKEN ? 1 : 0;
  a.top_k = top_k; a.num_experts = num_experts;
  a.y = y; a.y_scales = y_scales; a.ldy = N; a.y_type = y_type;
  a.swiglu = swiglu ? out_mode : 0;
  a.zero_dropped = out_mode != MXFP4_OUT_COMBINE;
  if (out_mode == MXFP4_OUT_COMBINE) {
    a.y = rows;
    a.y_type = MXFP4_F32;
  }
  hipError_t e = prepare_routes(a, plan, L, workspace, topk_ids, T, reuse, faults, s);
  if (e != hipSuccess) return NVFP4_ERR_LAUNCH;
  e = plan.scan || plan.slots ? launch_mx_stream(a, act_kind, (R + active - 1) / active, s)
                              : launch_mx_tiled(a, act_kind, s);
  if (e != hipSuccess) return NVFP4_ERR_LAUNCH;
  if (out_mode == MXFP4_OUT_COMBINE)
    e = launch_mx_combine(rows, N, topk_ids, topk_w, T, top_k, num_experts, N, y_type, y, N, s);
  return launch_status(e);
}

}  // extern "C"
