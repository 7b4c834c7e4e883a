// C ABI of the FP8 operators and the router (declared and documented in fp8.h): argument checks
// on the host, then kernel dispatch on the caller's stream. Nothing here allocates, synchronizes
// or keeps state.
#include <stdint.h>

#include "f8_kernels.hpp"
#include "mx_plan.hpp"

using namespace nvfp4;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxK = (int64_t)1 << 22;
constexpr int64_t kMaxRows = (int64_t)1 << 22;
constexpr int kMaxExperts = 4096;  // route grouping keeps per-expert counters in LDS
constexpr int kMaxTopK = 64;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

nvfp4_status launch_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH; }

bool is_type(int32_t t) { return t == FP8_BF16 || t == FP8_F32; }

int64_t type_bytes(int32_t t) { return t == FP8_BF16 ? 2 : 4; }

int64_t blocks_of(int64_t n) { return (n + kF8Block - 1) / kF8Block; }

nvfp4_status check_k(int64_t K) {
  return K <= 0 || K > kMaxK || K % 16 != 0 ? NVFP4_ERR_SHAPE : NVFP4_OK;
}

nvfp4_status check_act(int32_t act_kind, const void* x, const float* x_scales, int64_t ldx,
                       int64_t K) {
  if (act_kind != FP8_ACT_BF16 && act_kind != FP8_ACT_FP8) return NVFP4_ERR_ARG;
  if (!x) return NVFP4_ERR_NULL;
  if (!aligned(x, 16)) return NVFP4_ERR_ALIGN;
  if (ldx < K || ldx > kMaxDim) return NVFP4_ERR_SHAPE;
  if (act_kind == FP8_ACT_BF16) {
    if (x_scales) return NVFP4_ERR_ARG;
    return ldx % 8 == 0 ? NVFP4_OK : NVFP4_ERR_ALIGN;
  }
  if (!x_scales) return NVFP4_ERR_NULL;
  return ldx % 16 == 0 && aligned(x_scales, 4) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

nvfp4_status check_weight(const uint8_t* w_codes, const float* w_scales) {
  if (!w_codes || !w_scales) return NVFP4_ERR_NULL;
  return aligned(w_codes, 16) && aligned(w_scales, 4) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

nvfp4_status check_flags(uint32_t flags, const uint32_t* faults) {
  if (flags & ~(uint32_t)NVFP4_F_CHECK) return NVFP4_ERR_ARG;
  if ((flags & NVFP4_F_CHECK) && !faults) return NVFP4_ERR_NULL;
  return faults && !aligned(faults, 4) ? NVFP4_ERR_ALIGN : NVFP4_OK;
}

// check mode: `experts` weights of N x K and `rows` activation rows
hipError_t check_data(int32_t act_kind, const void* x, const float* x_scales, int64_t ldx,
                      int64_t rows, int64_t N, int64_t K, int64_t experts, const uint8_t* w_codes,
                      const float* w_scales, uint32_t* faults, hipStream_t s) {
  hipError_t e = launch_f8_check_scales(w_scales, experts * blocks_of(N) * blocks_of(K), faults, s);
  if (e == hipSuccess) e = launch_f8_check_codes(w_codes, K, experts * N, K, faults, s);
  if (e != hipSuccess) return e;
  if (act_kind == FP8_ACT_BF16) return launch_check_bf16(x, ldx, rows, K, faults, s);
  e = launch_f8_check_scales(x_scales, rows * blocks_of(K), faults, s);
  return e != hipSuccess ? e
                         : launch_f8_check_codes(static_cast<const uint8_t*>(x), ldx, rows, K, faults, s);
}

// The kernels address activation rows and one expert's weight with 32-bit buffer offsets.
bool fits(int64_t rows, int64_t pitch_bytes) { return rows * pitch_bytes < (int64_t)1 << 31; }

// The kernels' kind of activations. FP8 ones are multiplied by FP8 matrix instructions where the
// result is rounded to BF16 and nothing more: not fp32 ones, and not SwiGLU's, which are quantized
// again. (What those sums lose moves block scales and codes: a prompt's layer, 2048 / 768, was
// 0.0025 off its 64-bit result in the 2-norm, with fp32 sums 0.0017, most of it y's own rounding; its
// gate_up takes 290 us against 200.)
int kernel_kind(int32_t act_kind, bool plain_bf16) {
  return act_kind == FP8_ACT_FP8 && !plain_bf16 ? kF8Exact : act_kind;
}

int64_t x_pitch(int32_t act_kind, int64_t ldx) { return act_kind == FP8_ACT_FP8 ? ldx : ldx * 2; }

// Whether a dense product streams the weight, for runs of 48 (BF16 activations) or 64 rows x 32
// columns, or takes LDS tiles. Up to 32 rows the weight is read once. For more, what counts is how
// many such runs there are for 256 CUs: K = 4096, BF16, 384 of them (128 x 4096) take 19.7 us against
// 32.4 in tiles, 768 (256 x 4096) 28.9 against 33.1, 1152 (128 x 12288) 47.0 against 33.6; W8A8, 256
// take 9.0 against 18.7, 512 16.4 against 18.9, 768 25.4 against 19.5; with fp32 results 512 19.9
// against 26.9, 768 28.8 against 27.6. Both sides grow with K, tiles less while launches of few
// stages cost their latency: with K = 512 704 runs take 10.7 against 7.4 (BF16), with 1024 448 take
// 9.0 against 7.7 (W8A8). (On the same operands again and again, which stay in the last-level
// cache; with weights from HBM up to 3 us more.) The borders lie between those figures and know
// nothing of K: two of the pairs above fall on their slower side, BF16's 768 runs, which go to tiles,
// and W8A8's 448 with K = 1024, which stream.
bool streams(int32_t kind, int64_t M, int64_t N) {
  const int64_t rows = kind == FP8_ACT_BF16 ? 48 : 64, most = kind == FP8_ACT_BF16 ? 600 : kind == FP8_ACT_FP8 ? 550 : 700;
  return M <= 32 || (M + rows - 1) / rows * ((N + 31) / 32) <= most;
}

// Routes per active expert from which the grouped call works in tiles, and in tiles of 128
// routes (see RoutePlan); both calls of a layer have to agree, whatever their activations are, so
// the borders are a middle between the kinds: BF16 layers of four routes an expert are 11 % slower
// by slots, W8A8 ones of six 3 % slower in tiles.
// gate_up and down of 128 experts, top-8, 2048 / 768: 64 tokens take 98 + 53 us by slots and 79 + 57
// in tiles (W8A8 83 + 52 and 90 + 58), 96 tokens 101 + 56 and 80 + 57 (89 + 56 and 91 + 59); of 32
// experts, top-4, 2048 / 1024: 48 tokens 31 + 21 and 29 + 24 (32 + 21 and 31 + 23), 96 tokens 42 + 28
// and 30 + 25 (44 + 25 and 31 + 23). 512 tokens of the latter take 44 + 36 in tiles of 64 and 58 + 45
// in tiles of 128 (53 + 36 and 75 + 40), 1024 tokens 65 + 51 and 65 + 52 (79 + 50 and 77 + 47).
constexpr int64_t kTiledRoutes = 6;
constexpr int64_t kTile128Routes = 96;

}  // namespace

extern "C" {

nvfp4_status fp8_quantize(int32_t x_type, const void* x, int64_t ldx, int64_t M, int64_t K,
                          int32_t block_rows, int32_t scale_rule, uint8_t* codes, float* scales,
                          uint32_t* faults, void* stream) {
  nvfp4_status st;
  if ((st = check_k(K)) != NVFP4_OK) return st;
  if (!is_type(x_type) || (block_rows != 1 && block_rows != kF8Block)) return NVFP4_ERR_ARG;
  if (scale_rule != FP8_SCALE_F32 && scale_rule != FP8_SCALE_POW2) return NVFP4_ERR_ARG;
  if (M <= 0 || M > kMaxRows || ldx < K || ldx > kMaxDim) return NVFP4_ERR_SHAPE;
  if (!x || !codes || !scales) return NVFP4_ERR_NULL;
  if (!aligned(x, 16) || (ldx * type_bytes(x_type)) % 16 != 0) return NVFP4_ERR_ALIGN;
  if (!aligned(codes, 16) || !aligned(scales, 4) || (faults && !aligned(faults, 4))) return NVFP4_ERR_ALIGN;
  return launch_status(launch_f8_quantize(x_type, x, ldx, M, K, block_rows, scale_rule, codes, scales,
                                          faults, static_cast<hipStream_t>(stream)));
}

nvfp4_status fp8_dequantize(const uint8_t* codes, const float* scales, int64_t M, int64_t K,
                            int32_t block_rows, int32_t y_type, void* y, int64_t ldy, void* stream) {
  nvfp4_status st;
  if ((st = check_k(K)) != NVFP4_OK) return st;
  if (!is_type(y_type) || (block_rows != 1 && block_rows != kF8Block)) return NVFP4_ERR_ARG;
  if (M <= 0 || M > kMaxRows || ldy < K || ldy > kMaxDim) return NVFP4_ERR_SHAPE;
  if (!y || !codes || !scales) return NVFP4_ERR_NULL;
  if (!aligned(y, 16) || (ldy * type_bytes(y_type)) % 16 != 0) return NVFP4_ERR_ALIGN;
  if (!aligned(codes, 16) || !aligned(scales, 4)) return NVFP4_ERR_ALIGN;
  return launch_status(launch_f8_dequantize(codes, scales, M, K, block_rows, y_type, y, ldy,
                                            static_cast<hipStream_t>(stream)));
}

nvfp4_status fp8_linear(int32_t act_kind, const void* x, const float* x_scales, int64_t ldx,
                        int64_t M, int64_t N, int64_t K, const uint8_t* w_codes,
                        const float* w_scales, int32_t y_type, void* y, int64_t ldy,
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
  if (!fits(M < 256 ? M : 256, x_pitch(act_kind, ldx))) return NVFP4_ERR_SHAPE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if ((flags & NVFP4_F_CHECK) &&
      check_data(act_kind, x, x_scales, ldx, M, N, K, 1, w_codes, w_scales, faults, s) != hipSuccess)
    return NVFP4_ERR_LAUNCH;
  F8Args a{};
  a.x = x; a.x_scales = x_scales; a.ldx = ldx;
  a.w_codes = w_codes; a.w_scales = w_scales;
  a.M = a.x_rows = M; a.N = N; a.K = K;
  a.y = y; a.ldy = ldy; a.y_type = y_type;
  const int kind = kernel_kind(act_kind, y_type == FP8_BF16);
  return launch_status(streams(kind, M, N) ? launch_f8_stream(a, kind, M, s) : launch_f8_tiled(a, kind, s));
}

nvfp4_status fp8_grouped_linear(int32_t act_kind, const void* x, const float* x_scales,
                                int64_t ldx, int32_t rows_mode, int64_t T, int32_t top_k,
                                int64_t N, int64_t K, int32_t num_experts,
                                const uint8_t* w_codes, const float* w_scales,
                                const int32_t* topk_ids, const float* topk_w, int32_t out_mode,
                                int32_t y_type, void* y, float* y_scales, void* workspace,
                                size_t* workspace_bytes, uint32_t flags, uint32_t* faults,
                                void* stream) {
  nvfp4_status st;
  if (!workspace_bytes) return NVFP4_ERR_NULL;
  if ((st = check_flags(flags, faults)) != NVFP4_OK) return st;
  const bool reuse = (out_mode & NVFP4_OUT_REUSE_GROUPING) != 0;
  out_mode &= ~(int32_t)NVFP4_OUT_REUSE_GROUPING;
  if (reuse && out_mode != FP8_OUT_COMBINE) return NVFP4_ERR_ARG;
  if ((st = check_k(K)) != NVFP4_OK) return st;
  if (num_experts <= 0 || num_experts > kMaxExperts) return NVFP4_ERR_ARG;
  if (top_k <= 0 || top_k > num_experts || top_k > kMaxTopK) return NVFP4_ERR_ARG;
  if (rows_mode != NVFP4_ROWS_PER_TOKEN && rows_mode != NVFP4_ROWS_PER_ROUTE) return NVFP4_ERR_ARG;
  const bool to_f8 = out_mode == FP8_OUT_SWIGLU_FP8, combine = out_mode == FP8_OUT_COMBINE;
  const bool swiglu = out_mode == FP8_OUT_SWIGLU_BF16 || to_f8;
  if (!swiglu && !combine && out_mode != FP8_OUT_ROUTES) return NVFP4_ERR_ARG;
  if (!is_type(y_type) || (swiglu && y_type != FP8_BF16)) return NVFP4_ERR_ARG;
  if (T <= 0 || N <= 0 || T > kMaxRows || N > kMaxRows || T * top_k > kMaxRows)
    return NVFP4_ERR_SHAPE;
  if (swiglu && N % (2 * kF8Block) != 0) return NVFP4_ERR_SHAPE;
  if (!fits(N, K)) return NVFP4_ERR_SHAPE;
  // rows that a later kernel of the call reads: fp32 to combine, BF16 to quantize
  const RoutePlan plan = plan_routes(T, top_k, num_experts, kTiledRoutes, kTile128Routes);
  const bool streams = plan.scan || plan.slots;  // (tiles quantize their own results)
  const size_t row_bytes = combine ? 4 * (size_t)N : to_f8 && streams ? (size_t)N : 0;
  const RouteLayout L = layout_routes(plan, T, top_k, num_experts, row_bytes);
  if (!workspace) {
    *workspace_bytes = L.total;
    return NVFP4_OK;
  }
  if (*workspace_bytes < L.total) return NVFP4_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return NVFP4_ERR_ALIGN;
  if ((st = check_act(act_kind, x, x_scales, ldx, K)) != NVFP4_OK) return st;
  if ((st = check_weight(w_codes, w_scales)) != NVFP4_OK) return st;
  if (!topk_ids || !y) return NVFP4_ERR_NULL;
  if (combine && !topk_w) return NVFP4_ERR_NULL;
  if (to_f8 != (y_scales != nullptr)) return y_scales ? NVFP4_ERR_ARG : NVFP4_ERR_NULL;
  if (!aligned(topk_ids, 4) || (topk_w && !aligned(topk_w, 4))) return NVFP4_ERR_ALIGN;
  if (!aligned(y, to_f8 ? 16 : (uintptr_t)type_bytes(y_type)) || !aligned(y_scales, 4)) return NVFP4_ERR_ALIGN;

  const int64_t R = T * top_k, active = R < num_experts ? R : num_experts;
  const int64_t xrows = rows_mode == NVFP4_ROWS_PER_TOKEN ? T : R;
  if (!fits(xrows, x_pitch(act_kind, ldx))) return NVFP4_ERR_SHAPE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if ((flags & NVFP4_F_CHECK) && check_data(act_kind, x, x_scales, ldx, xrows, N, K, num_experts, w_codes,
                                            w_scales, faults, s) != hipSuccess)
    return NVFP4_ERR_LAUNCH;
  void* const rows = static_cast<char*>(workspace) + L.rows;
  F8Args a{};
  a.x = x; a.x_scales = x_scales; a.ldx = ldx;
  a.w_codes = w_codes; a.w_scales = w_scales;
  a.N = N; a.K = K;
  a.R = R; a.x_rows = xrows; a.rows_per_token = rows_mode == NVFP4_ROWS_PER_TOKEN ? 1 : 0;
  a.top_k = top_k; a.num_experts = num_experts;
  a.y = row_bytes ? rows : y; a.y_scales = y_scales; a.ldy = N; a.y_type = combine ? FP8_F32 : y_type;
  a.swiglu = to_f8 && streams ? FP8_OUT_SWIGLU_BF16 : swiglu ? out_mode : 0;
  a.zero_dropped = !combine;
  hipError_t e = prepare_routes(a, plan, L, workspace, topk_ids, T, reuse, faults, s);
  const int kind = kernel_kind(act_kind, y_type == FP8_BF16 && !swiglu);
  if (e == hipSuccess)
    e = streams ? launch_f8_stream(a, kind, (R + active - 1) / active, s) : launch_f8_tiled(a, kind, s);
  if (e != hipSuccess) return NVFP4_ERR_LAUNCH;
  if (combine)
    e = launch_mx_combine(static_cast<float*>(rows), N, topk_ids, topk_w, T, top_k, num_experts, N, y_type, y, N, s);
  if (to_f8 && streams)
    e = launch_f8_quantize(FP8_BF16, rows, N / 2, R, N / 2, 1, FP8_SCALE_F32, static_cast<uint8_t*>(y),
                           y_scales, nullptr, s);
  return launch_status(e);
}

nvfp4_status moe_route(int32_t logits_type, const void* logits, int64_t ld, int64_t T,
                       int32_t num_experts, int32_t top_k, int32_t scoring, const float* bias,
                       int32_t num_groups, int32_t top_groups, int32_t group_score,
                       int32_t renormalize, float scale, int32_t* topk_ids, float* topk_w,
                       void* stream) {
  if (!is_type(logits_type)) return NVFP4_ERR_ARG;
  if (num_experts <= 0 || num_experts > kMaxExperts) return NVFP4_ERR_ARG;
  if (scoring != ROUTE_SOFTMAX && scoring != ROUTE_SIGMOID) return NVFP4_ERR_ARG;
  if (group_score != ROUTE_GROUP_MAX && group_score != ROUTE_GROUP_TOP2) return NVFP4_ERR_ARG;
  if (renormalize != 0 && renormalize != 1) return NVFP4_ERR_ARG;
  if (num_groups <= 0 || num_groups > num_experts || num_experts % num_groups != 0) return NVFP4_ERR_ARG;
  if (top_groups <= 0 || top_groups > num_groups) return NVFP4_ERR_ARG;
  if (top_k <= 0 || top_k > kMaxTopK || top_k > num_experts / num_groups * top_groups) return NVFP4_ERR_ARG;
  if (T <= 0 || T > kMaxRows || T * top_k > kMaxRows || ld < num_experts || ld > kMaxDim) return NVFP4_ERR_SHAPE;
  if (!logits || !topk_ids || !topk_w) return NVFP4_ERR_NULL;
  if (!aligned(logits, (uintptr_t)type_bytes(logits_type)) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) ||
      !aligned(bias, 4))
    return NVFP4_ERR_ALIGN;
  RouteArgs a{};
  a.logits = logits; a.bias = bias; a.ld = ld; a.T = T;
  a.logits_type = logits_type; a.num_experts = num_experts; a.top_k = top_k; a.scoring = scoring;
  a.num_groups = num_groups; a.top_groups = top_groups; a.group_score = group_score;
  a.renormalize = renormalize; a.scale = scale;
  a.topk_ids = topk_ids; a.topk_w = topk_w;
  return launch_status(launch_route(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
