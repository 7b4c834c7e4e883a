/* fp8.h — C ABI of the FP8 operators of libnvfp4.so with scales for blocks of 128, and of the
 * router, beside the NVFP4 calls of nvfp4.h and the MXFP4 ones of mxfp4.h.
 *
 * Codes are OCP E4M3FN bytes (bias 7, largest value 448, 0x7F/0xFF = NaN). Rows of activations
 * have one fp32 scale for 128 consecutive k, weights one for 128 rows x 128 k. An element is
 *     x(m, k) = e4m3(code[m][k]) * scale[m][k/128]         (activations)
 *     w(n, k) = e4m3(code[n][k]) * scale[n/128][k/128]     (weights).
 * The last block of a row, and of the rows, may be shorter.
 *
 * Layouts (row-major, caller-owned device memory):
 *   codes   [M][ld] or [N][K] uint8, K and ld multiples of 16, base 16-byte aligned;
 *   scales  [M][KB] or [NB][KB] fp32, KB = ceil(K/128), NB = ceil(N/128), contiguous, 4-byte
 *           aligned.
 * M, N and T * top_k may be any positive size up to 2^22, K likewise; there are at most 4096
 * experts, and top_k is at most 64 and at most their number. Offsets into the activations (of a
 * dense call: into 256 rows of them) and into one expert's codes are 32-bit: 2^31 bytes and
 * more are refused (NVFP4_ERR_SHAPE).
 *
 * Ownership, streams, argument errors, faults and determinism are as stated in nvfp4.h:
 * nothing is allocated or synchronized, bad arguments are refused on the host before
 * anything is enqueued, data faults are OR-ed into a device word, results are the same on
 * every run.
 */
#ifndef FP8_H
#define FP8_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* activation kinds */
enum { FP8_ACT_BF16 = 0, FP8_ACT_FP8 = 1 };
/* types of y, of the (de)quantizer's rows and of logits */
enum { FP8_BF16 = 0, FP8_F32 = 1 };
/* scale rules of the quantizer */
enum { FP8_SCALE_F32 = 0, FP8_SCALE_POW2 = 1 };
/* grouped call: what is written. The first three carry the values of NVFP4_OUT_*. */
enum {
  FP8_OUT_ROUTES = 0,
  FP8_OUT_SWIGLU_BF16 = 1,
  FP8_OUT_COMBINE = 2,
  FP8_OUT_SWIGLU_FP8 = 4
};

/* fp8_quantize — rows to FP8, bit-exactly by the rule, for each block b of block_rows x 128
 * (block_rows 1 for activations, 128 for weights), each step one correctly rounded fp32 operation:
 *     s_b    = amax_b / 448                     (FP8_SCALE_POW2: the least power of two not below that)
 *     code_k = E4M3_RNE(x_k / s_b)              (nearest, ties to the even code, saturating at 448;
 *                                               +-0 where s_b is 0; the sign is that of x)
 * A block holding a NaN or Inf gets a NaN scale and codes 0, and sets NVFP4_FAULT_NONFINITE in
 * *faults when faults is not NULL.
 * x_type FP8_BF16 or FP8_F32: x is [M][ldx], ldx >= K, rows 16-byte aligned.
 * codes [M][K], scales [ceil(M/block_rows)][KB].
 * Errors: NVFP4_ERR_NULL, _SHAPE, _ALIGN, _ARG, _LAUNCH. */
nvfp4_status fp8_quantize(int32_t x_type, const void* x, int64_t ldx, int64_t M, int64_t K,
                          int32_t block_rows, int32_t scale_rule, uint8_t* codes, float* scales,
                          uint32_t* faults, void* stream);

/* fp8_dequantize — codes [M][K] and scales [ceil(M/block_rows)][KB] to rows y [M][ldy] of y_type
 * (ldy >= K, rows 16-byte aligned): code times scale, rounded to fp32, and for BF16 once more.
 * Errors: NVFP4_ERR_NULL, _SHAPE, _ALIGN, _ARG, _LAUNCH. */
nvfp4_status fp8_dequantize(const uint8_t* codes, const float* scales, int64_t M, int64_t K,
                            int32_t block_rows, int32_t y_type, void* y, int64_t ldy, void* stream);

/* fp8_linear — y[m][n] = sum_k x(m, k) * w(n, k), written as y_type (FP8_F32, or FP8_BF16
 * rounded once to nearest even).
 *
 * W8A16 (act_kind FP8_ACT_BF16): x is BF16 [M][ldx] (ldx >= K, ldx % 8 == 0, base 16-byte
 *   aligned), x_scales NULL. The codes are decoded to BF16, which holds them exactly.
 * W8A8 (act_kind FP8_ACT_FP8): x is codes [M][ldx] (ldx >= K, ldx % 16 == 0, base 16-byte
 *   aligned) with x_scales [M][KB], as fp8_quantize writes them with block_rows 1.
 * Products are summed over at most 128 k, each such sum is multiplied by its scales (W8A8: by
 *   the fp32 product of both) and added in fp32. The sums of products are fp32 ones where x is
 *   BF16 or y is FP8_F32. W8A8 with y in BF16 takes the FP8 matrix instructions, which are twice
 *   as fast and, of eight products of consecutive k, drop what lies below 2^-13 of the largest, up
 *   to 7 * 2^-13 of that one. Measured, that is 1.4e-5 to 3e-5 of the results in the 2-norm (their
 *   rounding to BF16: 1.7e-3); a result whose large products cancel may lose more of itself than
 *   BF16 would, and asks for FP8_F32.
 *   Where the product of two scales, or that of a sum with it, leaves fp32's normal range, results
 *   are lost to zero or infinity.
 * Weight: w_codes [N][K] (16-byte aligned), w_scales [NB][KB]. y [M][ldy], ldy >= N, aligned
 *   to its type.
 * flags: 0 or NVFP4_F_CHECK: the operands are scanned first; a scale that is NaN or infinite
 *   sets NVFP4_FAULT_NAN_SCALE, a NaN code of either side or a non-finite BF16 activation
 *   NVFP4_FAULT_NONFINITE; the product still runs (a NaN gives NaN in the outputs it touches).
 *   faults: a device word, or NULL without NVFP4_F_CHECK.
 * Errors: NVFP4_ERR_NULL, _SHAPE, _ALIGN, _ARG, _LAUNCH. */
nvfp4_status fp8_linear(int32_t act_kind, const void* x, const float* x_scales, int64_t ldx,
                        int64_t M, int64_t N, int64_t K, const uint8_t* w_codes,
                        const float* w_scales, int32_t y_type, void* y, int64_t ldy,
                        uint32_t flags, uint32_t* faults, void* stream);

/* fp8_grouped_linear — the expert-grouped form, for groups of any sizes.
 *
 * w_codes [E][N][K], w_scales [E][NB][KB]; T tokens each pick top_k distinct experts,
 * topk_ids [T][top_k] int32 (moe_route writes them). Routes, rows_mode, the workspace (NULL: its
 * size is returned in *workspace_bytes), NVFP4_OUT_REUSE_GROUPING, bad routes
 * (NVFP4_FAULT_BAD_ROUTE, dropped) and flags are as in nvfp4_grouped_linear; act_kind, x,
 * x_scales and ldx as in fp8_linear. A reused workspace that does not hold this call's grouping
 * gives unspecified results, but no access outside the call's buffers, whatever it holds.
 * out_mode FP8_OUT_ROUTES: y is [T*top_k][N] of y_type, row r = x_row(r) w_e^T.
 *          FP8_OUT_SWIGLU_BF16: N/2 % 128 == 0 (gate and up share no block of scales); y is BF16
 *            [T*top_k][N/2], row r = bf16_rne(silu(g) * u) with g = h[0:N/2], u = h[N/2:N] of
 *            the route's fp32 row h; silu as in nvfp4_grouped_linear. y_type must be FP8_BF16.
 *          FP8_OUT_SWIGLU_FP8: the rows of FP8_OUT_SWIGLU_BF16, quantized by the rule of
 *            fp8_quantize (block_rows 1, FP8_SCALE_F32): codes [T*top_k][N/2] to y (16-byte
 *            aligned), scales [T*top_k][N/256] to y_scales; what a W8A8 down projection reads.
 *            A block that is not finite gets a NaN scale and codes 0. y_type is FP8_BF16.
 *          FP8_OUT_COMBINE: needs topk_w [T][top_k] fp32; y is [T][N] of y_type, y[t] =
 *            sum over t's routes in ascending expert id of topk_w[t][j] * (x_row(r) w_e^T),
 *            accumulated in fp32 in that order.
 * y_scales must be NULL in the other modes. topk_w is ignored unless combining. W8A8 sums as in
 * fp8_linear, by y_type; SwiGLU's are fp32 ones, because its results are quantized again.
 * Rows of dropped routes are zeros (FP8: codes 0 and scales 0).
 * The workspace of every out_mode begins with the grouping, so one that is large enough for
 * both serves a layer's gate_up and down calls.
 * Errors: NVFP4_ERR_NULL, _SHAPE, _ALIGN, _ARG, _WORKSPACE, _LAUNCH. */
nvfp4_status fp8_grouped_linear(int32_t act_kind, const void* x, const float* x_scales,
                                int64_t ldx, int32_t rows_mode, int64_t T, int32_t top_k,
                                int64_t N, int64_t K, int32_t num_experts,
                                const uint8_t* w_codes, const float* w_scales,
                                const int32_t* topk_ids, const float* topk_w, int32_t out_mode,
                                int32_t y_type, void* y, float* y_scales, void* workspace,
                                size_t* workspace_bytes, uint32_t flags, uint32_t* faults,
                                void* stream);

/* the router's scores, and how a group of experts is scored */
enum { ROUTE_SOFTMAX = 0, ROUTE_SIGMOID = 1 };
enum { ROUTE_GROUP_MAX = 0, ROUTE_GROUP_TOP2 = 1 };

/* moe_route — each token's experts and their weights, as the grouped calls of this library
 * (nvfp4_, mxfp4_ and fp8_grouped_linear) read them.
 *
 * For each row l of logits [T][ld] (logits_type FP8_BF16 or FP8_F32, E values, aligned to their
 * type):
 *     s_e = softmax(l)_e over all E experts, or 1 / (1 + exp(-l_e))
 *     c_e = s_e + bias_e                   (bias [E] fp32, or NULL: none)
 *   A logit of NaN or -infinity makes s_e 0 and adds nothing to softmax's sum; +infinity counts as
 *   the largest fp32 number. An expert is open when neither its logit nor its bias is NaN or
 *   -infinity; others are never picked.
 *   With num_groups > 1 the experts form num_groups equal groups of consecutive ones (their
 *   number divides num_experts); a group's score is the largest c of its open experts
 *   (ROUTE_GROUP_MAX) or the sum of the two largest (ROUTE_GROUP_TOP2: of the one there is, if
 *   so); the top_groups best groups keep their experts, and the others are not picked from.
 *   topk_ids[t] holds the top_k best experts by descending c, topk_w[t] their s (without the bias):
 *   divided by the sum of the picked ones' with renormalize (zeros if that is 0), then times
 *   `scale`.
 *   Of equals, experts or groups, the lower index comes first. Without a bias, and unless groups
 *   are scored by their two best, experts and groups are compared by the logits themselves, whose
 *   order is that of the scores. Otherwise they are compared by c in 64 bits, where scores that
 *   round to the same number are equals (sigmoids of logits above 37; softmax's that are 0).
 *   Where fewer than top_k experts are open to a token (a masked row), the rest of its ids are -1
 *   and their weights 0, which the grouped calls take as dropped routes.
 * 1 <= top_k <= 64, num_experts <= 4096, top_k at most the experts of top_groups groups.
 * topk_ids [T][top_k] int32 and topk_w [T][top_k] fp32, contiguous.
 * Errors: NVFP4_ERR_NULL, _SHAPE, _ALIGN, _ARG, _LAUNCH. */
nvfp4_status moe_route(int32_t logits_type, const void* logits, int64_t ld, int64_t T,
                       int32_t num_experts, int32_t top_k, int32_t scoring, const float* bias,
                       int32_t num_groups, int32_t top_groups, int32_t group_score,
                       int32_t renormalize, float scale, int32_t* topk_ids, float* topk_w,
                       void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8_H */
