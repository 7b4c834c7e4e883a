/* mxfp4.h — C ABI of the MXFP4 operators of libnvfp4, beside the NVFP4 ones of nvfp4.h.
 *
 * MXFP4 is the OCP Microscaling format with 4-bit elements: E2M1 codes (as in nvfp4.h: bit
 * 3 = sign, bits 0..2 index {0, 0.5, 1, 1.5, 2, 3, 4, 6}) and one E8M0 scale per 32
 * consecutive elements along K, a byte s standing for 2^(s - 127), 0xFF for NaN. Element
 * (n, k) of a weight has the value
 *     e2m1(code[n][k]) * 2^(scale[n][k/32] - 127).
 * There is no tensor scale. The matrix cores of gfx950 multiply this format as it is.
 *
 * Layouts (row-major, caller-owned device memory):
 *   codes   [N][K/2]  uint8, byte j of a row holds k = 2j in its low nibble and
 *                      k = 2j+1 in its high nibble; rows contiguous, base 16-byte aligned;
 *   scales  [N][K/32] uint8, any alignment.
 * K % 32 == 0; M, N and T * top_k may be any positive size up to 2^22, K likewise; there are at
 * most 4096 experts, and top_k is at most 64 and at most their number. Offsets into
 * the activations (of a dense call: into 256 rows of them) and into one expert's codes are
 * 32-bit: 2^31 bytes and more are refused (NVFP4_ERR_SHAPE).
 *
 * Ownership, streams, argument errors, faults and determinism are as stated in nvfp4.h:
 * nothing is allocated or synchronized, bad arguments are refused on the host before
 * anything is enqueued, data faults are OR-ed into a device word, results are the same on
 * every run.
 */
#ifndef MXFP4_H
#define MXFP4_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* activation kinds */
enum { MXFP4_ACT_BF16 = 0, MXFP4_ACT_MXFP4 = 1 };
/* types of y, and of the (de)quantizer's rows */
enum { MXFP4_BF16 = 0, MXFP4_F32 = 1 };
/* grouped call: what is written. The first three carry the values of NVFP4_OUT_*. */
enum {
  MXFP4_OUT_ROUTES = 0,
  MXFP4_OUT_SWIGLU_BF16 = 1,
  MXFP4_OUT_COMBINE = 2,
  MXFP4_OUT_SWIGLU_MXFP4 = 3
};

/* mxfp4_quantize — rows to MXFP4, bit-exactly by the rule, for each block b of 32:
 *     e_b    = floor(log2(amax_b)) - 2      (2: the exponent of E2M1's largest value, 6)
 *     s_b    = clamp(e_b + 127, 0, 254)     (0 for a block of zeros)
 *     code_k = E2M1_RNE(x_k / 2^(s_b - 127)) (nearest, ties to the even code, saturating at
 *                                            6; the sign is the sign bit of x, so -0 -> 0x8)
 * (the scale rule of the OCP Microscaling specification; division by a power of two is exact
 * or rounds below E2M1's smallest decision point, so no step before the last one matters).
 * A block holding a NaN or Inf gets the scale 0xFF (NaN) and codes 0, and sets
 * NVFP4_FAULT_NONFINITE in *faults when faults is not NULL.
 * x_type MXFP4_BF16 or MXFP4_F32: x is [M][ldx], ldx >= K, rows 16-byte aligned.
 * codes [M][K/2], scales [M][K/32].
 * Errors: NVFP4_ERR_NULL, _SHAPE, _ALIGN, _ARG, _LAUNCH. */
nvfp4_status mxfp4_quantize(int32_t x_type, const void* x, int64_t ldx, int64_t M, int64_t K,
                            uint8_t* codes, uint8_t* scales, uint32_t* faults, void* stream);

/* mxfp4_dequantize — codes [M][K/2] and scales [M][K/32] to rows y [M][ldy] of y_type
 * (ldy >= K, rows 16-byte aligned): the value each code stands for, rounded once to y_type
 * where that cannot hold it (magnitudes of 2^128 and more become infinite; every other
 * value is exact in both types). The scale 0xFF gives NaN.
 * Errors: NVFP4_ERR_NULL, _SHAPE, _ALIGN, _ARG, _LAUNCH. */
nvfp4_status mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K,
                              int32_t y_type, void* y, int64_t ldy, void* stream);

/* mxfp4_linear — y[m][n] = sum_k x[m][k] * w(n, k), accumulated in fp32, written as y_type
 * (MXFP4_F32, or MXFP4_BF16 rounded once to nearest even).
 *
 * W4A16 (act_kind MXFP4_ACT_BF16): x is BF16 [M][ldx] (ldx >= K, ldx % 8 == 0, base 16-byte
 *   aligned), x_scales NULL. The weight is decoded to BF16, which holds every value below
 *   2^128 exactly.
 * W4A4 (act_kind MXFP4_ACT_MXFP4): x is codes [M][K/2] (16-byte aligned) with x_scales
 *   [M][K/32], as mxfp4_quantize writes them; ldx is ignored. Products of codes are exact.
 * Weight: w_codes [N][K/2] (16-byte aligned), w_scales [N][K/32]. y [M][ldy], ldy >= N,
 *   aligned to its type.
 * flags: 0 or NVFP4_F_CHECK: the operands are scanned first, and a NaN scale byte sets
 *   NVFP4_FAULT_NAN_SCALE, a non-finite BF16 activation NVFP4_FAULT_NONFINITE; the product
 *   still runs (a NaN scale gives NaN in the outputs it touches). faults: a device word, or
 *   NULL without NVFP4_F_CHECK.
 * Errors: NVFP4_ERR_NULL, _SHAPE, _ALIGN, _ARG, _LAUNCH. */
nvfp4_status mxfp4_linear(int32_t act_kind, const void* x, const uint8_t* x_scales, int64_t ldx,
                          int64_t M, int64_t N, int64_t K, const uint8_t* w_codes,
                          const uint8_t* w_scales, int32_t y_type, void* y, int64_t ldy,
                          uint32_t flags, uint32_t* faults, void* stream);

/* mxfp4_grouped_linear — the expert-grouped form, for groups of any sizes.
 *
 * w_codes [E][N][K/2], w_scales [E][N][K/32]; T tokens each pick top_k distinct experts,
 * topk_ids [T][top_k] int32. Routes, rows_mode, the workspace (NULL: its size is returned in
 * *workspace_bytes), NVFP4_OUT_REUSE_GROUPING, bad routes (NVFP4_FAULT_BAD_ROUTE, dropped)
 * and flags are as in nvfp4_grouped_linear; act_kind, x, x_scales and ldx as in mxfp4_linear.
 * A reused workspace that does not hold this call's grouping gives unspecified results, but no
 * access outside the call's buffers, whatever it holds.
 * out_mode MXFP4_OUT_ROUTES: y is [T*top_k][N] of y_type, row r = x_row(r) w_e^T.
 *          MXFP4_OUT_SWIGLU_BF16: N even; y is BF16 [T*top_k][N/2], row r =
 *            bf16_rne(silu(g) * u) with g = h[0:N/2], u = h[N/2:N] of the route's fp32 row
 *            h; silu as in nvfp4_grouped_linear. y_type must be MXFP4_BF16.
 *          MXFP4_OUT_SWIGLU_MXFP4: N/2 % 32 == 0; the rows of MXFP4_OUT_SWIGLU_BF16,
 *            quantized by the rule of mxfp4_quantize: codes [T*top_k][N/4] to y (16-byte
 *            aligned), scales [T*top_k][N/64] to y_scales; what a W4A4 down projection
 *            reads. A block that is not finite gets the scale 0xFF. y_type is MXFP4_BF16.
 *          MXFP4_OUT_COMBINE: needs topk_w [T][top_k] fp32; y is [T][N] of y_type, y[t] =
 *            sum over t's routes in ascending expert id of topk_w[t][j] * (x_row(r) w_e^T),
 *            accumulated in fp32 in that order.
 * y_scales must be NULL in the other modes. topk_w is ignored unless combining.
 * Rows of dropped routes are zeros (MXFP4: codes 0 and scales 0).
 * The workspace of every out_mode begins with the grouping, so one that is large enough for
 * both serves a layer's gate_up and down calls.
 * Errors: NVFP4_ERR_NULL, _SHAPE, _ALIGN, _ARG, _WORKSPACE, _LAUNCH. */
nvfp4_status mxfp4_grouped_linear(int32_t act_kind, const void* x, const uint8_t* x_scales,
                                  int64_t ldx, int32_t rows_mode, int64_t T, int32_t top_k,
                                  int64_t N, int64_t K, int32_t num_experts,
                                  const uint8_t* w_codes, const uint8_t* w_scales,
                                  const int32_t* topk_ids, const float* topk_w,
                                  int32_t out_mode, int32_t y_type, void* y, uint8_t* y_scales,
                                  void* workspace, size_t* workspace_bytes, uint32_t flags,
                                  uint32_t* faults, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
