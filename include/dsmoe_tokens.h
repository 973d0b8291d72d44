/*
 * dsmoe_tokens.h - operators on a token's way through an expert layer, in the
 * library of dsmoe.h (libdsmoe.so), one MI355X (gfx950):
 *   - RMS norm, forward (residual sum, rows and / or E4M3 tiles out) and
 *     backward;
 *   - tokens sorted by expert and returned with weights, and the gradients of
 *     both, for any selections: pairs without an expert here, any row type;
 *   - microscaled 4-bit values (OCP MX: E2M1, blocks of 32, E8M0 scales):
 *     quantization, dequantization, products grouped by expert.
 *
 * The conventions of dsmoe.h and dsmoe_ops.h hold: device pointers,
 * caller-owned buffers, all work on `stream`, arguments checked on the host
 * before anything is enqueued, moe_status and moe_last_error() for errors, no
 * allocation and no synchronization. Row matrices need the alignment of their
 * element type and may be strided (strides in elements, columns contiguous).
 * Index arrays need 4 bytes; vectors, statistics, 4-bit codes and their
 * scales, and workspaces 16. Outputs must not overlap inputs unless said
 * otherwise.
 */
#ifndef DSMOE_TOKENS_H
#define DSMOE_TOKENS_H

#include "dsmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- RMS norm
 *
 * For each of n rows of d values, with v = x + residual (v = x without one):
 *   rstd = 1 / sqrt(sum_i v_i^2 / d + eps),  o_i = v_i * rstd * weight_i.
 * v, rstd and o are fp32; each output is rounded once. rstd is that of the fp32
 * v, also where `sum` stores it in bf16. Two forms of o, either or both:
 *   y       rows in `dtype`
 *   codes   E4M3 codes of 1x128 tiles of a row (the last one shorter where 128
 *           does not divide d), scales fp32 [n, ceil(d / 128)]: amax = max|o|
 *           of the tile, scale = amax / 448, code = e4m3(o * (448 / amax)), to
 *           nearest even, the rule of moe_quantize_fp8_rows. amax below 2^-100:
 *           scale 1, zero codes. A NaN or infinity in a tile: codes 0x7F (NaN),
 *           scale amax / 448.
 *   n        rows (>= 0), below 2^31
 *   d        row length, 1 .. 2^20
 *   dtype    MOE_DT_BF16 or MOE_DT_F32: all row matrices but codes
 *   eps      >= 0, finite
 *   ld_x, ld_r, ld_y, ld_s, ld_q   row strides, each 0 (contiguous) or d ..
 *     2^31 - 1: forward: x, residual, y, sum, codes; backward: x, dresidual,
 *     dy, dx */
typedef struct moe_rmsnorm_desc {
  int64_t n;
  int32_t d;
  int32_t dtype;
  float eps;
  int64_t ld_x;
  int64_t ld_r;
  int64_t ld_y;
  int64_t ld_s;
  int64_t ld_q;
} moe_rmsnorm_desc;

/* x [n, d]; residual [n, d] or NULL; weight [d] fp32 or NULL (1). Out: y [n, d]
 * or NULL; codes [n, d] with scale, or both NULL (not all three); sum [n, d] = v
 * (required with a residual, else NULL); rstd [n] fp32 or NULL. y may be x or
 * residual (and sum the other one) where their strides agree. */
moe_status moe_rmsnorm_forward(const moe_rmsnorm_desc* desc, const void* x, const void* residual,
                               const float* weight, void* y, uint8_t* codes, float* scale,
                               void* sum, float* rstd, hipStream_t stream);

/* Workspace of the backward. Host only. */
moe_status moe_rmsnorm_backward_workspace_size(const moe_rmsnorm_desc* desc, size_t* bytes);

/* Gradients for z = x rstd, where x holds what was normalized (the forward's x,
 * or its `sum`), and g = dy * weight:
 *   dx = rstd (g - z mean_i(g z)) + dresidual,  dweight = sum over rows of dy z.
 * dy is the gradient in o (with codes: taken as if they had not been rounded).
 * In: dy, x [n, d]; weight [d] or NULL; rstd [n] of the forward; dresidual
 * [n, d] or NULL: the gradient that reaches v past the norm. Out: dx [n, d];
 * dweight [d] fp32 or NULL. Sums run in fp32 in a fixed order. dx may be dy or
 * dresidual where their strides agree. n == 0 writes zeros to dweight. ws: as
 * sized above (NULL without dweight). */
moe_status moe_rmsnorm_backward(const moe_rmsnorm_desc* desc, const void* dy, const void* x,
                                const float* weight, const float* rstd, const void* dresidual,
                                void* dx, float* dweight, void* ws, size_t ws_bytes,
                                hipStream_t stream);

/* ---- Tokens sorted by expert and back
 *
 * T tokens with K selections each. A pair (t, k) whose expert topk_idx[t, k] is
 * outside 0 .. n_experts - 1 (an expert of another rank, a masked token) has no
 * place. The others are sorted by expert, pairs of one expert in ascending t * K
 * + k, into `rows` places; where there are more pairs than places, the last ones
 * of this order have none. An expert may occur twice in a token.
 *   T          tokens (>= 0);  T * K < 2^31 - 2^20
 *   d          row length, >= 1;  d * 4 < 2^31
 *   n_experts  1 .. 512
 *   top_k      K, 1 .. 64
 *   dtype      MOE_DT_BF16, MOE_DT_F32 or (dispatch only) MOE_DT_FP8_E4M3: codes
 *              with fp32 scales of 1x128 tiles
 *   rows       places of the sorted matrices, 0 (T * K) or 1 .. T * K
 *   ld_t, ld_p row strides of token and of sorted matrices, 0 (contiguous) or
 *              d .. 2^31 - 1 */
typedef struct moe_dispatch_desc {
  int64_t T;
  int32_t d;
  int32_t n_experts;
  int32_t top_k;
  int32_t dtype;
  int64_t rows;
  int64_t ld_t;
  int64_t ld_p;
} moe_dispatch_desc;

/* Bytes of workspace of moe_token_dispatch (0 for few pairs; ws may then be
 * NULL). Host only. */
moe_status moe_token_dispatch_workspace_size(const moe_dispatch_desc* desc, size_t* bytes);

/* In: topk_idx [T, K] int32; x [T, d] or NULL (sort only); x_scale [T, ceil(d /
 * 128)] fp32 with E4M3 rows, else NULL.
 * Out: offsets [n_experts + 1] int32, expert e has places offsets[e] ..
 *   offsets[e + 1] - 1; perm [rows] int32, the token of each place, -1 behind
 *   the last; inv [T, K] int32, the place of each pair, -1 for none; x_perm
 *   [rows, d] = x[perm] and x_perm_scale [rows, ceil(d / 128)]: rows behind the
 *   last place are left as they were.
 * offsets, perm and x_perm are what moe_grouped_gemm, moe_expert_ffn and
 * moe_mx4_gemm read. ws: as sized above. */
moe_status moe_token_dispatch(const moe_dispatch_desc* desc, const int32_t* topk_idx,
                              const void* x, const float* x_scale, int32_t* offsets,
                              int32_t* perm, int32_t* inv, void* x_perm, float* x_perm_scale,
                              void* ws, size_t ws_bytes, hipStream_t stream);

/* y[t] = base[t] + sum_k weight[t, k] * y_perm[inv[t, k]], in fp32 in slot order,
 * rounded once; pairs with inv outside 0 .. rows - 1 are left out. y_perm [rows,
 * d]; inv [T, K]; weight [T, K] fp32 or NULL (1); base [T, d] or NULL (0). Out: y
 * [T, d] (may be base). A token without places gets base, or zeros.
 * With weight NULL this is the gradient of moe_token_dispatch in x. */
moe_status moe_token_combine(const moe_dispatch_desc* desc, const void* y_perm,
                             const int32_t* inv, const float* weight, const void* base, void* y,
                             hipStream_t stream);

/* Gradients of moe_token_combine: dy_perm[inv[t, k]] = weight[t, k] * dy[t] (rows
 * no pair has are left as they were) and dweight[t, k] = <dy[t], y_perm[inv[t,
 * k]]>, 0 for a pair without a place. dy [T, d]; y_perm [rows, d], NULL where
 * dweight is; inv, weight as above, no place twice. Out: dy_perm [rows, d] (may be
 * y_perm) or NULL; dweight [T, K] fp32 or NULL. The gradient in base is dy
 * itself. */
moe_status moe_token_combine_backward(const moe_dispatch_desc* desc, const void* dy,
                                      const void* y_perm, const int32_t* inv,
                                      const float* weight, void* dy_perm, float* dweight,
                                      hipStream_t stream);

/* ---- Microscaled 4-bit values (OCP MX, MXFP4)
 *
 * A row of k values is cut into blocks of 32 (the last one filled up with zeros);
 * a block has 32 E2M1 codes (sign, magnitudes 0 0.5 1 1.5 2 3 4 6) and one E8M0
 * byte b that stands for 2^(b - 127). With amax the block's largest magnitude
 *   e = floor(log2(amax)) - 2, at least -127;  b = e + 127;
 *   code = e2m1(v * 2^-e), to nearest even, magnitudes past 6 to 6.
 * amax == 0: b = 0 and codes of zeros with their signs. A NaN or infinity in a block:
 * b = 255 (NaN: every value of the block) and codes 0.
 * Layout of n_mats matrices of `rows` rows, KB = ceil(k / 32):
 *   codes   [n_mats, rows, KB * 16] bytes, value 2 i of a row in the low half of
 *           byte i
 *   scales  [n_mats, ceil(KB / 4), rows, 4] bytes: block 4 j + i of row r at
 *           [j, r, i], so that a step of the product reads the scales of adjacent
 *           rows as adjacent words; bytes past block KB - 1 are 0.
 *   n_mats   >= 0;  rows  >= 0;  n_mats * rows < 2^31
 *   k        1 .. 2^20
 *   dtype    MOE_DT_BF16 or MOE_DT_F32: the values' type
 *   act      quantize only: MOE_MX4_PLAIN or MOE_MX4_SWIGLU: rows of 2 k values
 *            hold gate | up, and what is quantized is silu(gate) * up in fp32
 *   ld       row stride of the values, 0 (contiguous) or a row's length ..
 *            2^31 - 1; matrices are rows * ld apart
 *   n_src    quantize with perm: rows of src */
enum { MOE_MX4_PLAIN = 0, MOE_MX4_SWIGLU = 1 };
typedef struct moe_mx4_desc {
  int64_t n_mats;
  int64_t rows;
  int32_t k;
  int32_t dtype;
  int32_t act;
  int64_t ld;
  int64_t n_src;
} moe_mx4_desc;

/* src [n_mats, rows, k] (gate | up: 2 k); perm NULL, or [rows] int32 with n_mats
 * == 1: row r is src[perm[r]], zeros for perm outside 0 .. n_src - 1 (the sorted
 * rows of moe_token_dispatch, quantized without writing them first); src may be NULL
 * with n_src == 0. */
moe_status moe_mx4_quantize(const moe_mx4_desc* desc, const void* src, const int32_t* perm,
                            uint8_t* codes, uint8_t* scales, hipStream_t stream);

/* dst [n_mats, rows, k]: the values of codes and scales, exact in bf16 and fp32
 * (infinity past their range: magnitudes of 2^128 and more). */
moe_status moe_mx4_dequantize(const moe_mx4_desc* desc, const uint8_t* codes,
                              const uint8_t* scales, void* dst, hipStream_t stream);

/* Products grouped by expert on 4-bit operands: with rows sorted by group as for
 * moe_grouped_gemm, y [rows, n] = x W_g^T for x [rows, k] (codes and scales of one
 * matrix) and W [n_groups, n, k] (of n_groups). Products of a block are exact,
 * sums fp32, one rounding on output. Rows outside offsets[0] ..
 * offsets[n_groups] are not written; offsets out of range or order are clamped
 * to a valid split.
 *   rows       rows of x and y (>= 0), below 2^28;  rows * ceil(k / 128) * 4 <
 *              2^31
 *   n_groups   1 .. 512
 *   n, k       1 .. 2^20;  n * ceil(k / 32) * 16 < 2^31
 *   out_dtype  MOE_DT_BF16 or MOE_DT_F32
 *   ld_y       row stride of y, 0 (contiguous) or n .. 2^31 - 1 */
typedef struct moe_mx4_gemm_desc {
  int64_t rows;
  int32_t n_groups;
  int32_t n;
  int32_t k;
  int32_t out_dtype;
  int64_t ld_y;
} moe_mx4_gemm_desc;

moe_status moe_mx4_gemm(const moe_mx4_gemm_desc* desc, const uint8_t* x_codes,
                        const uint8_t* x_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                        const int32_t* offsets, void* y, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSMOE_TOKENS_H */
