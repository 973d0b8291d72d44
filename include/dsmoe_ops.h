/*
 * dsmoe_ops.h - operators around the expert layer of dsmoe.h, same library
 * (libdsmoe.so), one MI355X (gfx950):
 *   - layer norm (the norm in front of the layer), forward and backward, with
 *     the residual sum of a pre-norm block fused in;
 *   - matrix products grouped by expert over ragged row groups (the experts'
 *     own linear maps, for expert networks other than the layer's SwiGLU):
 *     forward, input gradient, weight gradient;
 *   - the orthogonalized update of expert weights (momentum, then
 *     Newton-Schulz products).
 *
 * The conventions of dsmoe.h hold: device pointers, caller-owned buffers, all
 * work on `stream`, arguments checked on the host before anything is
 * enqueued, moe_status and moe_last_error() for errors, no allocation and no
 * synchronization. In addition:
 *   - bf16 and fp32 matrices of these entry points need only the alignment of
 *     their element type, and rows may be strided (row strides in elements,
 *     columns contiguous). Offsets need 4 bytes; vectors, statistics, the
 *     matrices of moe_orthogonalize and workspaces 16.
 *   - Outputs must not overlap inputs unless said otherwise.
 */
#ifndef DSMOE_OPS_H
#define DSMOE_OPS_H

#include "dsmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Layer norm
 *
 * For each of n rows of d values, with v = x + residual (v = x without one):
 *   mean = sum_i v_i / d,  rstd = 1 / sqrt(sum_i (v_i - mean)^2 / d + eps),
 *   y_i = (v_i - mean) * rstd * weight_i + bias_i.
 * v, the statistics and y are computed in fp32 and rounded once on output.
 * The statistics are the fp32 v's, also where `sum` stores it in bf16.
 *   n        rows (>= 0; 0 writes no rows)
 *   d        row length, 1 .. 2^20
 *   dtype    MOE_DT_BF16 or MOE_DT_F32: all row matrices
 *   eps      >= 0, finite
 *   ld_x, ld_r, ld_y, ld_s   row strides, each 0 (contiguous) or >= d:
 *     forward:  x, residual, y, sum;  backward: x, dresidual, dy, dx */
typedef struct moe_norm_desc {
  int64_t n;
  int32_t d;
  int32_t dtype;
  float eps;
  int64_t ld_x;
  int64_t ld_r;
  int64_t ld_y;
  int64_t ld_s;
} moe_norm_desc;

/* x [n, d]; residual [n, d] or NULL; weight, bias [d] fp32 (either may be
 * NULL: 1 and 0). Out: y [n, d]; sum [n, d] = v (required with a residual,
 * else must be NULL); mean, rstd [n] fp32 (both or neither). y may be x or
 * residual (and sum the other one) where their strides agree. */
moe_status moe_layernorm_forward(const moe_norm_desc* desc, const void* x, const void* residual,
                                 const float* weight, const float* bias, void* y, void* sum,
                                 float* mean, float* rstd, hipStream_t stream);

/* Workspace of the backward. Host only. */
moe_status moe_layernorm_backward_workspace_size(const moe_norm_desc* desc, size_t* bytes);

/* Gradients for z = (x - mean) rstd, where x holds what was normalized (the
 * forward's x, or its `sum`), and g = dy * weight:
 *   dx = rstd (g - mean_i(g) - z mean_i(g z)) + dresidual,
 *   dweight = sum over rows of dy z,  dbias = sum over rows of dy.
 * In: dy, x [n, d]; weight [d] or NULL (1); mean, rstd [n] of the forward;
 * dresidual [n, d] or NULL: the gradient that reaches v past the norm.
 * Out: dx [n, d]; dweight, dbias [d] fp32 (either may be NULL). Sums run in
 * fp32 in a fixed order. dx may be dy or dresidual where their strides agree.
 * n == 0 writes zeros to dweight and dbias. ws: as sized above. */
moe_status moe_layernorm_backward(const moe_norm_desc* desc, const void* dy, const void* x,
                                  const float* weight, const float* mean, const float* rstd,
                                  const void* dresidual, void* dx, float* dweight, float* dbias,
                                  void* ws, size_t ws_bytes, hipStream_t stream);

/* ---- Matrix products grouped by expert
 *
 * Rows of x and dy come sorted by group, as moe_permute leaves them: group g
 * owns rows offsets[g] .. offsets[g+1] - 1 (offsets: n_groups + 1 int32 on
 * the device, ascending, within 0 .. rows). With W_g = w[g]:
 *   moe_grouped_gemm        y  = x W_g^T      x [rows, k]  -> y [rows, n]
 *   moe_grouped_gemm_dgrad  dx = dy W_g       dy [rows, n] -> dx [rows, k]
 *   moe_grouped_gemm_wgrad  dw[g] = dy_g^T x_g             -> dw [n_groups, n, k]
 * bf16 operands, fp32 accumulation, one rounding on output. Rows outside
 * offsets[0] .. offsets[n_groups] are not written; groups may be empty (their
 * dw is zero). Offsets out of range or order are clamped to a valid split
 * before use: the rows concerned hold other products, and nothing out of the
 * buffers is touched.
 *   rows       rows of x, y, dy and dx (>= 0)
 *   n_groups   1 .. 512
 *   n, k       output and input features of every group, >= 1;
 *              n * k * 4 < 2^31
 *   ld_k       row stride of x or dx, ld_n: of y or dy; 0 (contiguous) or
 *              >= k, >= n; below 2^21
 *   out_dtype  MOE_DT_BF16 or MOE_DT_F32: y or dx (dw is always fp32)
 *   accumulate wgrad only: nonzero adds to dw instead of overwriting it */
typedef struct moe_grouped_desc {
  int64_t rows;
  int32_t n_groups;
  int32_t n;
  int32_t k;
  int32_t out_dtype;
  int64_t ld_k;
  int64_t ld_n;
  int32_t accumulate;
} moe_grouped_desc;

enum { MOE_GROUPED_FORWARD = 0, MOE_GROUPED_DGRAD = 1, MOE_GROUPED_WGRAD = 2 };

/* Bytes of workspace for the product `op`: partial sums where the outputs (or
 * the last ones of a long contraction) are too few to occupy the GPU, 0
 * otherwise (ws may then be NULL). Host only. */
moe_status moe_grouped_gemm_workspace_size(const moe_grouped_desc* desc, int32_t op,
                                           size_t* bytes);

moe_status moe_grouped_gemm(const moe_grouped_desc* desc, const void* x, const void* w,
                            const int32_t* offsets, void* y, void* ws, size_t ws_bytes,
                            hipStream_t stream);
moe_status moe_grouped_gemm_dgrad(const moe_grouped_desc* desc, const void* dy, const void* w,
                                  const int32_t* offsets, void* dx, void* ws, size_t ws_bytes,
                                  hipStream_t stream);
moe_status moe_grouped_gemm_wgrad(const moe_grouped_desc* desc, const void* dy, const void* x,
                                  const int32_t* offsets, float* dw, void* ws, size_t ws_bytes,
                                  hipStream_t stream);

/* ---- Orthogonalized update of weight matrices
 *
 * For each of n_mats matrices [rows, cols], with momentum
 *   m_out = momentum * m_in + grad,
 *   u = grad + momentum * m_out (nesterov) or m_out,
 * and without (m_in == m_out == NULL) u = grad; then with X_0 = u / (|u|_F +
 * 1e-7) and `steps` times
 *   A = X X^T,  X <- a X + (b A + c A A) X,  (a, b, c) = (3.4445, -4.7750,
 *   2.0315)
 * (X^T in place of X where rows > cols), out = X: the singular vectors of u
 * with singular values near 1, the update direction of the Muon optimizer.
 * The products run on fp16 matrix cores with fp32 accumulation; the diagonals
 * of A and of the polynomial and the low part of X are kept apart. Off the exact
 * result before its rounding to bf16 (2-norm, five steps, as measured): 4e-4 for
 * 2048 x 7168, 1e-3 for 128 x 256, 1.4e-3 for 16 x 16, rank-deficient updates
 * included; with 1 to 8 rows of few values, where roundings do not average,
 * 1.5e-3 to 3.6e-3 and 9e-3 at worst. Three more steps leave 2e-3, 16 in all 3e-3
 * to 5e-3 from 64 x 64 on, up to 4.5e-3 and 1.6e-2 (on average) below. From nine
 * steps on a rank-deficient update is ill-conditioned: steps grow what
 * rounding left in its null space, the 24th bit of grad included, 3.44 times
 * each, up to 5e-2 off after ten and all of it after 14, as in fp32 throughout.
 * The norm is summed in fp64, so grad's scale does not matter beyond the 1e-7.
 *   n_mats       >= 0;  rows, cols 1 .. 16384
 *   grad_dtype   MOE_DT_F32 or MOE_DT_BF16
 *   steps        1 .. 16
 *   momentum     0 <= momentum < 1 (ignored without m_in)
 *   nesterov     0 or 1 */
typedef struct moe_orth_desc {
  int64_t n_mats;
  int32_t rows;
  int32_t cols;
  int32_t grad_dtype;
  int32_t steps;
  float momentum;
  int32_t nesterov;
} moe_orth_desc;

/* Bytes of workspace, 0 for matrices of up to 128 x 256 (ws may then be NULL).
 * Host only. */
moe_status moe_orthogonalize_workspace_size(const moe_orth_desc* desc, size_t* bytes);

/* grad [n_mats, rows, cols]; m_in, m_out fp32 of the same shape, both or
 * neither (m_out may be m_in); out bf16 of the same shape. All contiguous. */
moe_status moe_orthogonalize(const moe_orth_desc* desc, const void* grad, const float* m_in,
                             float* m_out, void* out, void* ws, size_t ws_bytes,
                             hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSMOE_OPS_H */
