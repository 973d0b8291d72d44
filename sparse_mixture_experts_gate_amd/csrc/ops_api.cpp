// C entry points of dsmoe_ops.h: argument validation (host only, before any
// launch) and launches on the caller's stream. Nothing here allocates, frees
// or synchronizes.
#include <cmath>
#include <initializer_list>

#include <hip/hip_runtime.h>

#include "api_common.h"
#include "dsmoe_ops.h"
#include "internal.h"

using namespace dsmoe;

namespace {

struct Need {
  const void* p;
  const char* name;
  unsigned align;
  bool required;
};

moe_status check(std::initializer_list<Need> all) {
  for (const Need& n : all) {
    if (!n.p) {
      if (n.required) return fail(MOE_ERR_INVALID_ARGUMENT, "%s is NULL", n.name);
      continue;
    }
    if (reinterpret_cast<uintptr_t>(n.p) % n.align)
      return fail(MOE_ERR_MISALIGNED, "%s is not %u-byte aligned", n.name, n.align);
  }
  return MOE_OK;
}

int64_t pitch(int64_t ld, int64_t width) { return ld ? ld : width; }

// ---- layer norm ------------------------------------------------------------------

moe_status validate(const moe_norm_desc* d) {
  if (!d) return fail(MOE_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->n < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "n = %lld < 0", (long long)d->n);
  if (d->n >= (int64_t(1) << 31))
    return fail(MOE_ERR_UNSUPPORTED, "n = %lld: below 2^31 rows", (long long)d->n);
  if (d->d < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "d = %d < 1", d->d);
  if (d->d > (1 << 20)) return fail(MOE_ERR_UNSUPPORTED, "d = %d > 2^20", d->d);
  if (d->dtype != MOE_DT_BF16 && d->dtype != MOE_DT_F32)
    return fail(MOE_ERR_UNSUPPORTED, "dtype = %d: rows are bf16 or fp32", d->dtype);
  if (!(d->eps >= 0.0f) || !std::isfinite(d->eps))
    return fail(MOE_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  const std::pair<int64_t, const char*> lds[] = {
      {d->ld_x, "ld_x"}, {d->ld_r, "ld_r"}, {d->ld_y, "ld_y"}, {d->ld_s, "ld_s"}};
  for (auto& l : lds)
    if (l.first && (l.first < d->d || l.first >= (int64_t(1) << 31)))
      return fail(MOE_ERR_INVALID_ARGUMENT, "%s = %lld: 0, or d = %d .. 2^31 - 1", l.second,
                  (long long)l.first, d->d);
  return MOE_OK;
}

NormArgs norm_args(const moe_norm_desc* d) {
  NormArgs a{};
  a.n = d->n;
  a.d = d->d;
  a.bf16 = d->dtype == MOE_DT_BF16;
  a.eps = d->eps;
  a.ldx = pitch(d->ld_x, d->d);
  a.ldr = pitch(d->ld_r, d->d);
  a.ldy = pitch(d->ld_y, d->d);
  a.lds = pitch(d->ld_s, d->d);
  return a;
}

size_t norm_ws(const moe_norm_desc* d) {
  return d->n == 0 ? 0 : sizeof(float) * 2 * size_t(d->d) * norm_backward_parts(d->n, d->d);
}

// ---- grouped products ---------------------------------------------------------------

moe_status validate(const moe_grouped_desc* d, bool wgrad) {
  if (!d) return fail(MOE_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->rows < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "rows = %lld < 0", (long long)d->rows);
  if (d->n_groups < 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n_groups = %d < 1", d->n_groups);
  if (d->n_groups > 512) return fail(MOE_ERR_UNSUPPORTED, "n_groups = %d > 512", d->n_groups);
  if (d->n < 1 || d->k < 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n = %d, k = %d: both >= 1", d->n, d->k);
  if (int64_t(d->n) * d->k * 4 >= (int64_t(1) << 31))
    return fail(MOE_ERR_UNSUPPORTED, "n * k * 4 must be < 2^31 bytes");
  const int64_t lk = pitch(d->ld_k, d->k), ln = pitch(d->ld_n, d->n);
  if (lk < d->k || ln < d->n)
    return fail(MOE_ERR_INVALID_ARGUMENT, "ld_k = %lld, ld_n = %lld: 0, or at least k, n",
                (long long)d->ld_k, (long long)d->ld_n);
  // the kernels address the 256 rows of a tile with 32-bit byte offsets
  if (lk >= (int64_t(1) << 21) || ln >= (int64_t(1) << 21))
    return fail(MOE_ERR_UNSUPPORTED, "row strides must be < 2^21 elements");
  // rows and tiles (of at least 64 x 64 outputs) are counted in 32 bits
  if (d->rows >= (int64_t(1) << 31) - 256)
    return fail(MOE_ERR_UNSUPPORTED, "rows = %lld: below 2^31 - 256", (long long)d->rows);
  const int64_t wide = d->n > d->k ? d->n : d->k;
  if ((d->rows / 32 + d->n_groups) * (wide / 64 + 1) >= (int64_t(1) << 30) ||
      int64_t(d->n_groups) * (d->n / 64 + 1) * (d->k / 64 + 1) >= (int64_t(1) << 30))
    return fail(MOE_ERR_UNSUPPORTED, "rows * max(n, k): below 2^41 outputs a call");
  if (!wgrad && d->out_dtype != MOE_DT_BF16 && d->out_dtype != MOE_DT_F32)
    return fail(MOE_ERR_UNSUPPORTED, "out_dtype = %d: bf16 or fp32", d->out_dtype);
  return MOE_OK;
}

GroupedArgs grouped_args(const moe_grouped_desc* d, int mode, const void* a, const void* b,
                         const int32_t* offsets, void* out) {
  GroupedArgs g{};
  g.mode = mode;
  g.a = a;
  g.b = b;
  g.offsets = offsets;
  g.out = out;
  g.rows = d->rows;
  g.ld_k = pitch(d->ld_k, d->k);
  g.ld_n = pitch(d->ld_n, d->n);
  g.n_groups = d->n_groups;
  g.n = d->n;
  g.k = d->k;
  g.out_f32 = mode == 2 || d->out_dtype == MOE_DT_F32;
  g.accumulate = mode == 2 && d->accumulate;
  return g;
}

moe_status check_ws(const GroupedArgs& g, const void* ws, size_t ws_bytes) {
  const size_t need = grouped_workspace(g);
  if (!need) return MOE_OK;
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "this product needs %zu workspace bytes, got %zu", need,
                ws_bytes);
  return check({{ws, "ws", 16, true}});
}

// ---- orthogonalized updates ------------------------------------------------------------

moe_status validate(const moe_orth_desc* d) {
  if (!d) return fail(MOE_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->n_mats < 0)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n_mats = %lld < 0", (long long)d->n_mats);
  if (d->n_mats > 65535)
    return fail(MOE_ERR_UNSUPPORTED, "n_mats = %lld > 65535", (long long)d->n_mats);
  if (d->rows < 1 || d->cols < 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "rows = %d, cols = %d: both >= 1", d->rows, d->cols);
  if (d->rows > 16384 || d->cols > 16384)
    return fail(MOE_ERR_UNSUPPORTED, "rows = %d, cols = %d: up to 16384", d->rows, d->cols);
  if (d->n_mats * ((d->rows + 63) / 64) * ((d->cols + 63) / 64) >= (int64_t(1) << 31))
    return fail(MOE_ERR_UNSUPPORTED, "n_mats * rows * cols: below 2^43 elements");
  if (d->grad_dtype != MOE_DT_F32 && d->grad_dtype != MOE_DT_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "grad_dtype = %d: bf16 or fp32", d->grad_dtype);
  if (d->steps < 1 || d->steps > 16)
    return fail(MOE_ERR_INVALID_ARGUMENT, "steps = %d outside 1..16", d->steps);
  if (!(d->momentum >= 0.0f && d->momentum < 1.0f))
    return fail(MOE_ERR_INVALID_ARGUMENT, "momentum must be in [0, 1)");
  if (d->nesterov != 0 && d->nesterov != 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "nesterov = %d: 0 or 1", d->nesterov);
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_layernorm_forward(const moe_norm_desc* desc, const void* x, const void* residual,
                                 const float* weight, const float* bias, void* y, void* sum,
                                 float* mean, float* rstd, hipStream_t stream) {
  moe_status st = validate(desc);
  if (st) return st;
  if (desc->n == 0) return MOE_OK;
  const unsigned el = desc->dtype == MOE_DT_BF16 ? 2 : 4;
  st = check({{x, "x", el, true}, {residual, "residual", el, false}, {weight, "weight", 16, false},
              {bias, "bias", 16, false}, {y, "y", el, true}, {sum, "sum", el, false},
              {mean, "mean", 16, false}, {rstd, "rstd", 16, false}});
  if (st) return st;
  if (!residual != !sum)
    return fail(MOE_ERR_INVALID_ARGUMENT, "residual and sum: both or neither");
  if (!mean != !rstd) return fail(MOE_ERR_INVALID_ARGUMENT, "mean and rstd: both or neither");
  NormArgs a = norm_args(desc);
  a.x = x;
  a.r = residual;
  a.w = weight;
  a.b = bias;
  a.y = y;
  a.s = sum;
  a.mean = mean;
  a.rstd = rstd;
  HIP_TRY(launch_norm_forward(a, stream), "layer norm");
  return MOE_OK;
}

moe_status moe_layernorm_backward_workspace_size(const moe_norm_desc* desc, size_t* bytes) {
  moe_status st = validate(desc);
  if (st) return st;
  if (!bytes) return fail(MOE_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = norm_ws(desc);
  return MOE_OK;
}

moe_status moe_layernorm_backward(const moe_norm_desc* desc, const void* dy, const void* x,
                                  const float* weight, const float* mean, const float* rstd,
                                  const void* dresidual, void* dx, float* dweight, float* dbias,
                                  void* ws, size_t ws_bytes, hipStream_t stream) {
  moe_status st = validate(desc);
  if (st) return st;
  const unsigned el = desc->dtype == MOE_DT_BF16 ? 2 : 4;
  const bool rows = desc->n > 0, sums = dweight || dbias;
  st = check({{dy, "dy", el, rows}, {x, "x", el, rows}, {weight, "weight", 16, false},
              {mean, "mean", 16, rows}, {rstd, "rstd", 16, rows},
              {dresidual, "dresidual", el, false}, {dx, "dx", el, rows},
              {dweight, "dweight", 16, false}, {dbias, "dbias", 16, false},
              {ws, "ws", 16, rows && sums}});
  if (st) return st;
  if (sums && ws_bytes < norm_ws(desc))
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL,
                "moe_layernorm_backward needs %zu workspace bytes, got %zu", norm_ws(desc), ws_bytes);
  NormArgs a = norm_args(desc);
  a.x = x;
  a.r = dresidual;
  a.w = weight;
  a.y = const_cast<void*>(dy);
  a.s = dx;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  HIP_TRY(launch_norm_backward(a, dweight, dbias, static_cast<float*>(ws), stream),
          "layer norm backward");
  return MOE_OK;
}

moe_status moe_grouped_gemm_workspace_size(const moe_grouped_desc* desc, int32_t op,
                                           size_t* bytes) {
  if (op < 0 || op > 2) return fail(MOE_ERR_INVALID_ARGUMENT, "op = %d: 0, 1 or 2", op);
  moe_status st = validate(desc, op == MOE_GROUPED_WGRAD);
  if (st) return st;
  if (!bytes) return fail(MOE_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = grouped_workspace(grouped_args(desc, op, nullptr, nullptr, nullptr, nullptr));
  return MOE_OK;
}

moe_status moe_grouped_gemm(const moe_grouped_desc* desc, const void* x, const void* w,
                            const int32_t* offsets, void* y, void* ws, size_t ws_bytes,
                            hipStream_t stream) {
  moe_status st = validate(desc, false);
  if (st) return st;
  if (desc->rows == 0) return MOE_OK;
  st = check({{x, "x", 2, true}, {w, "w", 2, true}, {offsets, "offsets", 4, true},
              {y, "y", desc->out_dtype == MOE_DT_F32 ? 4u : 2u, true}});
  if (st) return st;
  const GroupedArgs g = grouped_args(desc, MOE_GROUPED_FORWARD, x, w, offsets, y);
  st = check_ws(g, ws, ws_bytes);
  if (st) return st;
  HIP_TRY(launch_grouped(g, ws, stream), "grouped product");
  return MOE_OK;
}

moe_status moe_grouped_gemm_dgrad(const moe_grouped_desc* desc, const void* dy, const void* w,
                                  const int32_t* offsets, void* dx, void* ws, size_t ws_bytes,
                                  hipStream_t stream) {
  moe_status st = validate(desc, false);
  if (st) return st;
  if (desc->rows == 0) return MOE_OK;
  st = check({{dy, "dy", 2, true}, {w, "w", 2, true}, {offsets, "offsets", 4, true},
              {dx, "dx", desc->out_dtype == MOE_DT_F32 ? 4u : 2u, true}});
  if (st) return st;
  const GroupedArgs g = grouped_args(desc, MOE_GROUPED_DGRAD, dy, w, offsets, dx);
  st = check_ws(g, ws, ws_bytes);
  if (st) return st;
  HIP_TRY(launch_grouped(g, ws, stream), "grouped input gradient");
  return MOE_OK;
}

moe_status moe_grouped_gemm_wgrad(const moe_grouped_desc* desc, const void* dy, const void* x,
                                  const int32_t* offsets, float* dw, void* ws, size_t ws_bytes,
                                  hipStream_t stream) {
  moe_status st = validate(desc, true);
  if (st) return st;
  const bool rows = desc->rows > 0;
  st = check({{dy, "dy", 2, rows}, {x, "x", 2, rows}, {offsets, "offsets", 4, true},
              {dw, "dw", 4, true}});
  if (st) return st;
  const GroupedArgs g = grouped_args(desc, MOE_GROUPED_WGRAD, dy, x, offsets, dw);
  st = check_ws(g, ws, ws_bytes);
  if (st) return st;
  HIP_TRY(launch_grouped(g, ws, stream), "grouped weight gradient");
  return MOE_OK;
}

moe_status moe_orthogonalize_workspace_size(const moe_orth_desc* desc, size_t* bytes) {
  moe_status st = validate(desc);
  if (st) return st;
  if (!bytes) return fail(MOE_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = orth_workspace(desc->n_mats, desc->rows, desc->cols);
  return MOE_OK;
}

moe_status moe_orthogonalize(const moe_orth_desc* desc, const void* grad, const float* m_in,
                             float* m_out, void* out, void* ws, size_t ws_bytes,
                             hipStream_t stream) {
  moe_status st = validate(desc);
  if (st) return st;
  if (desc->n_mats == 0) return MOE_OK;
  st = check({{grad, "grad", 16, true}, {m_in, "m_in", 16, false}, {m_out, "m_out", 16, false},
              {out, "out", 16, true}});
  if (st) return st;
  if (!m_in != !m_out) return fail(MOE_ERR_INVALID_ARGUMENT, "m_in and m_out: both or neither");
  const size_t need = orth_workspace(desc->n_mats, desc->rows, desc->cols);
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "moe_orthogonalize needs %zu workspace bytes, got %zu",
                need, ws_bytes);
  st = check({{ws, "ws", 16, need > 0}});
  if (st) return st;
  OrthArgs a{};
  a.mats = desc->n_mats;
  a.rows = desc->rows;
  a.cols = desc->cols;
  a.steps = desc->steps;
  a.bf16 = desc->grad_dtype == MOE_DT_BF16;
  a.nesterov = desc->nesterov;
  a.momentum = desc->momentum;
  a.grad = grad;
  a.m_in = m_in;
  a.m_out = m_out;
  a.out = out;
  a.ws = ws;
  HIP_TRY(launch_orth(a, stream), "orthogonalized update");
  return MOE_OK;
}

}  // extern "C"
