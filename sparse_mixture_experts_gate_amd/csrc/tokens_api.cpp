// C entry points of dsmoe_tokens.h: argument validation (host only, before any
// launch) and launches on the caller's stream. Nothing here allocates, frees
// or synchronizes.
#include <cmath>
#include <initializer_list>

#include <hip/hip_runtime.h>

#include "api_common.h"
#include "dsmoe_tokens.h"
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

constexpr int64_t kInt31 = int64_t(1) << 31;

int64_t pitch(int64_t ld, int64_t width) { return ld ? ld : width; }

moe_status check_ld(int64_t ld, int64_t width, const char* name) {
  if (ld && (ld < width || ld >= kInt31))
    return fail(MOE_ERR_INVALID_ARGUMENT, "%s = %lld: 0, or %lld .. 2^31 - 1", name, (long long)ld,
                (long long)width);
  return MOE_OK;
}

unsigned size_of(int32_t dtype) {
  return dtype == MOE_DT_F32 ? 4 : dtype == MOE_DT_BF16 ? 2 : 1;
}

// ---- RMS norm ---------------------------------------------------------------------

moe_status validate(const moe_rmsnorm_desc* d) {
  if (!d) return fail(MOE_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->n < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "n = %lld < 0", (long long)d->n);
  if (d->n >= kInt31)
    return fail(MOE_ERR_UNSUPPORTED, "n = %lld: below 2^31 rows", (long long)d->n);
  if (d->d < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "d = %d < 1", d->d);
  if (d->d > (1 << 20)) return fail(MOE_ERR_UNSUPPORTED, "d = %d > 2^20", d->d);
  if (d->dtype != MOE_DT_BF16 && d->dtype != MOE_DT_F32)
    return fail(MOE_ERR_UNSUPPORTED, "dtype = %d: rows are bf16 or fp32", d->dtype);
  if (!(d->eps >= 0.0f) || !std::isfinite(d->eps))
    return fail(MOE_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  const std::pair<int64_t, const char*> lds[] = {{d->ld_x, "ld_x"},
                                                 {d->ld_r, "ld_r"},
                                                 {d->ld_y, "ld_y"},
                                                 {d->ld_s, "ld_s"},
                                                 {d->ld_q, "ld_q"}};
  for (auto& l : lds)
    if (moe_status st = check_ld(l.first, d->d, l.second)) return st;
  return MOE_OK;
}

RmsArgs rms_args(const moe_rmsnorm_desc* d) {
  RmsArgs a{};
  a.n = d->n;
  a.d = d->d;
  a.bf16 = d->dtype == MOE_DT_BF16;
  a.eps = d->eps;
  a.ldx = pitch(d->ld_x, d->d);
  a.ldr = pitch(d->ld_r, d->d);
  a.ldy = pitch(d->ld_y, d->d);
  a.lds = pitch(d->ld_s, d->d);
  a.ldq = pitch(d->ld_q, d->d);
  return a;
}

size_t rms_ws(const moe_rmsnorm_desc* d) {
  return d->n == 0 ? 0 : sizeof(float) * size_t(d->d) * rmsnorm_backward_parts(d->n, d->d);
}

// ---- dispatch and return -------------------------------------------------------------

moe_status validate(const moe_dispatch_desc* d, bool fp8) {
  if (!d) return fail(MOE_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->T < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "T = %lld < 0", (long long)d->T);
  if (d->d < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "d = %d < 1", d->d);
  if (int64_t(d->d) * 4 >= kInt31) return fail(MOE_ERR_UNSUPPORTED, "d * 4 must be < 2^31");
  if (d->n_experts < 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n_experts = %d < 1", d->n_experts);
  if (d->n_experts > 512) return fail(MOE_ERR_UNSUPPORTED, "n_experts = %d > 512", d->n_experts);
  if (d->top_k < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "top_k = %d < 1", d->top_k);
  if (d->top_k > 64) return fail(MOE_ERR_UNSUPPORTED, "top_k = %d > 64", d->top_k);
  if (d->T >= (kInt31 - (1 << 20)) / d->top_k)
    return fail(MOE_ERR_UNSUPPORTED, "T * top_k must be < 2^31 - 2^20");
  if (d->dtype != MOE_DT_BF16 && d->dtype != MOE_DT_F32 && !(fp8 && d->dtype == MOE_DT_FP8_E4M3))
    return fail(MOE_ERR_UNSUPPORTED, "dtype = %d: rows are bf16 or fp32%s", d->dtype,
                fp8 ? " or E4M3" : "");
  if (d->rows < 0 || d->rows > d->T * d->top_k)
    return fail(MOE_ERR_INVALID_ARGUMENT, "rows = %lld: 0 .. T * top_k = %lld", (long long)d->rows,
                (long long)(d->T * d->top_k));
  if (moe_status st = check_ld(d->ld_t, d->d, "ld_t")) return st;
  return check_ld(d->ld_p, d->d, "ld_p");
}

int64_t rows_of(const moe_dispatch_desc* d) { return d->rows ? d->rows : d->T * d->top_k; }

CombineArgs combine_args(const moe_dispatch_desc* d) {
  CombineArgs a{};
  a.T = d->T;
  a.rows = rows_of(d);
  a.K = d->top_k;
  a.d = d->d;
  a.bf16 = d->dtype == MOE_DT_BF16;
  a.ldt = pitch(d->ld_t, d->d);
  a.ldp = pitch(d->ld_p, d->d);
  return a;
}

// ---- microscaled 4-bit values ----------------------------------------------------------

moe_status validate(const moe_mx4_desc* d, bool quantize) {
  if (!d) return fail(MOE_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->n_mats < 0 || d->rows < 0)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n_mats = %lld, rows = %lld: both >= 0",
                (long long)d->n_mats, (long long)d->rows);
  if (d->k < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "k = %d < 1", d->k);
  if (d->k > (1 << 20)) return fail(MOE_ERR_UNSUPPORTED, "k = %d > 2^20", d->k);
  if (d->n_mats >= kInt31 || d->rows >= kInt31 ||
      (d->rows > 0 && d->n_mats >= (kInt31 + d->rows - 1) / d->rows))
    return fail(MOE_ERR_UNSUPPORTED, "n_mats * rows must be < 2^31");
  if (d->dtype != MOE_DT_BF16 && d->dtype != MOE_DT_F32)
    return fail(MOE_ERR_UNSUPPORTED, "dtype = %d: values are bf16 or fp32", d->dtype);
  if (d->act != MOE_MX4_PLAIN && !(quantize && d->act == MOE_MX4_SWIGLU))
    return fail(MOE_ERR_INVALID_ARGUMENT, "act = %d: MOE_MX4_PLAIN%s", d->act,
                quantize ? " or MOE_MX4_SWIGLU" : "");
  if (quantize && d->n_src < 0)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n_src = %lld < 0", (long long)d->n_src);
  return check_ld(d->ld, int64_t(d->k) * (d->act == MOE_MX4_SWIGLU ? 2 : 1), "ld");
}

Mx4Args mx4_args(const moe_mx4_desc* d) {
  Mx4Args a{};
  a.mats = d->n_mats;
  a.rows = d->rows;
  a.k = d->k;
  a.bf16 = d->dtype == MOE_DT_BF16;
  a.swiglu = d->act == MOE_MX4_SWIGLU;
  a.ld = pitch(d->ld, int64_t(d->k) * (a.swiglu ? 2 : 1));
  a.n_src = d->n_src;
  return a;
}

moe_status validate(const moe_mx4_gemm_desc* d) {
  if (!d) return fail(MOE_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->rows < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "rows = %lld < 0", (long long)d->rows);
  if (d->n_groups < 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n_groups = %d < 1", d->n_groups);
  if (d->n_groups > 512) return fail(MOE_ERR_UNSUPPORTED, "n_groups = %d > 512", d->n_groups);
  if (d->n < 1 || d->k < 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n = %d, k = %d: both >= 1", d->n, d->k);
  if (d->n > (1 << 20) || d->k > (1 << 20))
    return fail(MOE_ERR_UNSUPPORTED, "n = %d, k = %d: up to 2^20", d->n, d->k);
  const int64_t kb = (d->k + 31) / 32, kg = (kb + 3) / 4;
  if (d->n * kb * 16 >= kInt31)
    return fail(MOE_ERR_UNSUPPORTED, "n * ceil(k / 32) * 16 must be < 2^31 bytes");
  // the kernels address a step's scales with 32-bit byte offsets, one word of rows
  // past the last included
  if (d->rows >= (int64_t(1) << 28) || d->rows * kg * 4 >= kInt31)
    return fail(MOE_ERR_UNSUPPORTED, "rows * ceil(k / 128) * 4 must be < 2^31, rows < 2^28");
  // tiles (of at least 32 x 128 outputs) are counted in 32 bits
  if ((d->rows / 32 + d->n_groups) * (d->n / 128 + 1) >= (int64_t(1) << 30))
    return fail(MOE_ERR_UNSUPPORTED, "rows * n: below 2^42 outputs a call");
  if (d->out_dtype != MOE_DT_BF16 && d->out_dtype != MOE_DT_F32)
    return fail(MOE_ERR_UNSUPPORTED, "out_dtype = %d: bf16 or fp32", d->out_dtype);
  return check_ld(d->ld_y, d->n, "ld_y");
}

}  // namespace

extern "C" {

moe_status moe_rmsnorm_forward(const moe_rmsnorm_desc* desc, const void* x, const void* residual,
                               const float* weight, void* y, uint8_t* codes, float* scale,
                               void* sum, float* rstd, hipStream_t stream) {
  moe_status st = validate(desc);
  if (st) return st;
  if (desc->n == 0) return MOE_OK;
  const unsigned el = size_of(desc->dtype);
  st = check({{x, "x", el, true}, {residual, "residual", el, false}, {weight, "weight", 16, false},
              {y, "y", el, false}, {scale, "scale", 16, false}, {sum, "sum", el, false},
              {rstd, "rstd", 16, false}});
  if (st) return st;
  if (!y && !codes) return fail(MOE_ERR_INVALID_ARGUMENT, "y and codes: at least one");
  if (!codes != !scale) return fail(MOE_ERR_INVALID_ARGUMENT, "codes and scale: both or neither");
  if (!residual != !sum)
    return fail(MOE_ERR_INVALID_ARGUMENT, "residual and sum: both or neither");
  RmsArgs a = rms_args(desc);
  a.x = x;
  a.r = residual;
  a.w = weight;
  a.y = y;
  a.q = codes;
  a.scale = scale;
  a.s = sum;
  a.rstd = rstd;
  HIP_TRY(launch_rmsnorm_forward(a, stream), "RMS norm");
  return MOE_OK;
}

moe_status moe_rmsnorm_backward_workspace_size(const moe_rmsnorm_desc* desc, size_t* bytes) {
  moe_status st = validate(desc);
  if (st) return st;
  if (!bytes) return fail(MOE_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = rms_ws(desc);
  return MOE_OK;
}

moe_status moe_rmsnorm_backward(const moe_rmsnorm_desc* desc, const void* dy, const void* x,
                                const float* weight, const float* rstd, const void* dresidual,
                                void* dx, float* dweight, void* ws, size_t ws_bytes,
                                hipStream_t stream) {
  moe_status st = validate(desc);
  if (st) return st;
  const unsigned el = size_of(desc->dtype);
  const bool rows = desc->n > 0;
  st = check({{dy, "dy", el, rows}, {x, "x", el, rows}, {weight, "weight", 16, false},
              {rstd, "rstd", 16, rows}, {dresidual, "dresidual", el, false}, {dx, "dx", el, rows},
              {dweight, "dweight", 16, false}, {ws, "ws", 16, rows && dweight}});
  if (st) return st;
  if (dweight && ws_bytes < rms_ws(desc))
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL,
                "moe_rmsnorm_backward needs %zu workspace bytes, got %zu", rms_ws(desc), ws_bytes);
  RmsArgs a = rms_args(desc);
  a.x = x;
  a.r = dresidual;
  a.w = weight;
  a.y = const_cast<void*>(dy);
  a.s = dx;
  a.rstd = const_cast<float*>(rstd);
  HIP_TRY(launch_rmsnorm_backward(a, dweight, static_cast<float*>(ws), stream),
          "RMS norm backward");
  return MOE_OK;
}

moe_status moe_token_dispatch_workspace_size(const moe_dispatch_desc* desc, size_t* bytes) {
  moe_status st = validate(desc, true);
  if (st) return st;
  if (!bytes) return fail(MOE_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = dispatch_workspace(desc->T, desc->top_k, desc->n_experts);
  return MOE_OK;
}

moe_status moe_token_dispatch(const moe_dispatch_desc* desc, const int32_t* topk_idx,
                              const void* x, const float* x_scale, int32_t* offsets,
                              int32_t* perm, int32_t* inv, void* x_perm, float* x_perm_scale,
                              void* ws, size_t ws_bytes, hipStream_t stream) {
  moe_status st = validate(desc, true);
  if (st) return st;
  const unsigned el = size_of(desc->dtype);
  const bool pairs = desc->T > 0, moved = pairs && x;
  const bool fp8 = desc->dtype == MOE_DT_FP8_E4M3;
  st = check({{topk_idx, "topk_idx", 4, pairs}, {x, "x", el, false},
              {x_scale, "x_scale", 4, moved && fp8}, {offsets, "offsets", 4, true},
              {perm, "perm", 4, pairs}, {inv, "inv", 4, pairs}, {x_perm, "x_perm", el, moved},
              {x_perm_scale, "x_perm_scale", 4, moved && fp8}});
  if (st) return st;
  if (!x && x_perm) return fail(MOE_ERR_INVALID_ARGUMENT, "x_perm without x");
  if ((!fp8 || !x) && (x_scale || x_perm_scale))
    return fail(MOE_ERR_INVALID_ARGUMENT, "scales without E4M3 rows");
  const size_t need = dispatch_workspace(desc->T, desc->top_k, desc->n_experts);
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "moe_token_dispatch needs %zu workspace bytes, got %zu",
                need, ws_bytes);
  st = check({{ws, "ws", 16, need > 0}});
  if (st) return st;
  DispatchArgs a{};
  a.T = desc->T;
  a.rows = rows_of(desc);
  a.E = desc->n_experts;
  a.K = desc->top_k;
  a.idx = topk_idx;
  a.x = static_cast<const uint8_t*>(x);
  a.x2 = reinterpret_cast<const uint8_t*>(x_scale);
  a.offsets = offsets;
  a.perm = perm;
  a.inv = inv;
  a.xp = static_cast<uint8_t*>(x_perm);
  a.xp2 = reinterpret_cast<uint8_t*>(x_perm_scale);
  a.row_bytes = int64_t(desc->d) * el;
  a.row2_bytes = (int64_t(desc->d) + 127) / 128 * 4;
  a.ldt = pitch(desc->ld_t, desc->d) * el;
  a.ldp = pitch(desc->ld_p, desc->d) * el;
  HIP_TRY(launch_dispatch(a, ws, stream), "token dispatch");
  return MOE_OK;
}

moe_status moe_token_combine(const moe_dispatch_desc* desc, const void* y_perm,
                             const int32_t* inv, const float* weight, const void* base, void* y,
                             hipStream_t stream) {
  moe_status st = validate(desc, false);
  if (st) return st;
  if (desc->T == 0) return MOE_OK;
  const unsigned el = size_of(desc->dtype);
  st = check({{y_perm, "y_perm", el, true}, {inv, "inv", 4, true}, {weight, "weight", 4, false},
              {base, "base", el, false}, {y, "y", el, true}});
  if (st) return st;
  CombineArgs a = combine_args(desc);
  a.yp = y_perm;
  a.inv = inv;
  a.w = weight;
  a.base = base;
  a.y = y;
  HIP_TRY(launch_token_combine(a, stream), "token combine");
  return MOE_OK;
}

moe_status moe_token_combine_backward(const moe_dispatch_desc* desc, const void* dy,
                                      const void* y_perm, const int32_t* inv,
                                      const float* weight, void* dy_perm, float* dweight,
                                      hipStream_t stream) {
  moe_status st = validate(desc, false);
  if (st) return st;
  if (desc->T == 0) return MOE_OK;
  const unsigned el = size_of(desc->dtype);
  st = check({{dy, "dy", el, true}, {y_perm, "y_perm", el, dweight != nullptr},
              {inv, "inv", 4, true}, {weight, "weight", 4, false}, {dy_perm, "dy_perm", el, false},
              {dweight, "dweight", 4, false}});
  if (st) return st;
  if (!dy_perm && !dweight)
    return fail(MOE_ERR_INVALID_ARGUMENT, "dy_perm and dweight: at least one");
  CombineArgs a = combine_args(desc);
  a.yp = y_perm;
  a.inv = inv;
  a.w = weight;
  a.base = dy;
  a.y = dy_perm;
  a.dw = dweight;
  HIP_TRY(launch_token_combine_backward(a, stream), "token combine backward");
  return MOE_OK;
}

moe_status moe_mx4_quantize(const moe_mx4_desc* desc, const void* src, const int32_t* perm,
                            uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  moe_status st = validate(desc, true);
  if (st) return st;
  if (desc->n_mats == 0 || desc->rows == 0) return MOE_OK;
  // no row of an empty src is read, whatever perm holds
  st = check({{src, "src", size_of(desc->dtype), !perm || desc->n_src > 0},
              {perm, "perm", 4, false}, {codes, "codes", 16, true}, {scales, "scales", 16, true}});
  if (st) return st;
  if (perm && desc->n_mats != 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "perm with n_mats = %lld: one matrix",
                (long long)desc->n_mats);
  Mx4Args a = mx4_args(desc);
  a.src = src;
  a.perm = perm;
  a.codes = codes;
  a.scales = scales;
  HIP_TRY(launch_mx4_quantize(a, stream), "4-bit quantization");
  return MOE_OK;
}

moe_status moe_mx4_dequantize(const moe_mx4_desc* desc, const uint8_t* codes,
                              const uint8_t* scales, void* dst, hipStream_t stream) {
  moe_status st = validate(desc, false);
  if (st) return st;
  if (desc->n_mats == 0 || desc->rows == 0) return MOE_OK;
  st = check({{codes, "codes", 16, true}, {scales, "scales", 16, true},
              {dst, "dst", size_of(desc->dtype), true}});
  if (st) return st;
  Mx4Args a = mx4_args(desc);
  a.codes = const_cast<uint8_t*>(codes);
  a.scales = const_cast<uint8_t*>(scales);
  a.dst = dst;
  HIP_TRY(launch_mx4_dequantize(a, stream), "4-bit dequantization");
  return MOE_OK;
}

moe_status moe_mx4_gemm(const moe_mx4_gemm_desc* desc, const uint8_t* x_codes,
                        const uint8_t* x_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                        const int32_t* offsets, void* y, hipStream_t stream) {
  moe_status st = validate(desc);
  if (st) return st;
  if (desc->rows == 0) return MOE_OK;
  st = check({{x_codes, "x_codes", 16, true}, {x_scales, "x_scales", 16, true},
              {w_codes, "w_codes", 16, true}, {w_scales, "w_scales", 16, true},
              {offsets, "offsets", 4, true}, {y, "y", size_of(desc->out_dtype), true}});
  if (st) return st;
  Mx4GemmArgs a{};
  a.rows = desc->rows;
  a.ldy = pitch(desc->ld_y, desc->n);
  a.G = desc->n_groups;
  a.n = desc->n;
  a.k = desc->k;
  a.out_f32 = desc->out_dtype == MOE_DT_F32;
  a.xc = x_codes;
  a.xs = x_scales;
  a.wc = w_codes;
  a.wsc = w_scales;
  a.offsets = offsets;
  a.y = y;
  HIP_TRY(launch_mx4_gemm(a, stream), "4-bit grouped product");
  return MOE_OK;
}

}  // extern "C"
