// Layer norm, forward and backward (definition in dsmoe_ops.h).
//
// Memory-bound: the forward reads x (and the residual) once and writes y (and
// the sum) once; the backward reads dy, x (and dresidual) once and writes dx
// once. A row lives in the registers of NW waves (1, 4 or 8 by its length), 8
// adjacent values per lane and chunk. Rows longer than kMaxRow are read again
// from memory for every pass instead.
//
// The backward of rows past 8192 values holds two rows, the weight and two
// column sums at 32 values a lane each, which fill 256 registers or do not fit them:
// 180 bytes a lane go to scratch memory with fp32 rows and dresidual, 20 without.
// 2048 x 16384 (replayed graphs): bf16 44 us, with dresidual 53; fp32 98 and 157, 3.4
// to 5.0 TB/s where a large copy reaches 4.8.
#include "device_common.h"
#include "internal.h"
#include "row_io.h"

namespace dsmoe {

namespace {

struct FwdArgs {
  const void* x;
  const void* r;
  const float* w;
  const float* b;
  void* y;
  void* sum;
  float* mean;
  float* rstd;
  int64_t n, ldx, ldr, ldy, lds;
  int d;
  float eps, inv_d;
  bool stream;  // row outputs past the caches
};

// A block of max(NW, 4) waves; NW waves own a row, CH chunks of 8 values per
// lane. One block per row (NW > 1) or per four rows (NW == 1).
//
// Mean first, then the squares of what is left, both from registers: merging
// per-lane moments in one pass is as stable but took ten times the vector
// operations, and those then bound the kernel. Bound by memory: 8192 x 7168
// bf16 with a residual takes 83 us, 470 MB at 5.7 TB/s, past a large copy's rate.
template <class T, int NW, int CH, bool RES>
__global__ __launch_bounds__(NW == 1 ? 256 : NW * 64) void norm_fwd_kernel(FwdArgs a) {
  __shared__ float slot[2][NW];
  constexpr int LANES = NW * 64;
  const int64_t row = NW == 1 ? int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (NW == 1 && row >= a.n) return;
  const int lane = threadIdx.x & (LANES - 1);
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  float v[CH][VEC];
  typename RawOf<T>::type rx[CH], rr[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i0 = (c * LANES + lane) * VEC;
    rx[c] = load8(x, i0, a.d);
    if constexpr (RES) rr[c] = load8(static_cast<const T*>(a.r) + row * a.ldr, i0, a.d);
  }
  float s = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    unpack(rx[c], v[c], a.d - (c * LANES + lane) * VEC);
    if constexpr (RES) {
      float r[VEC];
      unpack(rr[c], r, a.d - (c * LANES + lane) * VEC);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[c][j] += r[j];
    }
    s += ((v[c][0] + v[c][1]) + (v[c][2] + v[c][3])) + ((v[c][4] + v[c][5]) + (v[c][6] + v[c][7]));
  }
  const float mean = row_sum<NW>(s, slot[0]) * a.inv_d;
  float q = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i0 = (c * LANES + lane) * VEC;
    const int cnt = a.d - i0;
    if constexpr (RES) {
      if (cnt > 0) store8(static_cast<T*>(a.sum) + row * a.lds + i0, v[c], cnt, a.stream);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[c][j] -= mean;
    if (cnt >= VEC) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) q += v[c][j] * v[c][j];
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) q += j < cnt ? v[c][j] * v[c][j] : 0.0f;
    }
  }
  const float rstd = rsqrtf(row_sum<NW>(q, slot[1]) * a.inv_d + a.eps);
  if (lane == 0 && a.mean) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i0 = (c * LANES + lane) * VEC;
    const int cnt = a.d - i0;
    if (cnt <= 0) continue;
    float w[VEC], b[VEC], o[VEC];
    load_vec(a.w, w, i0, a.d, 1.0f);
    load_vec(a.b, b, i0, a.d, 0.0f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = v[c][j] * rstd * w[j] + b[j];
    store8(y + i0, o, cnt, a.stream);
  }
}

// Rows past the register path: 512 threads, the row read three times (after the
// first time from L2).
template <class T>
__global__ __launch_bounds__(512) void norm_fwd_long_kernel(FwdArgs a) {
  __shared__ float slot[2][8];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* r = a.r ? static_cast<const T*>(a.r) + row * a.ldr : nullptr;
  auto get = [&](int i0, float (&v)[VEC]) {
    unpack(load8(x, i0, a.d), v, a.d - i0);
    if (r) {
      float u[VEC];
      unpack(load8(r, i0, a.d), u, a.d - i0);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] += u[j];
    }
  };
  float s = 0.0f, q = 0.0f;
  for (int i0 = threadIdx.x * VEC; i0 < a.d; i0 += 512 * VEC) {
    float v[VEC];
    get(i0, v);
    s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
  }
  const float mean = row_sum<8>(s, slot[0]) * a.inv_d;
  for (int i0 = threadIdx.x * VEC; i0 < a.d; i0 += 512 * VEC) {
    float v[VEC];
    get(i0, v);
    const int cnt = a.d - i0;
#pragma unroll
    for (int j = 0; j < VEC; ++j) q += j < cnt ? (v[j] - mean) * (v[j] - mean) : 0.0f;
  }
  const float rstd = rsqrtf(row_sum<8>(q, slot[1]) * a.inv_d + a.eps);
  if (threadIdx.x == 0 && a.mean) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  for (int i0 = threadIdx.x * VEC; i0 < a.d; i0 += 512 * VEC) {
    float v[VEC], w[VEC], b[VEC], o[VEC];
    get(i0, v);
    const int cnt = a.d - i0;
    if (r) store8(static_cast<T*>(a.sum) + row * a.lds + i0, v, cnt, a.stream);
    load_vec(a.w, w, i0, a.d, 1.0f);
    load_vec(a.b, b, i0, a.d, 0.0f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = (v[j] - mean) * rstd * w[j] + b[j];
    store8(static_cast<T*>(a.y) + row * a.ldy + i0, o, cnt, a.stream);
  }
}

// ---- backward ---------------------------------------------------------------

struct BwdNormArgs {
  const void* dy;
  const void* x;
  const float* w;
  const float* mean;
  const float* rstd;
  const void* dr;
  void* dx;
  float* part;  // [gridDim.x][2][d] partial dweight, dbias; NULL: not wanted
  int64_t n, ldx, ldr, ldy, lds;
  int d;
  bool stream;  // row outputs past the caches
};

template <int NW>
__device__ __forceinline__ float2 row_sum2(float2 s, float2* slot) {
  s.x = wave_sum(s.x);
  s.y = wave_sum(s.y);
  if constexpr (NW > 1) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = s;
    __syncthreads();
    s = slot[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      s.x += slot[w].x;
      s.y += slot[w].y;
    }
  }
  return s;
}

// A row group (NW waves) takes rows slot, slot + slots, ... and keeps the
// column sums of dy z and dy for its columns in registers over all of them;
// each block then writes one partial sum per column. The next row is loaded
// while the current one is reduced. With NW == 1 the block's four waves add
// their column sums through LDS, in wave order.
// Bound by memory: 8192 x 7168 bf16 with dresidual, both kernels: 87 us, 470 MB
// at 5.4 TB/s.
// WHOLE: no row ends inside a lane's eight values, so nothing is shifted at its end.
template <class T, int NW, int CH, bool RES, bool WHOLE>
__global__ __launch_bounds__(NW == 1 ? 256 : NW * 64) void norm_bwd_kernel(BwdNormArgs a) {
  constexpr int LANES = NW * 64, GROUPS = NW == 1 ? 4 : 1;
  // Four chunks leave no registers for the next row's dresidual: the row's own is loaded
  // behind its other loads (2048 x 16384 bf16: 64 us before, 53 so; fp32 189 and 157).
  constexpr bool LATE = RES && CH == 4;
  // Whether large dx goes past the caches. bf16 without dresidual, past them / through them,
  // inputs from memory and (replayed graphs) from the caches as far as they fit: 8192 x 4096
  // 46.4 / 45.1 us and 38.2 / 38.1, 4096 x 16384 91 / 88, 2048 x 16384 53 / 51 and 44.4 / 43.7,
  // but 8192 x 7168 73 / 71 and 58 / 70. With it: 8192 x 7168 91.7 / 91.9 and 88 / 89, 32768 x
  // 4096 196 / 200, 2048 x 16384 65 / 64 and 53 / 56.
  constexpr bool PAST = RES || (NW == 8 && CH == 2);
  __shared__ float2 slot[2][NW];
  const int lane = threadIdx.x & (LANES - 1);
  auto load = [&](const void* rows, int64_t at, int i0) {
    if constexpr (WHOLE)
      return load8_whole(static_cast<const T*>(rows) + at, i0, a.d);
    else
      return load8(static_cast<const T*>(rows) + at, i0, a.d);
  };
  auto open = [&](const typename RawOf<T>::type& r, float (&v)[VEC], int cnt) {
    if constexpr (WHOLE)
      unpack_whole(r, v);
    else
      unpack(r, v, cnt);
  };
  const int64_t first = int64_t(blockIdx.x) * GROUPS + (NW == 1 ? threadIdx.x >> 6 : 0);
  const int64_t stride = int64_t(gridDim.x) * GROUPS;
  float aw[CH][VEC], ab[CH][VEC], w[CH][VEC];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i0 = (c * LANES + lane) * VEC;
    load_vec(a.w, w[c], i0, a.d, 1.0f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) aw[c][j] = ab[c][j] = 0.0f;
  }
  typename RawOf<T>::type rx[CH], rg[CH], rr[CH];
  float mu = 0.0f, rs = 0.0f;
  auto fetch = [&](int64_t row) {
    mu = a.mean[row];
    rs = a.rstd[row];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i0 = (c * LANES + lane) * VEC;
      rx[c] = load(a.x, row * a.ldx, i0);
      rg[c] = load(a.dy, row * a.ldy, i0);
      if constexpr (RES && !LATE) rr[c] = load(a.dr, row * a.ldr, i0);
    }
  };
  if (first < a.n) fetch(first);
  int par = 0;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  for (int64_t row = first; row < a.n; row += stride) {
    float z[CH][VEC], g[CH][VEC];
    typename RawOf<T>::type kr[CH];
    float2 s = make_float2(0.0f, 0.0f);
    const float m = mu, r = rs;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int cnt = a.d - (c * LANES + lane) * VEC;
      open(rx[c], z[c], cnt);
      open(rg[c], g[c], cnt);
      if constexpr (LATE)
        kr[c] = load(a.dr, row * a.ldr, (c * LANES + lane) * VEC);
      else if constexpr (RES)
        kr[c] = rr[c];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        z[c][j] = (WHOLE ? 0 : j) < cnt ? (z[c][j] - m) * r : 0.0f;
        aw[c][j] += g[c][j] * z[c][j];
        ab[c][j] += g[c][j];
        g[c][j] *= w[c][j];
        s.x += g[c][j];
        s.y += g[c][j] * z[c][j];
      }
    }
    if (row + stride < a.n) fetch(row + stride);
    s = row_sum2<NW>(s, slot[par]);
    par ^= 1;  // the next row's sums go to the other slots: one barrier per row
    const float c1 = s.x * inv_d, c2 = s.y * inv_d;
    T* dx = static_cast<T*>(a.dx) + row * a.lds;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i0 = (c * LANES + lane) * VEC;
      if (i0 >= a.d) continue;
      float o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = r * (g[c][j] - c1 - z[c][j] * c2);
      if constexpr (RES) {
        float e[VEC];
        open(kr[c], e, a.d - i0);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] += e[j];
      }
      store8(dx + i0, o, a.d - i0, PAST && a.stream);
    }
  }
  if (!a.part) return;
  float* pw = a.part + int64_t(blockIdx.x) * 2 * a.d;
  if constexpr (NW == 1) {
    __shared__ float red[4][2][CH * 64 * VEC];
    const int wv = threadIdx.x >> 6;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        red[wv][0][(c * 64 + lane) * VEC + j] = aw[c][j];
        red[wv][1][(c * 64 + lane) * VEC + j] = ab[c][j];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < a.d; i += 256) {
      pw[i] = ((red[0][0][i] + red[1][0][i]) + red[2][0][i]) + red[3][0][i];
      pw[a.d + i] = ((red[0][1][i] + red[1][1][i]) + red[2][1][i]) + red[3][1][i];
    }
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i0 = (c * LANES + lane) * VEC;
      if (i0 >= a.d) continue;
      store8(pw + i0, aw[c], a.d - i0);
      store8(pw + a.d + i0, ab[c], a.d - i0);
    }
  }
}

// Rows past the register path: dx in two passes over the row; the column sums
// come from norm_cols_kernel.
template <class T>
__global__ __launch_bounds__(512) void norm_bwd_long_kernel(BwdNormArgs a) {
  __shared__ float2 slot[8];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* dy = static_cast<const T*>(a.dy) + row * a.ldy;
  const float m = a.mean[row], r = a.rstd[row];
  auto get = [&](int i0, float (&z)[VEC], float (&g)[VEC]) {
    float w[VEC];
    const int cnt = a.d - i0;
    unpack(load8(x, i0, a.d), z, a.d - i0);
    unpack(load8(dy, i0, a.d), g, a.d - i0);
    load_vec(a.w, w, i0, a.d, 1.0f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      z[j] = j < cnt ? (z[j] - m) * r : 0.0f;
      g[j] *= w[j];
    }
  };
  float2 s = make_float2(0.0f, 0.0f);
  for (int i0 = threadIdx.x * VEC; i0 < a.d; i0 += 512 * VEC) {
    float z[VEC], g[VEC];
    get(i0, z, g);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      s.x += g[j];
      s.y += g[j] * z[j];
    }
  }
  s = row_sum2<8>(s, slot);
  const float c1 = s.x / static_cast<float>(a.d), c2 = s.y / static_cast<float>(a.d);
  for (int i0 = threadIdx.x * VEC; i0 < a.d; i0 += 512 * VEC) {
    float z[VEC], g[VEC], o[VEC];
    get(i0, z, g);
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = r * (g[j] - c1 - z[j] * c2);
    if (a.dr) {
      float e[VEC];
      unpack(load8(static_cast<const T*>(a.dr) + row * a.ldr, i0, a.d), e, a.d - i0);
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] += e[j];
    }
    store8(static_cast<T*>(a.dx) + row * a.lds + i0, o, a.d - i0);
  }
}

// Partial column sums of dy z and dy: block (x, y) takes 512 columns and rows
// y, y + gridDim.y, ...
template <class T>
__global__ __launch_bounds__(64) void norm_cols_kernel(BwdNormArgs a) {
  const int i0 = (blockIdx.x * 64 + threadIdx.x) * VEC;
  if (i0 >= a.d) return;
  const int cnt = a.d - i0;
  float aw[VEC] = {}, ab[VEC] = {};
  for (int64_t row = blockIdx.y; row < a.n; row += gridDim.y) {
    float z[VEC], g[VEC];
    unpack(load8(static_cast<const T*>(a.x) + row * a.ldx, i0, a.d), z, a.d - i0);
    unpack(load8(static_cast<const T*>(a.dy) + row * a.ldy, i0, a.d), g, a.d - i0);
    const float m = a.mean[row], r = a.rstd[row];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      aw[j] += g[j] * ((z[j] - m) * r);
      ab[j] += g[j];
    }
  }
  float* pw = a.part + int64_t(blockIdx.y) * 2 * a.d;
  store8(pw + i0, aw, cnt);
  store8(pw + a.d + i0, ab, cnt);
}

// dweight, dbias = sums of the partial rows [parts][2 d], in a fixed order: a
// block takes 32 columns, its 32 half-waves a run of the parts each, whose sums
// are then added in order. Latency-bound: eight loads in flight per
// lane, half the columns of a wave per block (8192 x 2048 bf16, the whole
// backward: 31 us with one load and 64 columns, 23 so).
__global__ __launch_bounds__(1024) void norm_sum_parts_kernel(const float* part, int parts, int d,
                                                              float* dw, float* db) {
  __shared__ float red[32][32];
  const int run = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t width = 2 * int64_t(d), col = int64_t(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (col < width) {
    const int per = (parts + 31) / 32, p0 = run * per, p1 = min(parts, p0 + per);
    const float* at = part + p0 * width + col;
    int left = p1 - p0;
    for (; left >= 8; left -= 8, at += 8 * width) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = at[i * width];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; left > 0; --left, at += width) s += *at;
  }
  red[run][lane] = s;
  __syncthreads();
  if (run || col >= width) return;
#pragma unroll
  for (int w = 1; w < 32; ++w) s += red[w][lane];
  if (col < d) {
    if (dw) dw[col] = s;
  } else if (db) {
    db[col - d] = s;
  }
}

// ---- shapes ------------------------------------------------------------------

constexpr int kMaxRow = 16384;  // 8 waves x 64 lanes x 4 chunks x 8 values

// Waves and chunks of a row of d values.
struct RowShape {
  int nw, ch;
};
RowShape row_shape(int d) {
  if (d <= 512) return {1, 1};
  if (d <= 1024) return {1, 2};
  if (d <= 2048) return {4, 1};
  if (d <= 4096) return {4, 2};
  if (d <= 8192) return {8, 2};
  return {8, 4};
}

template <class T, bool RES>
void fwd_launch(const FwdArgs& a, hipStream_t s) {
  const unsigned rows = static_cast<unsigned>(a.n), quads = static_cast<unsigned>((a.n + 3) / 4);
  if (a.d > kMaxRow) {
    hipLaunchKernelGGL(norm_fwd_long_kernel<T>, dim3(rows), dim3(512), 0, s, a);
    return;
  }
  const RowShape r = row_shape(a.d);
#define NORM_CASE(NW, CH)                                                                 \
  if (r.nw == NW && r.ch == CH) {                                                         \
    hipLaunchKernelGGL((norm_fwd_kernel<T, NW, CH, RES>), dim3(NW == 1 ? quads : rows),   \
                       dim3(NW == 1 ? 256 : NW * 64), 0, s, a);                           \
    return;                                                                               \
  }
  NORM_CASE(1, 1)
  NORM_CASE(1, 2)
  NORM_CASE(4, 1)
  NORM_CASE(4, 2)
  NORM_CASE(8, 2)
  NORM_CASE(8, 4)
#undef NORM_CASE
}

template <class T, bool RES>
void fwd_dispatch(const FwdArgs& a, hipStream_t s) {
  const int64_t per = kMaxBlocks * (a.d <= kMaxRow && row_shape(a.d).nw == 1 ? 4 : 1);
  for (int64_t row = 0; row < a.n; row += per) {
    FwdArgs b = a;
    b.n = a.n - row < per ? a.n - row : per;
    b.x = static_cast<const T*>(a.x) + row * a.ldx;
    if (RES) b.r = static_cast<const T*>(a.r) + row * a.ldr;
    b.y = static_cast<T*>(a.y) + row * a.ldy;
    if (RES) b.sum = static_cast<T*>(a.sum) + row * a.lds;
    if (a.mean) b.mean = a.mean + row;
    if (a.mean) b.rstd = a.rstd + row;
    fwd_launch<T, RES>(b, s);
  }
}

template <class T, bool RES>
void bwd_dispatch(const BwdNormArgs& a, int parts, hipStream_t s) {
  if (a.d > kMaxRow) {
    // the column sums first: dx may take dy's place
    if (a.part)
      hipLaunchKernelGGL(norm_cols_kernel<T>, dim3((a.d + 511) / 512, parts), dim3(64), 0, s, a);
    for (int64_t row = 0; row < a.n; row += kMaxBlocks) {
      BwdNormArgs b = a;
      b.n = a.n - row < kMaxBlocks ? a.n - row : kMaxBlocks;
      b.dy = static_cast<const T*>(a.dy) + row * a.ldy;
      b.x = static_cast<const T*>(a.x) + row * a.ldx;
      if (a.dr) b.dr = static_cast<const T*>(a.dr) + row * a.ldr;
      b.dx = static_cast<T*>(a.dx) + row * a.lds;
      b.mean = a.mean + row;
      b.rstd = a.rstd + row;
      hipLaunchKernelGGL(norm_bwd_long_kernel<T>, dim3(static_cast<unsigned>(b.n)), dim3(512), 0, s,
                         b);
    }
    return;
  }
  const RowShape r = row_shape(a.d);
  // bf16 rows that end inside no lane's eight values take a kernel without the shifts of
  // row ends, without / with dresidual (us, replayed graphs): 8192 x 512 9.7 / 10.2, with
  // the shifts 10.1 / 10.9; 8192 x 1024 14.6 / 16.8, 15.2 / 17.1; 8192 x 7168 58 / 87.7,
  // 60 / 89.5; 2048 x 8200 28 / 32, 36 / 39; 64 x 16384 14.8 / 15.0, 16.3 / 16.9. fp32 rows' ends are loaded value by value.
  const bool whole = sizeof(T) == 2 && a.d % VEC == 0;
#define NORM_CASE(NW, CH)                                                                  \
  if (r.nw == NW && r.ch == CH) {                                                          \
    hipLaunchKernelGGL(whole ? (norm_bwd_kernel<T, NW, CH, RES, sizeof(T) == 2>)           \
                             : (norm_bwd_kernel<T, NW, CH, RES, false>),                   \
                       dim3(parts), dim3(NW == 1 ? 256 : NW * 64), 0, s, a);               \
    return;                                                                                \
  }
  NORM_CASE(1, 1)
  NORM_CASE(1, 2)
  NORM_CASE(4, 1)
  NORM_CASE(4, 2)
  NORM_CASE(8, 2)
  NORM_CASE(8, 4)
#undef NORM_CASE
}

}  // namespace

// Blocks of the backward, each with a partial row of column sums: 8 waves per CU.
// More blocks hide more latency but write and add more partial rows. 8192 bf16 rows,
// without / with dresidual, of 256, 512 and 1024 blocks (us, replayed graphs): 512 values,
// where four rows share a block, 11.2 / 11.3, 10.0 / 10.3, 12.2 / 12.0; 2048 30 / 30, 23 /
// 26, 25 / 29; 2815 46 / 53, 35 / 41, 36 / 49; 4096 41 / 45, 38 / 46, 42 / 54; 7168, blocks
// of 8 waves, 59 / 87, 63 / 93, 76 / 106.
int norm_backward_parts(int64_t n, int d) {
  if (d > kMaxRow) return static_cast<int>(n < 1 ? 1 : n < 256 ? n : 256);
  const int nw = row_shape(d).nw;
  const int64_t groups = nw == 1 ? (n + 3) / 4 : n, most = nw == 8 ? 256 : 512;
  return static_cast<int>(groups < 1 ? 1 : groups < most ? groups : most);
}

namespace {
bool streamed(const NormArgs& p) { return p.n * p.d * (p.bf16 ? 2 : 4) >= kStreamBytes; }
}  // namespace

hipError_t launch_norm_forward(const NormArgs& p, hipStream_t s) {
  if (p.n == 0) return hipSuccess;
  const FwdArgs a{p.x, p.r, p.w, p.b, p.y, p.s, p.mean, p.rstd,
                  p.n, p.ldx, p.ldr, p.ldy, p.lds, p.d, p.eps, 1.0f / p.d, streamed(p)};
  if (p.bf16)
    p.r ? fwd_dispatch<uint16_t, true>(a, s) : fwd_dispatch<uint16_t, false>(a, s);
  else
    p.r ? fwd_dispatch<float, true>(a, s) : fwd_dispatch<float, false>(a, s);
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs& p, float* dw, float* db, float* part,
                                hipStream_t s) {
  const int parts = norm_backward_parts(p.n, p.d);
  const bool sums = dw || db;
  if (p.n > 0) {
    const BwdNormArgs a{p.y, p.x, p.w, p.mean, p.rstd, p.r, p.s, sums ? part : nullptr,
                        p.n, p.ldx, p.ldr, p.ldy, p.lds, p.d, streamed(p)};
    if (p.bf16)
      p.r ? bwd_dispatch<uint16_t, true>(a, parts, s) : bwd_dispatch<uint16_t, false>(a, parts, s);
    else
      p.r ? bwd_dispatch<float, true>(a, parts, s) : bwd_dispatch<float, false>(a, parts, s);
  }
  if (sums)
    hipLaunchKernelGGL(norm_sum_parts_kernel, dim3((2 * p.d + 31) / 32), dim3(1024), 0, s, part,
                       p.n > 0 ? parts : 0, p.d, dw, db);
  return hipGetLastError();
}

}  // namespace dsmoe
