// RMS norm, forward and backward (definition in dsmoe_tokens.h).
//
// Memory-bound: the forward reads x (and the residual) once and writes what is
// asked of rows, codes and the sum once; the backward reads dy, x (and
// dresidual) once and writes dx once. A row lives in the registers of NW waves
// (1, 4 or 8 by its length), 8 adjacent values per lane and chunk, so that 16
// lanes hold a 1x128 tile side by side and four lane rotations find its largest
// value. Rows longer than kMaxRow are read again from memory for every pass instead.
#include "device_common.h"
#include "internal.h"
#include "row_io.h"

namespace dsmoe {

namespace {

constexpr int kTile = 128;  // values that share an E4M3 scale

struct RmsFwdArgs {
  const void* x;
  const void* r;
  const float* w;
  void* y;        // NULL: no rows
  uint8_t* q;     // NULL: no codes
  float* scale;   // [n][tiles]
  void* sum;
  float* rstd;
  int64_t n, ldx, ldr, ldy, lds, ldq;
  int d, tiles;
  float eps, inv_d;
  bool stream;  // row outputs past the caches
};

// Largest of 16 adjacent lanes' values as unsigned integers, in all of them: for
// magnitudes of floats this orders NaN above infinity above all numbers.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
                    0, static_cast<int>(v), CTRL, 0xf, 0xf, true)));
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = dpp_max<0x128>(v);  // row_ror:8
  v = dpp_max<0x124>(v);
  v = dpp_max<0x122>(v);
  return dpp_max<0x121>(v);
}

typedef uint32_t u32x2_any_t __attribute__((ext_vector_type(2), aligned(1)));

// E4M3 codes of a lane's eight values of a tile; its lane 0 stores the scale.
__device__ __forceinline__ void store_codes(const float (&o)[VEC], int cnt, uint8_t* q,
                                            float* scale, bool first) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    top = max(top, __float_as_uint(o[j]) & 0x7fffffffu);
  top = max16(top);
  if (cnt <= 0) return;
  const float amax = __uint_as_float(top);
  uint32_t lo, hi;
  float sc = amax / 448.0f;
  if (top >= 0x7f800000u) {
    lo = hi = 0x7f7f7f7fu;
  } else if (amax < 0x1p-100f) {
    lo = hi = 0u;
    sc = 1.0f;
  } else {
    const float inv = 448.0f / amax;
    lo = e4m3_pack4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
    hi = e4m3_pack4(o[4] * inv, o[5] * inv, o[6] * inv, o[7] * inv);
  }
  if (first) *scale = sc;
  if (cnt >= VEC) {
    *reinterpret_cast<u32x2_any_t*>(q) = u32x2_any_t{lo, hi};
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < cnt) q[j] = static_cast<uint8_t>((j < 4 ? lo : hi) >> (8 * (j & 3)));
  }
}

// A block of max(NW, 4) waves; NW waves own a row, CH chunks of 8 values per
// lane. One block per row (NW > 1) or per four rows (NW == 1). All loads go out before
// the sum, so a row costs one trip to memory. Bound by memory: 8192 x 7168 bf16 with a
// residual 84 us, 470 MB at 5.6 TB/s; with codes too 93 us, 530 MB at 5.7.
template <class T, int NW, int CH, bool RES>
__global__ __launch_bounds__(NW == 1 ? 256 : NW * 64) void rms_fwd_kernel(RmsFwdArgs a) {
  __shared__ float slot[NW];
  constexpr int LANES = NW * 64;
  const int64_t row = NW == 1 ? int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (NW == 1 && row >= a.n) return;
  const int lane = threadIdx.x & (LANES - 1);
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  float v[CH][VEC], w[CH][VEC];
  typename RawOf<T>::type rx[CH], rr[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i0 = (c * LANES + lane) * VEC;
    rx[c] = load8(x, i0, a.d);
    if constexpr (RES) rr[c] = load8(static_cast<const T*>(a.r) + row * a.ldr, i0, a.d);
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i0 = (c * LANES + lane) * VEC;
    load_vec(a.w, w[c], i0, a.d, 1.0f);
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
    float q[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) q[j] = v[c][j] * v[c][j];
    s += ((q[0] + q[1]) + (q[2] + q[3])) + ((q[4] + q[5]) + (q[6] + q[7]));
  }
  const float rstd = rsqrtf(row_sum<NW>(s, slot) * a.inv_d + a.eps);
  if (lane == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i0 = (c * LANES + lane) * VEC;
    const int cnt = a.d - i0;
    float o[VEC];
    if constexpr (RES) {
      if (cnt > 0) store8(static_cast<T*>(a.sum) + row * a.lds + i0, v[c], cnt, a.stream);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = v[c][j] * rstd * w[c][j];
    if (a.y && cnt > 0) store8(static_cast<T*>(a.y) + row * a.ldy + i0, o, cnt, a.stream);
    if (a.q)
      store_codes(o, cnt, a.q + row * a.ldq + i0, a.scale + row * a.tiles + i0 / kTile,
                  (lane & 15) == 0);
  }
}

// Rows past the register path: 512 threads, the row read twice (the second time
// from L2). At the longest row that registers hold, 2048 x 16384 bf16: 58 us so, 42 in
// registers; the backward 60 and 39 (replayed graphs).
template <class T>
__global__ __launch_bounds__(512) void rms_fwd_long_kernel(RmsFwdArgs a) {
  __shared__ float slot[8];
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
  float s = 0.0f;
  for (int i0 = threadIdx.x * VEC; i0 < a.d; i0 += 512 * VEC) {
    float v[VEC];
    get(i0, v);
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] *= v[j];
    s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
  }
  const float rstd = rsqrtf(row_sum<8>(s, slot) * a.inv_d + a.eps);
  if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
  // whole tiles of lanes stay in the loop: the scales are met across 16 lanes
  for (int i0 = threadIdx.x * VEC; i0 < a.tiles * kTile; i0 += 512 * VEC) {
    float v[VEC], w[VEC], o[VEC];
    const int cnt = a.d - i0;
    get(i0, v);
    load_vec(a.w, w, i0, a.d, 1.0f);
    if (r && cnt > 0) store8(static_cast<T*>(a.sum) + row * a.lds + i0, v, cnt, a.stream);
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = v[j] * rstd * w[j];
    if (a.y && cnt > 0) store8(static_cast<T*>(a.y) + row * a.ldy + i0, o, cnt, a.stream);
    if (a.q)
      store_codes(o, cnt, a.q + row * a.ldq + i0, a.scale + row * a.tiles + i0 / kTile,
                  (threadIdx.x & 15) == 0);
  }
}

// ---- backward ---------------------------------------------------------------

struct RmsBwdArgs {
  const void* dy;
  const void* x;
  const float* w;
  const float* rstd;
  const void* dr;
  void* dx;
  float* part;  // [blocks][d] partial dweight; NULL: not wanted, or
  float* dw;    // dweight from blocks of this launch behind the rows' own
  int blocks;   // of rows
  int64_t n, ldx, ldr, ldy, lds;
  int d;
  bool stream;  // row outputs past the caches
};

// dweight of 32 columns: the block's half-waves take rows of dy and x each, eight of both
// in flight, and their sums are added in order. For few rows, beside the blocks that write
// dx; it reads dy itself, which dx must not overwrite.
template <class T, int HALVES>
__device__ void dweight_columns(const RmsBwdArgs& a, int block) {
  __shared__ float red[HALVES][32];
  const int half = threadIdx.x >> 5, lane = threadIdx.x & 31, col = block * 32 + lane;
  const int n = static_cast<int>(a.n);
  float s = 0.0f;
  if (col < a.d) {
    const T* x = static_cast<const T*>(a.x) + col;
    const T* dy = static_cast<const T*>(a.dy) + col;
    constexpr int N = 8;
    for (int r0 = half; r0 < n; r0 += N * HALVES) {
      float v[N], g[N], rs[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = min(r0 + i * HALVES, n - 1);
        v[i] = one_value(x[row * a.ldx]);
        g[i] = one_value(dy[row * a.ldy]);
        rs[i] = a.rstd[row];
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (r0 + i * HALVES < n) s += g[i] * (v[i] * rs[i]);
    }
  }
  red[half][lane] = s;
  __syncthreads();
  if (half || col >= a.d) return;
#pragma unroll
  for (int h = 1; h < HALVES; ++h) s += red[h][lane];
  a.dw[col] = s;
}

// A row group (NW waves) takes rows slot, slot + slots, ... and keeps the column
// sums of dy z for its columns in registers over all of them; each block then
// writes one partial sum per column. The next row is loaded while the current one
// is reduced. With NW == 1 the block's four waves add their column sums through
// LDS, in wave order.
// Bound by memory: 8192 x 7168 bf16 with dresidual, both kernels: 87 us, 470 MB at 5.4
// TB/s.
template <class T, int NW, int CH, bool RES>
__global__ __launch_bounds__(NW == 1 ? 256 : NW * 64) void rms_bwd_kernel(RmsBwdArgs a) {
  constexpr int LANES = NW * 64, GROUPS = NW == 1 ? 4 : 1;
  // Four chunks of fp32 rows leave no registers for the next row's dresidual: the row's
  // own is loaded behind its other loads (2048 x 16384: 145 us before, 118 so; bf16, which
  // has them, 48 and 53).
  constexpr bool LATE = RES && CH == 4 && sizeof(T) == 4;
  __shared__ float slot[2][NW];
  const int lane = threadIdx.x & (LANES - 1);
  if (static_cast<int>(blockIdx.x) >= a.blocks) {
    dweight_columns<T, (NW == 1 ? 4 : NW) * 2>(a, blockIdx.x - a.blocks);
    return;
  }
  const int64_t first = int64_t(blockIdx.x) * GROUPS + (NW == 1 ? threadIdx.x >> 6 : 0);
  const int64_t stride = int64_t(a.blocks) * GROUPS;
  float aw[CH][VEC], w[CH][VEC];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i0 = (c * LANES + lane) * VEC;
    load_vec(a.w, w[c], i0, a.d, 1.0f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) aw[c][j] = 0.0f;
  }
  typename RawOf<T>::type rx[CH], rg[CH], rr[CH];
  float rs = 0.0f;
  auto fetch = [&](int64_t row) {
    rs = a.rstd[row];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i0 = (c * LANES + lane) * VEC;
      rx[c] = load8(static_cast<const T*>(a.x) + row * a.ldx, i0, a.d);
      rg[c] = load8(static_cast<const T*>(a.dy) + row * a.ldy, i0, a.d);
      if constexpr (RES && !LATE)
        rr[c] = load8(static_cast<const T*>(a.dr) + row * a.ldr, i0, a.d);
    }
  };
  if (first < a.n) fetch(first);
  int par = 0;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  for (int64_t row = first; row < a.n; row += stride) {
    float z[CH][VEC], g[CH][VEC];
    typename RawOf<T>::type kr[CH];
    float s = 0.0f;
    const float r = rs;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int cnt = a.d - (c * LANES + lane) * VEC;
      unpack(rx[c], z[c], cnt);
      unpack(rg[c], g[c], cnt);
      if constexpr (LATE)
        kr[c] = load8(static_cast<const T*>(a.dr) + row * a.ldr, (c * LANES + lane) * VEC, a.d);
      else if constexpr (RES)
        kr[c] = rr[c];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        z[c][j] = j < cnt ? z[c][j] * r : 0.0f;
        aw[c][j] += g[c][j] * z[c][j];
        g[c][j] *= w[c][j];
        s += g[c][j] * z[c][j];
      }
    }
    if (row + stride < a.n) fetch(row + stride);
    const float c2 = row_sum<NW>(s, slot[par]) * inv_d;
    par ^= 1;  // the next row's sums go to the other slots: one barrier per row
    T* dx = static_cast<T*>(a.dx) + row * a.lds;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i0 = (c * LANES + lane) * VEC;
      if (i0 >= a.d) continue;
      float o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = r * (g[c][j] - z[c][j] * c2);
      if constexpr (RES) {
        float e[VEC];
        unpack(kr[c], e, a.d - i0);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] += e[j];
      }
      store8(dx + i0, o, a.d - i0, a.stream);
    }
  }
  if (!a.part) return;
  float* pw = a.part + int64_t(blockIdx.x) * a.d;
  if constexpr (NW == 1) {
    __shared__ float red[4][CH * 64 * VEC];
    const int wv = threadIdx.x >> 6;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < VEC; ++j) red[wv][(c * 64 + lane) * VEC + j] = aw[c][j];
    __syncthreads();
    for (int i = threadIdx.x; i < a.d; i += 256)
      pw[i] = ((red[0][i] + red[1][i]) + red[2][i]) + red[3][i];
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i0 = (c * LANES + lane) * VEC;
      if (i0 < a.d) store8(pw + i0, aw[c], a.d - i0);
    }
  }
}

// Rows past the register path: dx in two passes over the row; the column sums
// come from rms_cols_kernel.
template <class T>
__global__ __launch_bounds__(512) void rms_bwd_long_kernel(RmsBwdArgs a) {
  __shared__ float slot[8];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* dy = static_cast<const T*>(a.dy) + row * a.ldy;
  const float r = a.rstd[row];
  auto get = [&](int i0, float (&z)[VEC], float (&g)[VEC]) {
    float w[VEC];
    const int cnt = a.d - i0;
    unpack(load8(x, i0, a.d), z, a.d - i0);
    unpack(load8(dy, i0, a.d), g, a.d - i0);
    load_vec(a.w, w, i0, a.d, 1.0f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      z[j] = j < cnt ? z[j] * r : 0.0f;
      g[j] *= w[j];
    }
  };
  float s = 0.0f;
  for (int i0 = threadIdx.x * VEC; i0 < a.d; i0 += 512 * VEC) {
    float z[VEC], g[VEC];
    get(i0, z, g);
#pragma unroll
    for (int j = 0; j < VEC; ++j) s += g[j] * z[j];
  }
  const float c2 = row_sum<8>(s, slot) / static_cast<float>(a.d);
  for (int i0 = threadIdx.x * VEC; i0 < a.d; i0 += 512 * VEC) {
    float z[VEC], g[VEC], o[VEC];
    get(i0, z, g);
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = r * (g[j] - z[j] * c2);
    if (a.dr) {
      float e[VEC];
      unpack(load8(static_cast<const T*>(a.dr) + row * a.ldr, i0, a.d), e, a.d - i0);
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] += e[j];
    }
    store8(static_cast<T*>(a.dx) + row * a.lds + i0, o, a.d - i0, a.stream);
  }
}

// Partial column sums of dy z: block (x, y) takes 512 columns and rows y, y +
// gridDim.y, ...
template <class T>
__global__ __launch_bounds__(64) void rms_cols_kernel(RmsBwdArgs a) {
  const int i0 = (blockIdx.x * 64 + threadIdx.x) * VEC;
  if (i0 >= a.d) return;
  const int cnt = a.d - i0;
  float aw[VEC] = {};
  for (int64_t row = blockIdx.y; row < a.n; row += gridDim.y) {
    float z[VEC], g[VEC];
    unpack(load8(static_cast<const T*>(a.x) + row * a.ldx, i0, a.d), z, a.d - i0);
    unpack(load8(static_cast<const T*>(a.dy) + row * a.ldy, i0, a.d), g, a.d - i0);
    const float r = a.rstd[row];
#pragma unroll
    for (int j = 0; j < VEC; ++j) aw[j] += g[j] * (z[j] * r);
  }
  store8(a.part + int64_t(blockIdx.y) * a.d + i0, aw, cnt);
}

// dweight = sum of the partial rows [parts][d], in a fixed order: a block takes
// 32 columns, its 32 half-waves a run of the parts each, whose sums are then
// added in order; eight loads in flight per lane (latency-bound: 4 us for 256 parts of
// 1407 columns).
__global__ __launch_bounds__(1024) void rms_sum_parts_kernel(const float* part, int parts, int d,
                                                             float* dw) {
  __shared__ float red[32][32];
  const int run = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t width = d, col = int64_t(blockIdx.x) * 32 + lane;
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
  dw[col] = s;
}

// ---- shapes ------------------------------------------------------------------

constexpr int kMaxRow = 16384;  // 8 waves x 64 lanes x 4 chunks x 8 values

// Waves and chunks of a row of d values: the least of both that hold the row, one wave
// up to two chunks (no barrier), eight from four chunks of four waves on. Measured, 8192
// bf16 rows with a residual, forward / backward (us, replayed graphs), waves x chunks:
//   512   1x1 6.9 / 8.9   2x1  7.4 / 19     1024  1x2 12 / 14   2x1 13 / 19   4x1 12 / 22
//   2048  4x1  21 / 22    2x2   21 / 25     1x4    22 / 21    8x1  22 / 35
//   4096  4x2  39 / 36    8x1   39 / 35  (2816 values: 30 / 37 and 32 / 45)
//   7168  8x2  69 / 61    4x4   70 / 64     8x4    76 / 113
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
void fwd_launch(const RmsFwdArgs& a, hipStream_t s) {
  const unsigned rows = static_cast<unsigned>(a.n), quads = static_cast<unsigned>((a.n + 3) / 4);
  if (a.d > kMaxRow) {
    hipLaunchKernelGGL(rms_fwd_long_kernel<T>, dim3(rows), dim3(512), 0, s, a);
    return;
  }
  const RowShape r = row_shape(a.d);
#define RMS_CASE(NW, CH)                                                                 \
  if (r.nw == NW && r.ch == CH) {                                                        \
    hipLaunchKernelGGL((rms_fwd_kernel<T, NW, CH, RES>), dim3(NW == 1 ? quads : rows),   \
                       dim3(NW == 1 ? 256 : NW * 64), 0, s, a);                          \
    return;                                                                              \
  }
  RMS_CASE(1, 1)
  RMS_CASE(1, 2)
  RMS_CASE(4, 1)
  RMS_CASE(4, 2)
  RMS_CASE(8, 2)
  RMS_CASE(8, 4)
#undef RMS_CASE
}

template <class T, bool RES>
void fwd_dispatch(const RmsFwdArgs& a, hipStream_t s) {
  const int64_t per = kMaxBlocks * (a.d <= kMaxRow && row_shape(a.d).nw == 1 ? 4 : 1);
  for (int64_t row = 0; row < a.n; row += per) {
    RmsFwdArgs b = a;
    b.n = a.n - row < per ? a.n - row : per;
    b.x = static_cast<const T*>(a.x) + row * a.ldx;
    if (RES) b.r = static_cast<const T*>(a.r) + row * a.ldr;
    if (a.y) b.y = static_cast<T*>(a.y) + row * a.ldy;
    if (a.q) b.q = a.q + row * a.ldq;
    if (a.q) b.scale = a.scale + row * a.tiles;
    if (RES) b.sum = static_cast<T*>(a.sum) + row * a.lds;
    if (a.rstd) b.rstd = a.rstd + row;
    fwd_launch<T, RES>(b, s);
  }
}

template <class T, bool RES>
void bwd_dispatch(const RmsBwdArgs& a, int parts, hipStream_t s) {
  if (a.d > kMaxRow) {
    // the column sums first: dx may take dy's place
    if (a.part)
      hipLaunchKernelGGL(rms_cols_kernel<T>, dim3((a.d + 511) / 512, parts), dim3(64), 0, s, a);
    for (int64_t row = 0; row < a.n; row += kMaxBlocks) {
      RmsBwdArgs b = a;
      b.n = a.n - row < kMaxBlocks ? a.n - row : kMaxBlocks;
      b.dy = static_cast<const T*>(a.dy) + row * a.ldy;
      b.x = static_cast<const T*>(a.x) + row * a.ldx;
      if (a.dr) b.dr = static_cast<const T*>(a.dr) + row * a.ldr;
      b.dx = static_cast<T*>(a.dx) + row * a.lds;
      b.rstd = a.rstd + row;
      hipLaunchKernelGGL(rms_bwd_long_kernel<T>, dim3(static_cast<unsigned>(b.n)), dim3(512), 0, s,
                         b);
    }
    return;
  }
  const RowShape r = row_shape(a.d);
  const int grid = parts + (a.dw ? (a.d + 31) / 32 : 0);
#define RMS_CASE(NW, CH)                                                          \
  if (r.nw == NW && r.ch == CH) {                                                 \
    hipLaunchKernelGGL((rms_bwd_kernel<T, NW, CH, RES>), dim3(grid),              \
                       dim3(NW == 1 ? 256 : NW * 64), 0, s, a);                   \
    return;                                                                       \
  }
  RMS_CASE(1, 1)
  RMS_CASE(1, 2)
  RMS_CASE(4, 1)
  RMS_CASE(4, 2)
  RMS_CASE(8, 2)
  RMS_CASE(8, 4)
#undef RMS_CASE
}

}  // namespace

// Blocks of the backward, each with a partial row of column sums: 8 waves per CU. 8192
// bf16 rows with dresidual, 256 / 512 / 1024 blocks (us): 2048 values 34 / 28 / 29, 4096
// 52 / 53 / 56, 7168 87 / 94 / 96; fp32 rows of 2048 48 / 49 / 50; 512 values, where four
// rows share a block, 10 / 9 / 10 (replayed graphs).
int rmsnorm_backward_parts(int64_t n, int d) {
  if (d > kMaxRow) return static_cast<int>(n < 1 ? 1 : n < 256 ? n : 256);
  const int nw = row_shape(d).nw;
  const int64_t groups = nw == 1 ? (n + 3) / 4 : n, most = nw == 8 ? 256 : 512;
  return static_cast<int>(groups < 1 ? 1 : groups < most ? groups : most);
}

namespace {
// Rows up to which dweight comes from the same launch. With dresidual, one launch / two (us,
// replayed graphs): bf16 128 x 1407 3.7 / 7.0, 256 x 7168 5.5 / 11.5, 512 x 512 5.9 / 6.5, 512
// x 7168 10.9 / 13.6, 1003 x 1407 13.0 / 9.8; fp32 512 x 7168 17.5 / 17.0.
constexpr int64_t kOneLaunch = 512;
bool streamed(const RmsArgs& p) { return p.n * p.d * (p.bf16 ? 2 : 4) >= kStreamBytes; }
}  // namespace

hipError_t launch_rmsnorm_forward(const RmsArgs& p, hipStream_t s) {
  if (p.n == 0) return hipSuccess;
  const RmsFwdArgs a{p.x, p.r, p.w, p.y, p.q, p.scale, p.s, p.rstd, p.n, p.ldx, p.ldr, p.ldy,
                     p.lds, p.ldq, p.d, (p.d + kTile - 1) / kTile, p.eps, 1.0f / p.d, streamed(p)};
  if (p.bf16)
    p.r ? fwd_dispatch<uint16_t, true>(a, s) : fwd_dispatch<uint16_t, false>(a, s);
  else
    p.r ? fwd_dispatch<float, true>(a, s) : fwd_dispatch<float, false>(a, s);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_backward(const RmsArgs& p, float* dw, float* part, hipStream_t s) {
  const int parts = rmsnorm_backward_parts(p.n, p.d);
  const bool one = dw && p.n > 0 && p.n <= kOneLaunch && p.d <= kMaxRow && p.s != p.y;
  if (p.n > 0) {
    const RmsBwdArgs a{p.y, p.x, p.w, p.rstd, p.r, p.s, dw && !one ? part : nullptr,
                       one ? dw : nullptr, parts, p.n, p.ldx, p.ldr, p.ldy, p.lds, p.d, streamed(p)};
    if (p.bf16)
      p.r ? bwd_dispatch<uint16_t, true>(a, parts, s) : bwd_dispatch<uint16_t, false>(a, parts, s);
    else
      p.r ? bwd_dispatch<float, true>(a, parts, s) : bwd_dispatch<float, false>(a, parts, s);
  }
  if (dw && !one)
    hipLaunchKernelGGL(rms_sum_parts_kernel, dim3((p.d + 31) / 32), dim3(1024), 0, s, part,
                       p.n > 0 ? parts : 0, p.d, dw);
  return hipGetLastError();
}

}  // namespace dsmoe
