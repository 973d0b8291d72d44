// Rows of bf16 or fp32 values in registers, eight adjacent ones per lane: loads
// and stores of any alignment, sums over waves and row groups. In an anonymous
// namespace, so each translation unit gets its own copy.
#pragma once

#include "device_common.h"

namespace dsmoe {
namespace {

constexpr int VEC = 8;  // values of a row that one lane holds side by side

struct Raw16 {
  uint32_t w[4];
};
struct Raw32 {
  uint32_t w[8];
};
template <class T>
struct RawOf;
template <>
struct RawOf<uint16_t> {
  using type = Raw16;
};
template <>
struct RawOf<float> {
  using type = Raw32;
};

// The eight values i0 .. i0 + 7 (i0 a multiple of 8) of a row of d values, for unpack.
// Rows may start at any element, so the 16-byte accesses go through memcpy, which the
// compiler emits as one unaligned access.
// bf16: where the row ends among them, they are the row's last eight, which unpack
// shifts into place: one access like the others, not waited for before that. Value by
// value, the halves of words met here and each load of a row's end cost a wait of its
// own (RMS norm of 8192 x 2815 forward 38 us, 33 so; backward 77 and 40; return of 8192
// rows 17 and 12). A lane uses its own values of them only, so another lane may be storing
// the others. Lanes past the row load nothing; unpack gives them zeros.
__device__ __forceinline__ Raw16 load8(const uint16_t* row, int i0, int d) {
  Raw16 r;
  if (d >= VEC) {
    if (i0 < d) __builtin_memcpy(&r, row + min(i0, d - VEC), sizeof(r));
  } else {
    uint16_t tmp[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) tmp[j] = i0 == 0 && j >= VEC - d ? row[j - (VEC - d)] : 0;
    __builtin_memcpy(&r, tmp, sizeof(r));
  }
  return r;
}
// fp32: value by value at the end, zeros past it (shifts cost the registers that the
// backward's occupancy needs: 8192 x 2815 75 us, 78 with them).
__device__ __forceinline__ Raw32 load8(const float* row, int i0, int d) {
  Raw32 r;
  const float* p = row + i0;
  const int cnt = d - i0;
  if (cnt >= VEC) {
    __builtin_memcpy(&r, p, sizeof(r));
  } else {
    float tmp[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) tmp[j] = j < cnt ? p[j] : 0.0f;
    __builtin_memcpy(&r, tmp, sizeof(r));
  }
  return r;
}
// bf16 rows of a multiple of 8 values, which end inside no lane's eight: zeros past the
// row, and nothing for unpack to shift.
__device__ __forceinline__ Raw16 load8_whole(const uint16_t* row, int i0, int d) {
  Raw16 r{};
  if (i0 < d) __builtin_memcpy(&r, row + i0, sizeof(r));
  return r;
}
__device__ __forceinline__ void unpack_whole(const Raw16& r, float (&v)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    v[j] = __uint_as_float((j & 1) ? (r.w[j >> 1] & 0xFFFF0000u) : (r.w[j >> 1] << 16));
}
// load8's values in order, with cnt = d - i0: zeros past the row's end.
__device__ __forceinline__ void unpack(Raw16 r, float (&v)[VEC], int cnt) {
  if (cnt < VEC) {  // the first VEC - cnt are not this lane's
    const int by = VEC - cnt;
    if (by & 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) r.w[j] = (r.w[j] >> 16) | (j < 3 ? r.w[j + 1] << 16 : 0u);
    }
#pragma unroll
    for (int s = 1; s < 4; s *= 2)
#pragma unroll
      for (int j = 0; j < 4; ++j) r.w[j] = by & (2 * s) ? (j + s < 4 ? +r.w[j + s] : 0u) : +r.w[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[j] = cnt > 0 ? +r.w[j] : 0u;
  }
  unpack_whole(r, v);
}
__device__ __forceinline__ void unpack(const Raw32& r, float (&v)[VEC], int) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) v[j] = __uint_as_float(r.w[j]);
}
__device__ __forceinline__ float one_value(uint16_t v) {
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
__device__ __forceinline__ float one_value(float v) { return v; }
// Two fp32 -> bf16 to nearest even (one instruction; NaN stays NaN).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any2_t __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_any2_t __attribute__((aligned(2)));

// The first cnt (1 .. 7) of eight bf16 values: four, two and one of them.
__device__ __forceinline__ void store_end(uint16_t* p, u32x4_any_t r, int cnt) {
  if (cnt & 4) *reinterpret_cast<u32x2_any2_t*>(p) = u32x2_any2_t{r[0], r[1]};
  const uint32_t lo = cnt & 4 ? +r[2] : +r[0], hi = cnt & 4 ? +r[3] : +r[1];
  if (cnt & 2) *reinterpret_cast<u32_any2_t*>(p + (cnt & 4)) = lo;
  if (cnt & 1) p[cnt & 6] = static_cast<uint16_t>(cnt & 2 ? hi : lo);
}

// The first `cnt` of eight values. `stream`: past the caches, for outputs larger
// than the L2s together, which no reader would find there. The empty statements keep
// the compiler from merging the two stores into one without the hint.
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[VEC], int cnt,
                                       bool stream = false) {
  u32x4_any_t r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
  if (cnt >= VEC) {
    if (stream) {
      asm volatile("");
      __builtin_nontemporal_store(r, reinterpret_cast<u32x4_any_t*>(p));
      asm volatile("");
    } else {
      *reinterpret_cast<u32x4_any_t*>(p) = r;
    }
  } else if (cnt > 0) {
    store_end(p, r, cnt);
  }
}
// fp32 values leave in two stores per lane, 16 bytes of every 32 each, which the
// caches have to join: never past them.
__device__ __forceinline__ void store8(float* p, const float (&v)[VEC], int cnt, bool = false) {
  if (cnt >= VEC) {
    typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));
    f32x4_any_t* q = reinterpret_cast<f32x4_any_t*>(p);
    q[0] = f32x4_any_t{v[0], v[1], v[2], v[3]};
    q[1] = f32x4_any_t{v[4], v[5], v[6], v[7]};
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < cnt) p[j] = v[j];
  }
}
// A weight's values, `none` without one, zeros past its end; its last eight shifted into
// place as bf16 rows' are (layer norm of 8192 x 2816 bf16 31 us value by value, 28 so).
__device__ __forceinline__ void load_vec(const float* p, float (&v)[VEC], int i0, int d,
                                         float none) {
  if (!p) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = none;
    return;
  }
  const int cnt = d - i0;
  if (d < VEC) {
    unpack(load8(p, i0, d), v, cnt);
    return;
  }
  Raw32 r;
  if (cnt > 0) __builtin_memcpy(&r, p + min(i0, d - VEC), sizeof(r));
  if (cnt < VEC) {
    const int by = VEC - cnt;
#pragma unroll
    for (int s = 1; s < VEC; s *= 2)
#pragma unroll
      for (int j = 0; j < VEC; ++j) r.w[j] = by & s ? (j + s < VEC ? +r.w[j + s] : 0u) : +r.w[j];
#pragma unroll
    for (int j = 0; j < VEC; ++j) r.w[j] = cnt > 0 ? +r.w[j] : 0u;
  }
  unpack(r, v, cnt);
}

// Sum over the wave by DPP adds (rows of 16 lanes, then across rows; lane 63
// holds it), the same for all lanes.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, true));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111, 0xf>(v);  // row_shr:1
  v = dpp_add<0x112, 0xf>(v);  // row_shr:2
  v = dpp_add<0x114, 0xf>(v);  // row_shr:4
  v = dpp_add<0x118, 0xf>(v);  // row_shr:8
  v = dpp_add<0x142, 0xa>(v);  // row_bcast:15 into rows 1, 3
  v = dpp_add<0x143, 0xc>(v);  // row_bcast:31 into rows 2, 3
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
// Sum over the NW waves of a row group, in wave order. `slot`: NW floats of LDS
// that the next call does not use.
template <int NW>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  v = wave_sum(v);
  if constexpr (NW > 1) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += slot[w];
  }
  return v;
}

// bf16 row outputs of this many bytes or more are stored past the caches: eight L2s of 4
// MB (layer norm of 8192 x 7168, inputs from memory, 52.4 us through the caches and 51.7
// past them, with a residual the same; its backward's sides are in norm.hip; fp32 rows of
// 8192 x 7168, in both stores, 137 -> 155).
constexpr int64_t kStreamBytes = int64_t(32) << 20;
// The same for rows moved between tokens and experts, whose reader comes next and
// finds smaller outputs in the 256 MB that the L2s share: E4M3 rows of 8192 tokens to 8
// experts each (485 MB) 125 -> 102 us, the gradient of 4096 x 6 rows of 2048 (100 MB)
// with the return itself 69 -> 60; a return of 58 MB 32 -> 35, a dispatch of 69 MB 22
// -> 27.
constexpr int64_t kFarBytes = int64_t(96) << 20;

// Blocks of one launch: its work items, up to 512 a block, are counted in 32
// bits and wrap around silently. More rows take further launches.
constexpr int64_t kMaxBlocks = int64_t(1) << 22;

}  // namespace
}  // namespace dsmoe
