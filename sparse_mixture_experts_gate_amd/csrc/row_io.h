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

// Eight values at p, of which the first `cnt` exist (the rest read as zero).
// Rows may start at any element, so the 16-byte accesses go through memcpy,
// which the compiler emits as one unaligned access.
template <class T>
__device__ __forceinline__ typename RawOf<T>::type load8(const T* p, int cnt) {
  typename RawOf<T>::type r;
  if (cnt >= VEC) {
    __builtin_memcpy(&r, p, sizeof(r));
  } else {
    T tmp[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) tmp[j] = j < cnt ? p[j] : T(0);
    __builtin_memcpy(&r, tmp, sizeof(r));
  }
  return r;
}
__device__ __forceinline__ void unpack(const Raw16& r, float (&v)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    v[j] = __uint_as_float((j & 1) ? (r.w[j >> 1] & 0xFFFF0000u) : (r.w[j >> 1] << 16));
}
__device__ __forceinline__ void unpack(const Raw32& r, float (&v)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) v[j] = __uint_as_float(r.w[j]);
}
// Two fp32 -> bf16 to nearest even (one instruction; NaN stays NaN).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));

// The first `cnt` of eight values. `stream`: past the caches, for outputs larger
// than the L2s together, which no reader would find there. The empty statements keep
// the compiler from merging the two stores into one without the hint.
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[VEC], int cnt,
                                       bool stream = false) {
  if (cnt >= VEC) {
    u32x4_any_t r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
    if (stream) {
      asm volatile("");
      __builtin_nontemporal_store(r, reinterpret_cast<u32x4_any_t*>(p));
      asm volatile("");
    } else {
      *reinterpret_cast<u32x4_any_t*>(p) = r;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < cnt) p[j] = static_cast<uint16_t>(bf16_pair(v[j], 0.0f));
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
__device__ __forceinline__ void load_vec(const float* p, float (&v)[VEC], int cnt, float none) {
  if (p) {
    unpack(load8(p, cnt), v);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = none;
  }
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

// bf16 row outputs of this many bytes or more are stored past the caches: eight L2s
// of 4 MB (layer norm of 8192 x 7168 with a residual 98 -> 95 us, its backward 92 ->
// 89, 4096 x 4096 19 -> 17; fp32 rows of 8192 x 7168, in both stores, 137 -> 155).
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
