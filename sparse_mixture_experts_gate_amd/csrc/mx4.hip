// Microscaled 4-bit values: quantization and dequantization (formats and layouts
// in dsmoe_tokens.h).
//
// Memory-bound: a lane holds 8 adjacent values (one word of codes), four lanes a
// block, 16 lanes four blocks, whose scale bytes make one word. LANES lanes take a row,
// or 512 values of one; a workgroup takes PER rows for each, so that the scale words of a
// column of blocks, which lie row by row, leave as one run of words and not one by one
// from several XCDs. bf16 rows of 8192 x 7168: 28 us, 148 MB at 5.3 TB/s; 32 matrices of
// 4096 x 7168: 407 us, 2.4 GB at 5.8, and back 363 us at 6.5.
#include "device_common.h"
#include "internal.h"
#include "row_io.h"

namespace dsmoe {

namespace {

// Lanes of a row: 16 up to 128 values, 32 up to 256, else a wave (63 matrices of 1408 x
// 128 bf16 values: 18 us and back 13 by a wave a row, 7.2 and 7.1 by 16 lanes; 18 of 3343
// x 256 14 and 11, 8.9 and 8.6 by 32).
int lanes_of(int k) { return k <= 128 ? 16 : k <= 256 ? 32 : 64; }
// Blocks with PER = 4 from which on these are taken; fewer leave CUs idle, and PER = 2
// makes twice as many (3 x 613 x 1407 values the same). 8192 x 7168 bf16: 28 us with 4,
// 29 with 2, 30 with 8.
constexpr int64_t kWide = 1024;

struct QArgs {
  const void* src;
  const int32_t* perm;
  uint8_t* codes;
  uint8_t* scales;
  void* dst;
  int64_t rows, ld, n_src, mat;  // mat: values between matrices
  // blocks of a matrix's rows; this launch's first (rows < 2^31: both in 32 bits); spans
  uint32_t row_blocks, rb0, spans;
  int k, kb, kg;
  bool stream;  // the output past the caches
};

// A block's matrix, row block and span. Adjacent blocks take adjacent spans, so that
// those that run together read and write whole rows (32 matrices of 4096 x 7168,
// quantized and back: 436 and 365 us; the blocks of one span first 471 and 477, with
// 32 rows a block).
struct Block {
  int64_t mat, rows;
  int span;
  __device__ __forceinline__ explicit Block(const QArgs& a) {
    const uint32_t q = blockIdx.x / a.spans, rb = a.rb0 + q, m = rb / a.row_blocks;
    span = static_cast<int>(blockIdx.x - q * a.spans);
    mat = m;
    rows = rb - m * a.row_blocks;
  }
};

// 2^e, e = -127 .. 127 (2^-127 is below the normal numbers).
__device__ __forceinline__ float power_of_two(int e) {
  return __int_as_float(e > -127 ? (e + 127) << 23 : 1 << 22);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_get(uint32_t v) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true));
}
// Largest of four adjacent lanes' values (magnitude bits of floats), in all of them.
__device__ __forceinline__ uint32_t max4(uint32_t v) {
  v = max(v, dpp_get<0xb1>(v));  // quad_perm 1 0 3 2
  return max(v, dpp_get<0x4e>(v));  // quad_perm 2 3 0 1
}

// Codes (one word) and scale byte of a lane's eight values of a block. Scaling by
// a power of two is exact, so the conversion's rounding is the only one.
__device__ __forceinline__ uint32_t mx4_codes(const float (&v)[VEC], uint32_t& byte) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < VEC; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
  top = max4(top);
  if (top >= 0x7f800000u) {
    byte = 255;
    return 0;
  }
  // floor(log2) is the exponent; of numbers below the normal ones it is below -126,
  // where e is -127 either way
  const int e = max(static_cast<int>(top >> 23) - 127 - 2, -127);
  byte = static_cast<uint32_t>(e + 127);
  const float inv = power_of_two(-e);
  float q[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) q[j] = v[j] * inv;
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[0], q[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[2], q[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[4], q[5], 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[6], q[7], 1.0f, 3);
  return w;
}

// Rows of a workgroup: four waves, each of 64 / LANES groups of lanes.
template <int LANES, int PER>
constexpr int kRows = 4 * (64 / LANES) * PER;

// Block (matrix, rows, span of 8 LANES values).
template <class T, int LANES, int PER, bool SWIGLU>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(QArgs a) {
  constexpr int ROWS = kRows<LANES, PER>, GROUPS = 64 / LANES;
  __shared__ uint32_t words[LANES / 16][ROWS];
  const int lane = threadIdx.x & (LANES - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = wave * PER * GROUPS + (threadIdx.x & 63) / LANES;  // and every GROUPS rows
  const Block b(a);
  const int64_t mat = b.mat, r0 = b.rows * ROWS;
  const int i0 = (b.span * LANES + lane) * VEC;
  const T* src = static_cast<const T*>(a.src) + mat * a.mat;
  typename RawOf<T>::type raw[PER], raw2[SWIGLU ? PER : 1];
  int d[PER];  // lengths of the rows, 0 for none
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int64_t r = r0 + first + i * GROUPS;
    int64_t from = r < a.rows ? r : -1;
    if (a.perm && from >= 0) {
      from = a.perm[r];
      if (from >= a.n_src) from = -1;
    }
    d[i] = from >= 0 ? a.k : 0;
    if constexpr (GROUPS == 1) d[i] = __builtin_amdgcn_readfirstlane(d[i]);
    const T* p = src + (from >= 0 ? from : 0) * a.ld;
    raw[i] = load8(p, i0, d[i]);
    if constexpr (SWIGLU) raw2[i] = load8(p + a.k, i0, d[i]);
  }
  uint8_t* codes = a.codes + (mat * a.rows + r0) * a.kb * 16;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    float v[VEC];
    unpack(raw[i], v, d[i] - i0);
    if constexpr (SWIGLU) {
      float up[VEC];
      unpack(raw2[i], up, d[i] - i0);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = silu_f32(v[j]) * up[j];
    }
    uint32_t byte;
    const uint32_t w = mx4_codes(v, byte);
    const int row = first + i * GROUPS;
    if (r0 + row < a.rows && i0 < a.kb * 32) {
      uint32_t* to = reinterpret_cast<uint32_t*>(codes + int64_t(row) * a.kb * 16 + i0 / 2);
      if (a.stream) {  // (the empty statements keep the two stores apart)
        asm volatile("");
        __builtin_nontemporal_store(w, to);
        asm volatile("");
      } else {
        *to = w;
      }
    }
    // bytes of lanes 0, 4, 8 and 12 of each 16, blocks past the last one 0
    uint32_t s = (lane & 3) == 0 && i0 < a.kb * 32 ? byte << (8 * ((lane >> 2) & 3)) : 0u;
    s |= dpp_get<0x124>(s);  // row_ror:4
    s |= dpp_get<0x128>(s);  // row_ror:8
    if ((lane & 15) == 0) words[lane >> 4][row] = s;
  }
  __syncthreads();
  if (threadIdx.x < LANES / 16 * ROWS) {
    const int g = threadIdx.x / ROWS, row = threadIdx.x % ROWS;
    const int64_t kg = b.span * (LANES / 16) + g;
    if (kg < a.kg && r0 + row < a.rows)
      reinterpret_cast<uint32_t*>(a.scales)[(mat * a.kg + kg) * a.rows + r0 + row] = words[g][row];
  }
}

// The values of eight codes times 2^(byte - 127); byte 255 makes them NaN.
__device__ __forceinline__ void mx4_values(uint32_t w, uint32_t byte, float (&v)[VEC]) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const float s = byte == 255 ? __int_as_float(0x7fc00000) : power_of_two(static_cast<int>(byte) - 127);
  const f32x2_t p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3)};
#pragma unroll
  for (int j = 0; j < VEC; ++j) v[j] = p[j >> 1][j & 1] * s;
}

constexpr int kDeqPer = 2;
template <class T, int LANES>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(QArgs a) {
  constexpr int PER = kDeqPer, GROUPS = 64 / LANES;
  const int lane = threadIdx.x & (LANES - 1), wave = threadIdx.x >> 6;
  const Block b(a);
  const int64_t mat = b.mat, r0 = b.rows * kRows<LANES, PER> + wave * PER * GROUPS +
                                  (threadIdx.x & 63) / LANES;
  const int i0 = (b.span * LANES + lane) * VEC;
  if (i0 >= a.k) return;
  const int64_t kg = i0 / 128, col = i0 / 2;
  uint32_t w[PER], sc[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int64_t r = min(r0 + i * GROUPS, a.rows - 1);
    w[i] = *reinterpret_cast<const uint32_t*>(a.codes + (mat * a.rows + r) * a.kb * 16 + col);
    sc[i] = reinterpret_cast<const uint32_t*>(a.scales)[(mat * a.kg + kg) * a.rows + r];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (r0 + i * GROUPS >= a.rows) return;
    float v[VEC];
    mx4_values(w[i], (sc[i] >> (8 * ((i0 >> 5) & 3))) & 255u, v);
    store8(static_cast<T*>(a.dst) + mat * a.mat + (r0 + i * GROUPS) * a.ld + i0, v, a.k - i0,
           a.stream);
  }
}

QArgs q_args(const Mx4Args& p) {
  QArgs a{};
  a.src = p.src;
  a.perm = p.perm;
  a.codes = p.codes;
  a.scales = p.scales;
  a.dst = p.dst;
  a.rows = p.rows;
  a.ld = p.ld;
  a.n_src = p.n_src;
  a.mat = p.rows * p.ld;
  a.k = p.k;
  a.kb = (p.k + 31) / 32;
  a.kg = (a.kb + 3) / 4;
  a.spans = (p.k + lanes_of(p.k) * VEC - 1) / (lanes_of(p.k) * VEC);
  // (32 matrices of 4096 x 7168: codes 425 -> 407 us, values in bf16 400 -> 365)
  const int64_t out = p.dst ? int64_t(p.k) * (p.bf16 ? 2 : 4) : a.kb * 16;
  a.stream = p.mats * p.rows * out >= kFarBytes;
  return a;
}

// Blocks of `per` rows and one span, in launches of whole row blocks that count their
// work items in 32 bits.
template <class Go>
void in_launches(QArgs a, int64_t mats, int per, Go&& go) {
  const int64_t most = 2 * kMaxBlocks / a.spans;
  a.row_blocks = static_cast<uint32_t>((a.rows + per - 1) / per);
  const int64_t total = mats * a.row_blocks;
  for (int64_t rb = 0; rb < total; rb += most) {
    a.rb0 = static_cast<uint32_t>(rb);
    go(a, dim3(static_cast<unsigned>((total - rb < most ? total - rb : most) * a.spans)));
  }
}

template <class T, int LANES, int PER, bool SWIGLU>
void quantize_by(const QArgs& a, int64_t mats, hipStream_t s) {
  in_launches(a, mats, kRows<LANES, PER>, [&](const QArgs& b, dim3 grid) {
    hipLaunchKernelGGL((mx4_quantize_kernel<T, LANES, PER, SWIGLU>), grid, dim3(256), 0, s, b);
  });
}
template <class T, int LANES, bool SWIGLU>
void quantize_with(const QArgs& a, int64_t mats, hipStream_t s) {
  constexpr int rows = kRows<LANES, 4>;
  if (mats * ((a.rows + rows - 1) / rows) * a.spans >= kWide)
    quantize_by<T, LANES, 4, SWIGLU>(a, mats, s);
  else
    quantize_by<T, LANES, 2, SWIGLU>(a, mats, s);
}
template <class T, bool SWIGLU>
void quantize(const QArgs& a, int64_t mats, hipStream_t s) {
  const int lanes = lanes_of(a.k);
  if (lanes == 16)
    quantize_with<T, 16, SWIGLU>(a, mats, s);
  else if (lanes == 32)
    quantize_with<T, 32, SWIGLU>(a, mats, s);
  else
    quantize_with<T, 64, SWIGLU>(a, mats, s);
}

template <class T, int LANES>
void dequantize_with(const QArgs& a, int64_t mats, hipStream_t s) {
  in_launches(a, mats, kRows<LANES, kDeqPer>, [&](const QArgs& b, dim3 grid) {
    hipLaunchKernelGGL((mx4_dequantize_kernel<T, LANES>), grid, dim3(256), 0, s, b);
  });
}
template <class T>
void dequantize(const QArgs& a, int64_t mats, hipStream_t s) {
  const int lanes = lanes_of(a.k);
  if (lanes == 16)
    dequantize_with<T, 16>(a, mats, s);
  else if (lanes == 32)
    dequantize_with<T, 32>(a, mats, s);
  else
    dequantize_with<T, 64>(a, mats, s);
}

}  // namespace

hipError_t launch_mx4_quantize(const Mx4Args& p, hipStream_t s) {
  if (p.mats == 0 || p.rows == 0) return hipSuccess;
  const QArgs a = q_args(p);
  if (p.bf16)
    p.swiglu ? quantize<uint16_t, true>(a, p.mats, s) : quantize<uint16_t, false>(a, p.mats, s);
  else
    p.swiglu ? quantize<float, true>(a, p.mats, s) : quantize<float, false>(a, p.mats, s);
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const Mx4Args& p, hipStream_t s) {
  if (p.mats == 0 || p.rows == 0) return hipSuccess;
  const QArgs a = q_args(p);
  p.bf16 ? dequantize<uint16_t>(a, p.mats, s) : dequantize<float>(a, p.mats, s);
  return hipGetLastError();
}

}  // namespace dsmoe
