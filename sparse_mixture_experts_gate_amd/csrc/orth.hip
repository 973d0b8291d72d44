// Orthogonalized updates of weight matrices by Newton-Schulz products
// (definition in dsmoe_ops.h). With n = min(rows, cols), m = max(rows, cols)
// every matrix is worked on as X [n, m] (transposed on entry and exit where
// rows > cols).
//
// Number format. Every product takes fp16 operands and adds in fp32. fp16
// rather than bf16 because all values have known bounds (|X| <= 1.21, since
// the polynomial maps [0, 1.21] into itself; |A| <= 1.47; |b A + c A A| <= 7),
// so that fixed power-of-two scales use its 11 significant bits without range
// trouble. Three things are kept out of the 16-bit roundings:
//   X  = (hi + lo 2^-11) 2^-12, two fp16 planes: hi feeds the products, both
//        carry X through the a X term. A rank-deficient update needs this:
//        rounding noise in its null space would grow 3.44 times per step.
//   A  = D + R with the diagonal D in fp32, R (zero diagonal) in fp16:
//        A A = R R + D R + R D + D D, of which only R R is a product;
//   B  = b A + c A A = Q + S the same way: X <- (a + Q) X + S X.
// Near convergence D and Q dominate their matrices, so their fp16 roundings
// would be most of the error: on random matrices of 512 x 1024 the result is
// 6e-4 off (2-norm) this way, 1.7e-3 with the diagonals inside, 1.1e-2 in bf16
// throughout. Roundings average over a row: 4e-4 at 2048 x 7168, 1.2e-3 at 64 x
// 64, 1.4e-3 at 16 x 16, and with 1 to 8 rows of few values 1.5e-3 to 3.6e-3 (9e-3
// at worst seen). The polynomial repels at its fixed point (slope -1.58 at
// 0.868), so further steps grow what is there: 2e-3 after eight from 64 x 64 on.
// A null space grows too: rank 1 of 2040 x 3000 is 4e-3 off after eight steps,
// 4e-2 after ten, all of it after 14; in fp32 throughout 1e-2, 1e-1, all.
// Only the last two steps multiply all of X by Q. Before them Q multiplies hi
// alone, as S does: Q + S = B has the null space of X, and applied to two
// different roundings of X its parts would leave noise there that later steps
// amplify (64 x 1000 of rank 5: 3.1e-3 off, 7e-4 so).
//
// A and A A are symmetric: tiles on and below the diagonal are computed and
// stored twice. Per step that leaves n^2 m + n^3 + 2 n^2 m operations.
#include "device_common.h"
#include "gemm16_core.h"
#include "internal.h"
#include "resident_grid.h"

namespace dsmoe {

namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScaleX = 4096.0f;     // 2^12: X planes
constexpr float kScaleLo = 2048.0f;    // 2^11: lo against hi
constexpr float kScaleR = 4096.0f;     // 2^12: off-diagonal of A
constexpr float kScaleS = 1024.0f;     // 2^10: off-diagonal of B
constexpr double kNormEps = 1e-7;

typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));

// Workspace of one matrix (offsets in bytes, planes in rows of pitches mp, np:
// m, n rounded up to whole k-steps, the padding columns zero).
struct OrthShape {
  int n, m, np, mp;
  bool tall;
  int chunks;  // partial sums of squares per matrix
  size_t hi0, hi1, lo, r, s, d, q, part, bytes;
};

constexpr int kSlots = 256;       // workgroups of a round, counters of shared tiles
constexpr int kSumChunk = 16384;  // elements of one partial sum of squares

OrthShape shape_of(int rows, int cols) {
  OrthShape o{};
  o.tall = rows > cols;
  o.n = o.tall ? cols : rows;
  o.m = o.tall ? rows : cols;
  o.np = (o.n + 63) / 64 * 64;
  o.mp = (o.m + 63) / 64 * 64;
  const int64_t el = int64_t(rows) * cols;
  o.chunks = static_cast<int>((el + kSumChunk - 1) / kSumChunk);
  if (o.chunks > 256) o.chunks = 256;
  size_t at = 0;
  auto take = [&](size_t b) {
    const size_t r = at;
    at = (at + b + 255) & ~size_t(255);
    return r;
  };
  const size_t plane = size_t(o.n) * o.mp * 2, sq = size_t(o.n) * o.np * 2;
  o.hi0 = take(plane);
  o.hi1 = take(plane);
  o.lo = take(plane);
  o.r = take(sq);
  o.s = take(sq);
  o.d = take(size_t(o.np) * 4);
  o.q = take(size_t(o.np) * 4);
  o.part = take(size_t(o.chunks) * 8);
  o.bytes = at;
  return o;
}

struct PrepArgs {
  int32_t* count;  // counters of shared tiles, cleared here
  const void* grad;
  const float* m_in;
  float* m_out;
  char* ws;
  OrthShape o;
  int rows, cols;
  float momentum;
  int nesterov;
};

__device__ __forceinline__ float load_grad(const float* p) { return *p; }
__device__ __forceinline__ float load_grad(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float4 load_grad4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ float4 load_grad4(const uint16_t* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
}

// Momentum, and the partial sums of squares of u (fp64: any scale of the
// gradient squares without overflow or underflow). Block (chunk, matrix).
// Bound by memory: 16 matrices of 2048 x 7168 fp32 in 545 us, 5.2 TB/s.
template <class T, bool MOM>
__global__ __launch_bounds__(256) void orth_sum_kernel(PrepArgs a) {
  __shared__ double red[4];
  if (blockIdx.x == 0 && blockIdx.y == 0) a.count[threadIdx.x] = 0;
  if (blockIdx.x == 0)  // the padding of the diagonal
    for (int i = a.o.n + threadIdx.x; i < a.o.np; i += 256)
      reinterpret_cast<float*>(a.ws + blockIdx.y * a.o.bytes + a.o.d)[i] = 0.0f;
  static_assert(kSlots == 256, "one counter per thread");
  const int64_t el = int64_t(a.rows) * a.cols, mat = blockIdx.y;
  const T* g = static_cast<const T*>(a.grad) + mat * el;
  const int64_t per = ((el + a.o.chunks - 1) / a.o.chunks + 1023) / 1024 * 1024;
  const int64_t e0 = int64_t(blockIdx.x) * per, e1 = min(e0 + per, el);
  double s = 0.0;
  auto one = [&](float u, float mi, float& mo) {
    if constexpr (MOM) {
      mo = a.momentum * mi + u;
      u = a.nesterov ? u + a.momentum * mo : mo;
    }
    s += double(u) * u;
  };
  const float* mi = MOM ? a.m_in + mat * el : nullptr;
  float* mo = MOM ? a.m_out + mat * el : nullptr;
  if (el % 4 == 0) {  // every matrix starts on a vector
#pragma unroll 4
    for (int64_t i = e0 + threadIdx.x * 4; i < e1; i += 1024) {
      const float4 u = load_grad4(g + i);
      float4 m = make_float4(0.0f, 0.0f, 0.0f, 0.0f), o = m;
      if constexpr (MOM) m = *reinterpret_cast<const float4*>(mi + i);
      one(u.x, m.x, o.x);
      one(u.y, m.y, o.y);
      one(u.z, m.z, o.z);
      one(u.w, m.w, o.w);
      if constexpr (MOM) *reinterpret_cast<float4*>(mo + i) = o;
    }
  } else {
    for (int64_t i = e0 + threadIdx.x; i < e1; i += 256) {
      float o = 0.0f;
      one(load_grad(g + i), MOM ? mi[i] : 0.0f, o);
      if constexpr (MOM) mo[i] = o;
    }
  }
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) s += __shfl_xor(s, k, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0)
    reinterpret_cast<double*>(a.ws + mat * a.o.bytes + a.o.part)[blockIdx.x] =
        ((red[0] + red[1]) + red[2]) + red[3];
}

// v as a finished fp32 value. Without this the compiler may fold the product
// behind v into the conversion of one use of hi (one rounding) and not of the
// other (two), and in one element of some ten thousand the two differ.
__device__ __forceinline__ float rounded(float v) {
  asm("" : "+v"(v));
  return v;
}
__device__ __forceinline__ void split_x(float v, _Float16& hi, _Float16& lo) {
  v = rounded(v);
  hi = static_cast<_Float16>(v);
  lo = static_cast<_Float16>((v - static_cast<float>(hi)) * kScaleLo);
}

// X_0 = u / (|u| + eps) into the planes, 64 x 64 elements per block
// (transposed through LDS where rows > cols), padding columns zero.
// Bound by memory: the same matrices in 535 us, 5.3 TB/s. u is computed again
// rather than kept in fp32, which would move as much.
template <class T, bool MOM, bool TALL>
__global__ __launch_bounds__(256) void orth_scale_kernel(PrepArgs a) {
  __shared__ float tile[TALL ? 64 : 1][65];
  __shared__ double red[4];
  __shared__ float scale_s;
  const int64_t el = int64_t(a.rows) * a.cols, mat = blockIdx.z;
  char* ws = a.ws + mat * a.o.bytes;
  const double* part = reinterpret_cast<const double*>(ws + a.o.part);
  double s = static_cast<int>(threadIdx.x) < a.o.chunks ? part[threadIdx.x] : 0.0;
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) s += __shfl_xor(s, k, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0)
    scale_s = static_cast<float>(kScaleX / (sqrt(((red[0] + red[1]) + red[2]) + red[3]) + kNormEps));
  __syncthreads();
  const float scale = scale_s;
  const T* g = static_cast<const T*>(a.grad) + mat * el;
  const float* mo = MOM ? a.m_out + mat * el : nullptr;
  auto u_at = [&](int64_t i) {
    const float u = load_grad(g + i);
    if constexpr (MOM) return a.nesterov ? u + a.momentum * mo[i] : mo[i];
    return u;
  };
  _Float16* hi = reinterpret_cast<_Float16*>(ws + a.o.hi0);
  _Float16* lo = reinterpret_cast<_Float16*>(ws + a.o.lo);
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;  // of X
  if (!TALL && a.o.m % 4 == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = r0 + k * 16 + (threadIdx.x >> 4), c = c0 + (threadIdx.x & 15) * 4;
      if (r >= a.o.n) continue;  // c < mp: blocks cover whole k-steps
      float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (c < a.o.m) {
        const int64_t i = int64_t(r) * a.cols + c;
        u = load_grad4(g + i);
        if constexpr (MOM) {
          const float4 m = *reinterpret_cast<const float4*>(mo + i);
          u = a.nesterov ? make_float4(u.x + a.momentum * m.x, u.y + a.momentum * m.y,
                                       u.z + a.momentum * m.z, u.w + a.momentum * m.w)
                         : m;
        }
      }
      f16x4_t h, l;
      _Float16 hh, ll;
      split_x(u.x * scale, hh, ll);
      h[0] = hh, l[0] = ll;
      split_x(u.y * scale, hh, ll);
      h[1] = hh, l[1] = ll;
      split_x(u.z * scale, hh, ll);
      h[2] = hh, l[2] = ll;
      split_x(u.w * scale, hh, ll);
      h[3] = hh, l[3] = ll;
      *reinterpret_cast<f16x4_t*>(hi + int64_t(r) * a.o.mp + c) = h;
      *reinterpret_cast<f16x4_t*>(lo + int64_t(r) * a.o.mp + c) = l;
    }
    return;
  }
  if constexpr (TALL) {
    for (int i = ty; i < 64; i += 4) {  // row c0 + i of u, columns r0 ..
      const int ur = c0 + i, uc = r0 + tx;
      tile[i][tx] = (ur < a.rows && uc < a.cols) ? u_at(int64_t(ur) * a.cols + uc) : 0.0f;
    }
    __syncthreads();
  }
  for (int i = ty; i < 64; i += 4) {
    const int r = r0 + i, c = c0 + tx;
    if (r >= a.o.n || c >= a.o.mp) continue;
    float v;
    if constexpr (TALL)
      v = tile[tx][i];
    else
      v = c < a.o.m ? u_at(int64_t(r) * a.cols + c) : 0.0f;
    _Float16 h, l;
    split_x(v * scale, h, l);
    hi[int64_t(r) * a.o.mp + c] = h;
    lo[int64_t(r) * a.o.mp + c] = l;
  }
}

// ---- the three products of a step ------------------------------------------------
//
// 16 matrices of 2048 x 7168: R 528 us (0.54 TFLOP of lower tiles, 1.02
// PFLOP/s), S 217 us, X 1133 us (0.96 TFLOP, 0.85 PFLOP/s), the last X 1036 us.
// The matrix cores bound the loops; X's output adds to them, as it reads and
// writes both planes (256 KB each way per tile of 256 x 256, 16 us at the rates
// of one CU) and a CU has no second workgroup to multiply meanwhile.

enum Kind { kGram = 0, kSquare = 1, kApply = 2, kApplyLast = 3 };

struct StepArgs {
  char* ws;
  OrthShape o;
  size_t hi_in, hi_out;  // planes of X read and written
  void* out;             // last step: bf16 [rows, cols]
  int64_t mats;
  Tail tail;
  float low_q;           // 1: Q multiplies the low plane too (last two steps), else 0
};

// Lower-triangular tile p (row by row) of a symmetric product.
__device__ __forceinline__ void triangle(int p, int& i, int& j) {
  i = static_cast<int>((sqrtf(8.0f * p + 1.0f) - 1.0f) * 0.5f);
  while (i * (i + 1) / 2 > p) --i;
  while ((i + 1) * (i + 2) / 2 <= p) ++i;
  j = p - i * (i + 1) / 2;
}

struct OTile {
  int64_t mat;
  int m, n;
};

template <class C, int KIND>
__device__ __forceinline__ OTile orth_tile(const StepArgs& a, int tile) {
  const int tm = (a.o.n + C::BM - 1) / C::BM;
  OTile t;
  if constexpr (KIND == kGram || KIND == kSquare) {
    static_assert(C::BM == C::BN, "square tiles on the diagonal");
    const int per = tm * (tm + 1) / 2;
    t.mat = tile / per;
    triangle(tile - static_cast<int>(t.mat) * per, t.m, t.n);
  } else {
    const int tn = (a.o.m + C::BN - 1) / C::BN, per = tm * tn;
    t.mat = tile / per;
    const int r = tile - static_cast<int>(t.mat) * per;
    t.n = r / tm;  // m fastest: the row tiles that share columns of X run together
    t.m = r - t.n * tm;
  }
  return t;
}

// Only the Gram product is long enough to share tiles (without the code for it
// the others run 5% faster).
template <int KIND>
__device__ __forceinline__ Unit unit_at(const StepArgs& a, int unit) {
  if constexpr (KIND == kGram)
    return unit_of(a.tail, unit);
  else
    return {unit, 0, 1};
}

template <class C, int KIND, bool TALL, bool PHASED>
__global__ __launch_bounds__(C::NT, C::MINW) void orth_product_kernel(StepArgs a, int total) {
  constexpr bool BKM = KIND >= kApply;
  constexpr int kStageElems = PHASED ? 0 : C::NWAVES * RowPasses<C>::FLOATS * 2;
  __shared__ __attribute__((aligned(16))) uint16_t lds[C::LDS_ELEMS + kStageElems];
  __shared__ int flag;
  const int first = xcd_logical_block(blockIdx.x, gridDim.x);
  if (first >= total) return;
  const int nk = (KIND == kGram ? a.o.mp : a.o.np) / BK;
  auto next_ops = [&](int unit, Ops16<C>& op) {
    const Unit u = unit_at<KIND>(a, unit);
    const KRange kr = split_range(nk, u.s, u.splits);
    const OTile t = orth_tile<C, KIND>(a, u.tile);
    const char* ws = a.ws + t.mat * a.o.bytes;
    const uint32_t ldx = a.o.mp * 2, lds_ = a.o.np * 2;
    const int left = min(a.o.n - t.m * C::BM, C::BM);
    op.nk = kr.k1 - kr.k0;
    const int K = op.nk * BK;
    const char* A =
        ws + (KIND == kGram ? a.hi_in : KIND == kSquare ? a.o.r : a.o.s) + int64_t(kr.k0) * BK * 2;
    const uint32_t lda = KIND == kGram ? ldx : lds_;
    // rows end with the split's last k-step: the bytes after it are not read
    const int64_t cut = lda - int64_t(K) * 2;
    kcontig_operand<C>(op.ra, op.ao, op.tail_a, A + int64_t(t.m) * C::BM * lda, left, lda,
                       int64_t(left) * lda - cut, K);
    if constexpr (BKM) {
      const int64_t k0 = int64_t(kr.k0) * BK;
      kmajor_operand<C, C::BN>(op.rb, op.bo, op.base_b, op.left_b, op.step_b,
                               ws + a.hi_in + k0 * ldx, t.n * C::BN, ldx, (a.o.n - k0) * ldx);
    } else {
      const int nleft = min(a.o.n - t.n * C::BN, C::BN);
      kcontig_operand<C>(op.rb, op.bo, op.tail_b, A + int64_t(t.n) * C::BN * lda, nleft, lda,
                         int64_t(nleft) * lda - cut, K);
    }
  };
  struct Epilogue {
    const StepArgs& a;
    int nk;
    int* flag;
    __device__ int k_steps(int unit) const {
      const Unit u = unit_at<KIND>(a, unit);
      const KRange r = split_range(nk, u.s, u.splits);
      return r.k1 - r.k0;
    }
    __device__ void operator()(int unit, int wm, int wn, int lane, f32x16_t (&acc)[C::MI][C::NJ],
                               float* stage) const {
      using P = std::conditional_t<PHASED, StagePasses<C>, RowPasses<C>>;
      static_assert(P::PARTS == 1, "a wave's columns together");
      const Unit u = unit_at<KIND>(a, unit);
      if constexpr (KIND == kGram) {
        if (!join_splits<C>(acc, a.tail, unit, u, flag)) return;
      }
      const OTile t = orth_tile<C, KIND>(a, u.tile);
      char* ws = a.ws + t.mat * a.o.bytes;
      const int n = a.o.n, np = a.o.np, mp = a.o.mp, m = a.o.m;
      const int row0 = t.m * C::BM + wm * C::WM, col0 = t.n * C::BN + wn * C::WN;
      const int col = col0 + P::col(lane);
      float* D = reinterpret_cast<float*>(ws + a.o.d);
      float* Q = reinterpret_cast<float*>(ws + a.o.q);
      const _Float16* R = reinterpret_cast<const _Float16*>(ws + a.o.r);
      if constexpr (KIND == kGram || KIND == kSquare) {
        _Float16* dst = reinterpret_cast<_Float16*>(ws + (KIND == kGram ? a.o.r : a.o.s));
        const int cc = min(col, np - 8);
        f32x4_t dj[2] = {};
        if constexpr (KIND == kSquare) {
          dj[0] = *reinterpret_cast<const f32x4_t*>(D + cc);
          dj[1] = *reinterpret_cast<const f32x4_t*>(D + cc + 4);
        }
#pragma unroll
        for (int mi = 0; mi < C::MI; ++mi) {
          f16x8_t r8[P::N];
          float di[P::N];
          if constexpr (KIND == kSquare) {
#pragma unroll
            for (int p = 0; p < P::N; ++p) {
              const int row = min(row0 + mi * 32 + P::row(p, lane), n - 1);
              r8[p] = *reinterpret_cast<const f16x8_t*>(R + int64_t(row) * np + cc);
              di[p] = D[row];
            }
          }
          P::put(stage, lane, acc[mi]);
          f16x8_t o[P::N];
#pragma unroll
          for (int p = 0; p < P::N; ++p) {
            const int row = row0 + mi * 32 + P::row(p, lane);
            float v[8];
            P::get(stage, lane, p, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const bool diag = col + j == row;
              if constexpr (KIND == kGram) {
                if (diag && row < n) D[row] = v[j] * (1.0f / (kScaleX * kScaleX));
                v[j] *= kScaleR / (kScaleX * kScaleX);
              } else {
                const float rij = static_cast<float>(r8[p][j]);
                const float rr = v[j] * (1.0f / (kScaleR * kScaleR));
                if (diag && row < n) Q[row] = kB * di[p] + kC * (rr + di[p] * di[p]);
                v[j] = kScaleS * kC * rr +
                       rij * (kScaleS / kScaleR * (kB + kC * (di[p] + dj[j >> 2][j & 3])));
              }
              // rows past n only put zeros into the mirrored tile's padding
              o[p][j] = static_cast<_Float16>(diag || row >= n ? 0.0f : v[j]);
            }
          }
#pragma unroll
          for (int p = 0; p < P::N; ++p) {
            const int row = row0 + mi * 32 + P::row(p, lane);
            if (row < n && col < np) *reinterpret_cast<f16x8_t*>(dst + int64_t(row) * np + col) = o[p];
          }
          if (t.m != t.n) {
            // The mirrored tile: these 32 rows go back to LDS in fp16 (pitch
            // 144 bytes, so that four rows fall on distinct banks) and return
            // transposed, 8 of them for one column per lane.
            constexpr int kPitch = C::WN + 8;
            static_assert(32 * kPitch * 2 <= P::FLOATS * 4, "fits the wave's stage");
            _Float16* tile = reinterpret_cast<_Float16*>(stage);
#pragma unroll
            for (int p = 0; p < P::N; ++p)
              *reinterpret_cast<f16x8_t*>(tile + P::row(p, lane) * kPitch + P::col(lane)) = o[p];
            const int gr = lane >> 4, kj = (lane >> 2) & 3, cq = lane & 3;
#pragma unroll
            for (int c0 = 0; c0 < C::WN; c0 += 32)
#pragma unroll
              for (int k0 = 0; k0 < 32; k0 += 16) {
                const _Float16* src =
                    tile + (k0 + 8 * (gr >> 1) + kj) * kPitch + c0 + 16 * (gr & 1) + 4 * cq;
                const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_i16x4_t*)(uintptr_t)lds_addr(src));
                const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_i16x4_t*)(uintptr_t)lds_addr(src + 4 * kPitch));
                typedef short i16x8_t __attribute__((ext_vector_type(8)));
                const i16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                const int row = col0 + c0 + (lane & 31), c = row0 + mi * 32 + k0 + 8 * (lane >> 5);
                if (row < n && c < np) *reinterpret_cast<i16x8_t*>(dst + int64_t(row) * np + c) = v;
              }
          }
        }
      } else {
        // A wave's memory operations complete in order, so a load issued after a
        // store waits for it: rows are loaded kAhead passes ahead, before the
        // store of the pass in hand.
        constexpr int kPasses = C::MI * P::N, kAhead = 4;
        f16x8_t h[kAhead], l[kAhead];
        const int cc = col < mp ? col : 0;
        auto fetch = [&](int i) {
          const int row = min(row0 + i / P::N * 32 + P::row(i % P::N, lane), n - 1);
          const int64_t at = (int64_t(row) * mp + cc) * 2;
          h[i % kAhead] = *reinterpret_cast<const f16x8_t*>(ws + a.hi_in + at);
          l[i % kAhead] = *reinterpret_cast<const f16x8_t*>(ws + a.o.lo + at);
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(i);
        uint16_t* out = static_cast<uint16_t*>(a.out) + t.mat * n * int64_t(m);
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int mi = i / P::N, p = i % P::N;
          if (p == 0) P::put(stage, lane, acc[mi]);
          float x[8];
          P::get(stage, lane, p, x);
          const int row = row0 + mi * 32 + P::row(p, lane);
          const float q = Q[min(row, n - 1)];
          const float fh = kA + q, fl = (kA + a.low_q * q) * (1.0f / kScaleLo);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            x[j] = fh * static_cast<float>(h[i % kAhead][j]) +
                   fl * static_cast<float>(l[i % kAhead][j]) + x[j] * (1.0f / kScaleS);
          u32x4_t oh, ol;
          if constexpr (KIND == kApply) {
            f16x8_t hh, ll;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              _Float16 hi, lo;
              split_x(x[j], hi, lo);
              hh[j] = hi;
              ll[j] = lo;
            }
            oh = __builtin_bit_cast(u32x4_t, hh);
            ol = __builtin_bit_cast(u32x4_t, ll);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              oh[j] = pack_bf16x2(x[2 * j] * (1.0f / kScaleX), x[2 * j + 1] * (1.0f / kScaleX));
          }
          __builtin_amdgcn_sched_barrier(0);
          if (i + kAhead < kPasses) fetch(i + kAhead);
          __builtin_amdgcn_sched_barrier(0);
          if (row < n && col < mp) {
            if constexpr (KIND == kApply) {
              const int64_t at = (int64_t(row) * mp + col) * 2;
              *reinterpret_cast<u32x4_t*>(ws + a.hi_out + at) = oh;
              *reinterpret_cast<u32x4_t*>(ws + a.o.lo + at) = ol;
            } else if (!TALL && m % 8 == 0) {
              if (col < m) *reinterpret_cast<u32x4_t*>(out + int64_t(row) * m + col) = oh;
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (col + j < m)
                  out[TALL ? int64_t(col + j) * n + row : int64_t(row) * m + col + j] =
                      static_cast<uint16_t>(oh[j >> 1] >> (16 * (j & 1)));
            }
          }
        }
      }
    }
  } ep{a, nk, &flag};
  if constexpr (PHASED)
    stream_phased<C, TypeF16, false, BKM, true>(lds, first, gridDim.x, total, next_ops, ep);
  else
    stream_ring<C, TypeF16, false, BKM, true>(lds, first, gridDim.x, total, next_ops, ep);
}

// ---- small matrices ---------------------------------------------------------------

// One workgroup per matrix of up to 128 x 256, all steps in one launch: X stays
// in fp32 registers (the master) and as fp16 in LDS (the operand), the n x n
// matrices share one LDS buffer. Launch-bound otherwise: 17 launches a call
// took 233 us for 32 matrices of 128 x 256, this kernel 40: 15 dependent
// products of one workgroup, each bound by its LDS reads and barriers. (The
// tall form without momentum has 36 bytes a lane in scratch memory: 39 us for
// the same matrices transposed.)
//
// X [128][256] serves row reads (16-byte fragments of 16 rows at a time, for X
// X^T) and transpose reads (4 rows of 32 bytes, for S X), so its 16-byte chunks
// are XOR-swizzled with 2 (r & 7) + (r >> 3 & 1): 16 distinct values over 16
// rows, and distinct pairs of chunks over 4 rows.
constexpr int kSmallN = 128, kSmallM = 256;

struct SmallArgs {
  const void* grad;
  const float* m_in;
  float* m_out;
  uint16_t* out;
  int rows, cols, n, m, steps;
  float momentum;
  int nesterov;
};

__device__ __forceinline__ int x_off(int r, int c) {  // elements, c a multiple of 4
  const int f = ((r & 7) << 1) | ((r >> 3) & 1);
  return r * kSmallM + (((c >> 3) ^ f) << 3) + (c & 7);
}
__device__ __forceinline__ int r_off(int r, int c) {
  return r * kSmallN + (((c >> 3) ^ (r & 15)) << 3) + (c & 7);
}

template <class T, bool MOM, bool TALL>
__global__ __launch_bounds__(512, 2) void orth_small_kernel(SmallArgs a) {
  __shared__ __attribute__((aligned(16))) _Float16 X[kSmallN * kSmallM];
  __shared__ __attribute__((aligned(16))) _Float16 R[kSmallN * kSmallN];
  __shared__ __attribute__((aligned(16))) float D[kSmallN];
  __shared__ float Q[kSmallN];
  __shared__ double red[8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 2, wn = wave & 3, half = lane >> 5;
  const int64_t el = int64_t(a.rows) * a.cols, mat = blockIdx.x;
  const T* g = static_cast<const T*>(a.grad) + mat * el;

  // This wave's 64 x 64 of X: lane row, runs of four columns. All loads go out
  // before the first use: addresses past the matrix are clamped into it and
  // their values dropped, so no load hides behind a branch. (With one branch
  // per element the loads ran one after the other: 71 us for a call of 32
  // matrices of 128 x 256 that takes 40.)
  f32x16_t x[2][2];
  const bool runs = !TALL && a.m % 4 == 0;  // whole runs of four, aligned
  auto at = [&](int mi, int nj, int e) {
    const int r = min(wm * 64 + mi * 32 + (lane & 31), a.n - 1);
    const int c = min(wn * 64 + nj * 32 + 8 * (e >> 2) + 4 * half + (e & 3), a.m - 1);
    return TALL ? int64_t(c) * a.cols + r : int64_t(r) * a.cols + c;
  };
  auto inside = [&](int mi, int nj, int e) {
    return wm * 64 + mi * 32 + (lane & 31) < a.n &&
           wn * 64 + nj * 32 + 8 * (e >> 2) + 4 * half + (e & 3) < a.m;
  };
  auto fetch = [&](auto* src, f32x16_t (&v)[2][2]) {
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
      for (int nj = 0; nj < 2; ++nj) {
        if (runs) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            // a run past the last column starts on the last one
            const int c = min(wn * 64 + nj * 32 + 8 * q + 4 * half, a.m - 4);
            const int r = min(wm * 64 + mi * 32 + (lane & 31), a.n - 1);
            const float4 w = load_grad4(src + int64_t(r) * a.cols + c);
            v[mi][nj][4 * q] = w.x;
            v[mi][nj][4 * q + 1] = w.y;
            v[mi][nj][4 * q + 2] = w.z;
            v[mi][nj][4 * q + 3] = w.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[mi][nj][e] = load_grad(src + at(mi, nj, e));
        }
      }
  };
  fetch(g, x);
  f32x16_t mom[2][2];
  if constexpr (MOM) fetch(a.m_in + mat * el, mom);
  double sum = 0.0;
#pragma unroll
  for (int mi = 0; mi < 2; ++mi)
#pragma unroll
    for (int nj = 0; nj < 2; ++nj)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float u = x[mi][nj][e];
        if constexpr (MOM) {
          const float mo = a.momentum * mom[mi][nj][e] + u;
          mom[mi][nj][e] = mo;
          u = a.nesterov ? u + a.momentum * mo : mo;
        }
        u = inside(mi, nj, e) ? u : 0.0f;
        x[mi][nj][e] = u;
        sum += double(u) * u;
      }
  if constexpr (MOM) {
    // m_out may be m_in: every value is stored by the lane that read it, and
    // clamped reads take values of this lane's row or a neighbour's that no
    // inside element uses
    __syncthreads();
    float* mo = a.m_out + mat * el;
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
      for (int nj = 0; nj < 2; ++nj)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (runs) {
            if (inside(mi, nj, 4 * q))
              *reinterpret_cast<float4*>(mo + at(mi, nj, 4 * q)) =
                  make_float4(mom[mi][nj][4 * q], mom[mi][nj][4 * q + 1], mom[mi][nj][4 * q + 2],
                              mom[mi][nj][4 * q + 3]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (inside(mi, nj, 4 * q + j)) mo[at(mi, nj, 4 * q + j)] = mom[mi][nj][4 * q + j];
          }
        }
  }
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) sum += __shfl_xor(sum, k, 64);
  if (lane == 0) red[wave] = sum;
  __syncthreads();
  sum = red[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) sum += red[w];
  const float scale = static_cast<float>(kScaleX / (sqrt(sum) + kNormEps));

  auto store_x = [&]() {
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
      for (int nj = 0; nj < 2; ++nj)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = wm * 64 + mi * 32 + (lane & 31);
          const int c = wn * 64 + nj * 32 + 8 * q + 4 * half;
          f16x4_t h;
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = static_cast<_Float16>(rounded(x[mi][nj][4 * q + j]));
          *reinterpret_cast<f16x4_t*>(X + x_off(r, c)) = h;
        }
  };
  // fragments: 32 rows of X or R from r0, k columns 16 kk ..; columns c0 .. of
  // X over rows 16 kk .. (transpose reads)
  auto x_rows = [&](int r0, int kk) {
    return *reinterpret_cast<const bf16x8_t*>(X + x_off(r0 + (lane & 31), kk * 16 + 8 * half));
  };
  auto r_rows = [&](int r0, int kk) {
    return *reinterpret_cast<const bf16x8_t*>(R + r_off(r0 + (lane & 31), kk * 16 + 8 * half));
  };
  auto x_cols = [&](int c0, int kk) {
    const int gr = lane >> 4, j = (lane >> 2) & 3, q = lane & 3;
    const int c = c0 + 16 * (gr & 1) + 4 * q, k = kk * 16 + 8 * (gr >> 1) + j;
    const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_i16x4_t*)(uintptr_t)lds_addr(X + x_off(k, c)));
    const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_i16x4_t*)(uintptr_t)lds_addr(X + x_off(k + 4, c)));
    typedef short i16x8_t __attribute__((ext_vector_type(8)));
    const i16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8_t, v);
  };

#pragma unroll
  for (int mi = 0; mi < 2; ++mi)
#pragma unroll
    for (int nj = 0; nj < 2; ++nj)
#pragma unroll
      for (int e = 0; e < 16; ++e) x[mi][nj][e] *= scale;
  store_x();
  __syncthreads();

  // steps past the matrix's own rows and columns would multiply zeros
  const int nk = (a.n + 15) / 16, mk = (a.m + 15) / 16;
  for (int step = 0; step < a.steps; ++step) {
    const f32x16_t zero = {};
    // A = X X^T, this wave's 64 x 32
    f32x16_t r[2];
    {
      const bf16x8_t b = x_rows(wn * 32, 0);
#pragma unroll
      for (int mi = 0; mi < 2; ++mi)
        r[mi] = mma16<TypeF16, true>(x_rows(wm * 64 + mi * 32, 0), b, zero);
    }
#pragma unroll 5
    for (int kk = 1; kk < mk; ++kk) {
      const bf16x8_t b = x_rows(wn * 32, kk);
#pragma unroll
      for (int mi = 0; mi < 2; ++mi)
        r[mi] = mma16<TypeF16, true>(x_rows(wm * 64 + mi * 32, kk), b, r[mi]);
    }
    // v times s into R; only the wave's 32 x 32 block on the diagonal has
    // entries to keep apart
    auto put_r = [&](f32x16_t (&v)[2], float s, float* diag, float sd) {
#pragma unroll
      for (int mi = 0; mi < 2; ++mi) {
        const int row = wm * 64 + mi * 32 + (lane & 31);
        if (wm * 2 + mi == wn) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (8 * (e >> 2) + 4 * half + (e & 3) == (lane & 31)) {
              diag[row] = v[mi][e] * sd;
              v[mi][e] = 0.0f;
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f16x4_t h;
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = static_cast<_Float16>(v[mi][4 * q + j] * s);
          *reinterpret_cast<f16x4_t*>(R + r_off(row, wn * 32 + 8 * q + 4 * half)) = h;
        }
      }
    };
    constexpr float kUnitX = 1.0f / (kScaleX * kScaleX);  // r times this: A
    put_r(r, kScaleR * kUnitX, D, kUnitX);
    __syncthreads();
    // B = b A + c A A, diagonal apart: off it c (R R)_ij + R_ij (b + c (D_i +
    // D_j)), on it b D_i + c ((R R)_ii + D_i^2)
    f32x16_t p[2];
    {
      const bf16x8_t b = r_rows(wn * 32, 0);
#pragma unroll
      for (int mi = 0; mi < 2; ++mi)
        p[mi] = mma16<TypeF16, true>(r_rows(wm * 64 + mi * 32, 0), b, zero);
    }
#pragma unroll 7
    for (int kk = 1; kk < nk; ++kk) {
      const bf16x8_t b = r_rows(wn * 32, kk);
#pragma unroll
      for (int mi = 0; mi < 2; ++mi)
        p[mi] = mma16<TypeF16, true>(r_rows(wm * 64 + mi * 32, kk), b, p[mi]);
    }
#pragma unroll
    for (int mi = 0; mi < 2; ++mi) {
      const int row = wm * 64 + mi * 32 + (lane & 31);
      const float di = D[row], ti = kUnitX * (kB + kC * di);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4_t dj = *reinterpret_cast<const f32x4_t*>(D + wn * 32 + 8 * q + 4 * half);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 4 * q + j;
          p[mi][e] = p[mi][e] * (kC / (kScaleR * kScaleR)) +
                     r[mi][e] * (ti + (kUnitX * kC) * dj[j]);
        }
      }
      if (wm * 2 + mi == wn) {  // r is zero on the diagonal: the rest of its terms
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (8 * (e >> 2) + 4 * half + (e & 3) == (lane & 31))
            p[mi][e] += di * (kB + kC * di);
      }
    }
    __syncthreads();  // every wave has read R
    put_r(p, kScaleS, Q, 1.0f);
    __syncthreads();
    // X <- (a + Q) X + S X
    f32x16_t y[2][2];
    auto step_y = [&](int kk, bool first) {
      bf16x8_t b[2];
#pragma unroll
      for (int nj = 0; nj < 2; ++nj) b[nj] = x_cols(wn * 64 + nj * 32, kk);
#pragma unroll
      for (int mi = 0; mi < 2; ++mi) {
        const bf16x8_t s = r_rows(wm * 64 + mi * 32, kk);
#pragma unroll
        for (int nj = 0; nj < 2; ++nj)
          y[mi][nj] = mma16<TypeF16, true>(s, b[nj], first ? zero : y[mi][nj]);
      }
    };
    step_y(0, true);
#pragma unroll 3
    for (int kk = 1; kk < nk; ++kk) step_y(kk, false);
    const bool low_q = step + 2 >= a.steps;  // Q multiplies all of X, else its fp16 part
#pragma unroll
    for (int mi = 0; mi < 2; ++mi) {
      const float q = Q[wm * 64 + mi * 32 + (lane & 31)];
#pragma unroll
      for (int nj = 0; nj < 2; ++nj)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float v = rounded(x[mi][nj][e]);
          const float w = low_q ? v : static_cast<float>(static_cast<_Float16>(v));
          x[mi][nj][e] = kA * v + (q * w + y[mi][nj][e] * (1.0f / kScaleS));
        }
    }
    __syncthreads();  // every wave has read X and S
    if (step + 1 < a.steps) {
      store_x();
      __syncthreads();
    }
  }
  uint16_t* out = a.out + mat * el;
#pragma unroll
  for (int mi = 0; mi < 2; ++mi)
#pragma unroll
    for (int nj = 0; nj < 2; ++nj) {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[mi][nj][e] *= 1.0f / kScaleX;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16_t& v = x[mi][nj];
        if (runs) {
          if (inside(mi, nj, 4 * q))
            *reinterpret_cast<uint2*>(out + at(mi, nj, 4 * q)) =
                pack_bf16x4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (inside(mi, nj, 4 * q + j)) out[at(mi, nj, 4 * q + j)] = f32_to_bf16(v[4 * q + j]);
        }
      }
    }
}

template <class T, bool MOM>
void small(const SmallArgs& a, bool tall, int64_t mats, hipStream_t s) {
  const dim3 g(static_cast<unsigned>(mats));
  if (tall)
    hipLaunchKernelGGL((orth_small_kernel<T, MOM, true>), g, dim3(512), 0, s, a);
  else
    hipLaunchKernelGGL((orth_small_kernel<T, MOM, false>), g, dim3(512), 0, s, a);
}

// ---- launches ------------------------------------------------------------------------

using TileBig = Tile<256, 256, 128, 64, 2>;  // 8 waves, two-phase loop
using TileMid = Tile<128, 128, 64, 32, 3>;   // 8 waves, ring

// Tiles of a product and how its last round is shared. Big tiles run at the
// higher rate, small ones fill the GPU: the one with the lesser modelled time,
// rounds of 256 tiles at the measured times per k-step (256 x 256: 1.4 us with
// the GPU full, 1.05 us half full; 128 x 128: 0.65 and 0.38) and per tile (8 and
// 4 us).
struct Plan {
  bool big;
  int tiles, whole, splits;
  size_t bytes() const {  // of partial tiles
    return splits > 1 ? size_t(tiles - whole) * splits * (big ? 256 * 256 : 128 * 128) * 4 : 0;
  }
};
Plan plan(const OrthShape& o, int64_t mats, int kind) {
  const int nk = (kind == kGram ? o.mp : o.np) / BK;
  Plan best{};
  double least = 0.0;
  for (int big = 0; big < 2; ++big) {
    const int b = big ? 256 : 128;
    const int64_t tm = (o.n + b - 1) / b, tn = (o.m + b - 1) / b;
    Plan p{};
    p.big = big;
    p.tiles = static_cast<int>(mats * (kind < kApply ? tm * (tm + 1) / 2 : tm * tn));
    p.whole = p.tiles / kSlots * kSlots;
    const float busy = big ? 1.4f : 0.65f, kb = b * b / 256;
    p.splits = kind == kGram ? tail_splits(p.tiles - p.whole, nk, kSlots, busy, kb) : 1;
    if (p.splits == 1) p.whole = p.tiles;
    const double step = p.tiles * p.splits <= kSlots / 2 ? (big ? 1.05 : 0.38) : busy;
    const double fixed = big ? 8.0 : 4.0;
    double us = (p.whole + kSlots - 1) / kSlots * (nk * step + fixed);
    if (p.splits > 1)
      us += (nk + p.splits - 1) / p.splits * step + fixed + kb / 22.0 + p.splits * kb / 30.0;
    if (big == 0 || us <= least) {
      best = p;
      least = us;
    }
  }
  return best;
}

template <class C, int KIND, bool TALL, bool PHASED>
void launch_product(const StepArgs& a, const Plan& p, hipStream_t s) {
  const int units = p.whole + (p.tiles - p.whole) * p.splits;
  hipLaunchKernelGGL((orth_product_kernel<C, KIND, TALL, PHASED>),
                     dim3(grid_of<orth_product_kernel<C, KIND, TALL, PHASED>>(C::NT, units)),
                     dim3(C::NT), 0, s, a, units);
}

template <int KIND, bool TALL>
void product(StepArgs a, hipStream_t s) {
  const Plan p = plan(a.o, a.mats, KIND);
  a.tail.whole = p.whole;
  a.tail.splits = p.splits;
  if (p.big)
    launch_product<TileBig, KIND, TALL, true>(a, p, s);
  else
    launch_product<TileMid, KIND, TALL, false>(a, p, s);
}

// Partial tiles and counters behind the matrices' workspaces.
size_t tail_part_bytes(const OrthShape& o, int64_t mats) {
  return plan(o, mats, kGram).bytes();
}

void steps(StepArgs a, const OrthArgs& p, hipStream_t s) {
  for (int i = 0; i < p.steps; ++i) {
    a.hi_in = i & 1 ? a.o.hi1 : a.o.hi0;
    a.hi_out = i & 1 ? a.o.hi0 : a.o.hi1;
    a.low_q = i + 2 >= p.steps ? 1.0f : 0.0f;
    product<kGram, false>(a, s);
    product<kSquare, false>(a, s);
    if (i + 1 < p.steps)
      product<kApply, false>(a, s);
    else if (a.o.tall)
      product<kApplyLast, true>(a, s);
    else
      product<kApplyLast, false>(a, s);
  }
}

template <class T, bool MOM>
void prepare(const PrepArgs& a, int64_t mats, hipStream_t s) {
  hipLaunchKernelGGL((orth_sum_kernel<T, MOM>), dim3(a.o.chunks, static_cast<unsigned>(mats)),
                     dim3(256), 0, s, a);
  const dim3 g((a.o.mp + 63) / 64, (a.o.n + 63) / 64, static_cast<unsigned>(mats));
  if (a.o.tall)
    hipLaunchKernelGGL((orth_scale_kernel<T, MOM, true>), g, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((orth_scale_kernel<T, MOM, false>), g, dim3(256), 0, s, a);
}

}  // namespace

size_t orth_workspace(int64_t mats, int rows, int cols) {
  const OrthShape o = shape_of(rows, cols);
  if (o.n <= kSmallN && o.m <= kSmallM) return 0;
  return static_cast<size_t>(mats) * o.bytes + kSlots * sizeof(int32_t) + tail_part_bytes(o, mats);
}

hipError_t launch_orth(const OrthArgs& p, hipStream_t s) {
  if (p.mats == 0) return hipSuccess;
  const OrthShape o = shape_of(p.rows, p.cols);
  if (o.n <= kSmallN && o.m <= kSmallM) {
    const SmallArgs a{p.grad, p.m_in, p.m_out, static_cast<uint16_t*>(p.out), p.rows, p.cols, o.n,
                      o.m, p.steps, p.momentum, p.nesterov};
    if (p.bf16)
      p.m_in ? small<uint16_t, true>(a, o.tall, p.mats, s)
             : small<uint16_t, false>(a, o.tall, p.mats, s);
    else
      p.m_in ? small<float, true>(a, o.tall, p.mats, s) : small<float, false>(a, o.tall, p.mats, s);
    return hipGetLastError();
  }
  PrepArgs a{};
  a.grad = p.grad;
  a.m_in = p.m_in;
  a.m_out = p.m_out;
  a.ws = static_cast<char*>(p.ws);
  a.count = reinterpret_cast<int32_t*>(a.ws + p.mats * o.bytes);
  a.o = o;
  a.rows = p.rows;
  a.cols = p.cols;
  a.momentum = p.momentum;
  a.nesterov = p.nesterov;
  if (p.bf16)
    p.m_in ? prepare<uint16_t, true>(a, p.mats, s) : prepare<uint16_t, false>(a, p.mats, s);
  else
    p.m_in ? prepare<float, true>(a, p.mats, s) : prepare<float, false>(a, p.mats, s);
  StepArgs st{};
  st.ws = a.ws;
  st.o = a.o;
  st.out = p.out;
  st.mats = p.mats;
  st.tail.count = reinterpret_cast<int32_t*>(st.ws + p.mats * o.bytes);
  st.tail.part = reinterpret_cast<float*>(st.tail.count + kSlots);
  steps(st, p, s);
  return hipGetLastError();
}

}  // namespace dsmoe
