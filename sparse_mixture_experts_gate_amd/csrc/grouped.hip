// Matrix products grouped by expert over ragged row groups (definitions in
// dsmoe_ops.h): forward y = x W_g^T, input gradient dx = dy W_g, weight
// gradient dw_g = dy_g^T x_g. bf16 operands, fp32 accumulation.
//
// One launch per call: every workgroup builds the groups' tile table from the
// device offsets itself, so no planning kernel runs first.
#include <cmath>

#include "device_common.h"
#include "gemm16_core.h"
#include "internal.h"
#include "resident_grid.h"
#include "tile_schedule.h"

namespace dsmoe {

namespace {

constexpr float kBigStep = 1.4f;  // us per k-step of 256 x 256 tiles, operands from L2

enum Mode { kForward = 0, kDgrad = 1, kWgrad = 2 };

// Operands by mode (C[M, N] = A B, contraction K):
//   forward  A = x rows, B = W_g rows (both k-contiguous);  M = rows of g
//   dgrad    A = dy rows (k-contiguous), B = W_g (k-major); M = rows of g
//   wgrad    A = dy rows (k-major), B = x rows (k-major);   K = rows of g
struct GArgs {
  const uint16_t* a;
  const uint16_t* b;
  const int32_t* offsets;
  void* out;
  int64_t rows, lda, ldb, ldo;
  int G;
  int n, k;  // output and input features
  int out_f32, accumulate;
  int vec;   // rows of outputs can be stored eight at a time
  // The contraction is split over `splits` workgroups per tile: split s writes
  // fp32 partial sums at out + s * split_stride, which grouped_finish_kernel
  // adds in split order (one split: the output itself).
  int splits;
  int64_t split_stride;
  // 256 x 256 tiles: workspace of the last round's shared tiles (NULL: none)
  float* tail_part;
  int32_t* tail_count;
};

// Tile tables of the groups from the device offsets, clamped to an ascending
// split of [0, rows]: t.off the row offsets, t.gnext[g] the first tile of
// group g + 1, bm rows and tn column tiles per row tile. Called by all
// threads of the block.
__device__ __forceinline__ void build_group_tables(GroupTables& t, const int32_t* offsets, int G,
                                                   int64_t rows, int bm, int tn) {
  const int lim = static_cast<int>(rows);
  for (int i = threadIdx.x; i < kMaxGroups; i += blockDim.x)
    t.off[i] = i <= G ? min(max(offsets[i], 0), lim) : 0;
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int v[8], run = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      run = max(run, t.off[8 * lane + j]);
      v[j] = run;
    }
    // running maximum over the lanes before this one
    int m = run;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int o = __shfl_up(m, s, 64);
      if (lane >= s) m = max(m, o);
    }
    const int up = __shfl_up(m, 1, 64);
    const int before = lane ? up : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) t.off[8 * lane + j] = max(v[j], before);
    if (lane == 63) t.off[kMaxGroups - 1] = max(m, t.off[kMaxGroups - 1]);
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int c[8], sum = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int g = 8 * lane + j;
      const int r = g < G ? t.off[g + 1] - t.off[g] : 0;
      sum += (r + bm - 1) / bm * tn;
      c[j] = sum;
    }
    int p = sum;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int o = __shfl_up(p, s, 64);
      if (lane >= s) p += o;
    }
    const int before = p - sum;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      t.gnext[8 * lane + j] = 8 * lane + j < G ? before + c[j] : 0x7fffffff;
    if (lane == 63) t.total = p;
  }
  __syncthreads();
}

// Tile order inside a group: rows of 8 m-tiles, m fastest, so that the 32
// consecutive tiles an XCD runs at a time read 8 A panels and 4 B panels (one
// group of 8192 rows, 4096 x 7168: 431 us with m fastest over all 32 m-tiles,
// 380 this way).
constexpr int kSuper = 8;
__device__ __forceinline__ void super_tile(int rem, int tm, int tn, int& m, int& n) {
  const int per = kSuper * tn, gr = rem / per, r2 = rem - gr * per;
  const int sm = min(kSuper, tm - gr * kSuper);
  n = r2 / sm;
  m = gr * kSuper + (r2 - n * sm);
}

// Bytes from the first element of `rows` rows to the end of the last one.
__device__ __forceinline__ int64_t span(int rows, uint32_t ld_bytes, int width) {
  return rows > 0 ? int64_t(rows - 1) * ld_bytes + int64_t(width) * 2 : 0;
}

struct GTile {
  int g, m, n;       // group, tile indices
  int s, splits;     // split of the contraction
  int64_t row0;      // first row of the group
  int rows;          // rows of the group
};

template <int MODE, int BM, int BN>
__device__ __forceinline__ GTile tile_of(const GArgs& a, const GroupTables& t, int unit) {
  GTile c;
  const int tile = unit / a.splits;
  c.s = unit - tile * a.splits;
  c.splits = a.splits;
  if constexpr (MODE == kWgrad) {
    const int tm = (a.n + BM - 1) / BM, tn = (a.k + BN - 1) / BN;
    c.g = tile / (tm * tn);
    super_tile(tile - c.g * tm * tn, tm, tn, c.m, c.n);
    const int r0 = __builtin_amdgcn_readfirstlane(t.off[c.g]);
    c.row0 = r0;
    c.rows = __builtin_amdgcn_readfirstlane(t.off[c.g + 1]) - r0;
  } else {
    const TileCoord tc = tile_coord_lds(t, a.G, 0, tile, BM);
    c.g = tc.g;
    c.row0 = tc.rbase;
    c.rows = tc.rows;
    const int tm = (tc.rows + BM - 1) / BM;
    super_tile(tc.n * tm + tc.m, tm, ((MODE == kForward ? a.n : a.k) + BN - 1) / BN, c.m, c.n);
  }
  return c;
}

// Stores eight adjacent values of a row, of which `cnt` exist.
__device__ __forceinline__ void put8(const GArgs& a, int64_t at, int cnt, const float (&v)[8]) {
  if (a.out_f32) {
    float* p = static_cast<float*>(a.out) + at;
    if (a.vec && cnt >= 8) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < cnt) p[j] = v[j];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(a.out) + at;
    if (a.vec && cnt >= 8) {
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < cnt) p[j] = f32_to_bf16(v[j]);
    }
  }
}

// Output of a finished tile. Forward and dgrad hold the transposed tile and
// store rows through LDS; wgrad holds the tile itself (a lane owns a column, so
// one register across the wave is two 128-byte row pieces of fp32).
template <class C, int MODE, class P>
__device__ __forceinline__ void store_tile(const GArgs& a, const GTile& c, int wm, int wn, int lane,
                                           f32x16_t (&acc)[C::MI][C::NJ], float* stage) {
  if constexpr (MODE == kWgrad) {
    const int64_t base = int64_t(c.g) * a.n * a.k + c.s * a.split_stride;
#pragma unroll
    for (int nj = 0; nj < C::NJ; ++nj) {
      const int col = c.n * C::BN + wn * C::WN + nj * 32 + (lane & 31);
#pragma unroll
      for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int row = c.m * C::BM + wm * C::WM + mi * 32 + acc_row(lane, r);
          if (row < a.n && col < a.k) {
            float* p = static_cast<float*>(a.out) + base + int64_t(row) * a.k + col;
            if (a.accumulate)
              *p += acc[mi][nj][r];
            else
              __builtin_nontemporal_store(acc[mi][nj][r], p);
          }
        }
    }
  } else {
    const int N = MODE == kForward ? a.n : a.k;
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
      for (int part = 0; part < P::PARTS; ++part) {
        const int col = c.n * C::BN + wn * C::WN + part * P::COLS + P::col(lane);
        P::put(stage, lane, acc[mi], part);
#pragma unroll
        for (int p = 0; p < P::N; ++p) {
          float v[8];
          P::get(stage, lane, p, v);
          const int r = c.m * C::BM + wm * C::WM + mi * 32 + P::row(p, lane);
          if (r < c.rows && col < N)
            put8(a, c.s * a.split_stride + (c.row0 + r) * a.ldo + col, N - col, v);
        }
      }
  }
}

// ---- operands of any alignment ------------------------------------------------

// Eight elements at p (any element alignment), of which the first `cnt` exist;
// the others are read from `safe` and dropped, so that the loads of all chunks
// go out without a branch between them.
__device__ __forceinline__ uint4 chunk_any(const uint16_t* p, int cnt, const uint16_t* safe) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = *(2 * j < cnt ? p + 2 * j : safe);
    const uint32_t hi = *(2 * j + 1 < cnt ? p + 2 * j + 1 : safe);
    w[j] = (2 * j < cnt ? lo : 0u) | (2 * j + 1 < cnt ? hi << 16 : 0u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

using TileAny = Tile<128, 128, 64, 32, 2>;   // 8 waves
using TileAnyLow = Tile<64, 128, 32, 32, 2>;   // 8 waves, for groups of few rows
using TileAnyBig = Tile<128, 256, 64, 64, 2>;  // a quarter fewer loaded bytes per product

// Odd widths, pitches or base addresses: operands pass through registers
// (unaligned 16-byte loads, element loads at the ends) into the same LDS
// layouts, loaded two k-steps ahead of the MFMAs and stored to LDS one ahead.
// (The weight gradient's small tile fits 128 registers, two workgroups per CU:
// 8192 rows, 2047 x 4095: 305 us, 384 with one. The others would spill.)
// Bound by the way through registers: with one workgroup per CU loads, stores to
// LDS and matrix instructions take turns, 295 us for x [8192, 4095], 8 x 2048,
// 3.5 times what the operations need at a library product's rate.
template <class C, int MODE>
__global__ __launch_bounds__(C::NT, MODE == kWgrad && C::BN == 128 ? 4 : 2) void
grouped_any_kernel(GArgs a) {
  constexpr bool AKM = MODE == kWgrad, BKM = MODE != kForward, SWAP = MODE != kWgrad;
  // after the k-loop the stages are free and hold the output rows
  __shared__ __attribute__((aligned(16))) uint16_t lds[C::LDS_ELEMS];
  static_assert(C::NWAVES * RowPasses<C>::FLOATS * 2 <= C::LDS_ELEMS, "output stages fit");
  __shared__ GroupTables gt;
  const int N = MODE == kForward ? a.n : a.k, M_w = a.n;
  const int tn = (N + C::BN - 1) / C::BN;
  build_group_tables(gt, a.offsets, a.G, a.rows, C::BM, tn);
  const int total = (MODE == kWgrad ? a.G * ((M_w + C::BM - 1) / C::BM) * tn : gt.total) * a.splits;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  for (int tile = xcd_logical_block(blockIdx.x, gridDim.x); tile < total; tile += gridDim.x) {
    const GTile c = tile_of<MODE, C::BM, C::BN>(a, gt, tile);
    const int K = MODE == kForward ? a.k : MODE == kDgrad ? a.n : c.rows;
    const uint16_t* A = a.a + (MODE == kWgrad ? c.row0 : c.row0 + int64_t(c.m) * C::BM) * a.lda;
    const uint16_t* B = MODE == kWgrad ? a.b + c.row0 * a.ldb : a.b + int64_t(c.g) * a.n * a.k;
    const int a_rows = MODE == kWgrad ? a.n : c.rows - c.m * C::BM;
    const uint16_t* Bt = MODE == kForward ? B + int64_t(c.n) * C::BN * a.ldb : B;
    const int b_rows = a.n - c.n * C::BN;  // forward: rows of W_g from the tile's first
    const int nk = (K + BK - 1) / BK;
    struct Step {
      uint4 a[C::A_LOADS], b[C::B_LOADS];
    } s0, s1;
    // Element offset of the thread's chunk p in a k-step (LDS chunk p * NT +
    // tid). k-contiguous: rows past the operand's last take that one (their
    // outputs are not stored).
    uint32_t oa[C::A_LOADS], ob[C::B_LOADS];
    auto contig = [&](int p, int rows, int64_t ld) {
      const int r = (tid >> 3) + p * C::RPP;
      return static_cast<uint32_t>(min(r, rows - 1) * ld) + ((tid & 7) ^ ((r >> 1) & 7)) * 8;
    };
    auto kmajor = [&](int p, int W, int64_t ld, int col0, int width) {
      const int cpr = W / 8, row = p * (C::NT / cpr) + tid / cpr;
      const int col = col0 + ((tid % cpr) ^ (4 * (row & 3))) * 8;
      return static_cast<uint32_t>(row * ld) + (col < width ? col : 0);
    };
#pragma unroll
    for (int p = 0; p < C::A_LOADS; ++p)
      oa[p] = AKM ? kmajor(p, C::BM, a.lda, c.m * C::BM, a.n) : contig(p, a_rows, a.lda);
#pragma unroll
    for (int p = 0; p < C::B_LOADS; ++p)
      ob[p] = BKM ? kmajor(p, C::BN, a.ldb, c.n * C::BN, a.k) : contig(p, b_rows, a.ldb);
    // A k-step before the last: whole chunks, no checks. A k-major chunk may run
    // up to 7 elements past its row's end into the next row (columns whose
    // outputs are not stored): the last row is in the last k-step, and with
    // rows of fewer than 8 elements every step is checked.
    const bool inner = (!AKM || a.lda >= 8) && (!BKM || a.ldb >= 8);
    auto fetch_inner = [&](int ks, Step& s) {
      const uint16_t* pa = A + (AKM ? int64_t(ks) * BK * a.lda : int64_t(ks) * BK);
      const uint16_t* pb = Bt + (BKM ? int64_t(ks) * BK * a.ldb : int64_t(ks) * BK);
#pragma unroll
      for (int p = 0; p < C::A_LOADS; ++p) __builtin_memcpy(&s.a[p], pa + oa[p], 16);
#pragma unroll
      for (int p = 0; p < C::B_LOADS; ++p) __builtin_memcpy(&s.b[p], pb + ob[p], 16);
    };
    auto checked = [&](bool km, const uint16_t* P, int64_t ld, int rows, int col0, int width, int W,
                       int p, int ks) -> uint4 {
      if (km) {
        const int cpr = W / 8, row = p * (C::NT / cpr) + tid / cpr;
        const int kr = ks * BK + row;
        const int col = col0 + ((tid % cpr) ^ (4 * (row & 3))) * 8;
        return chunk_any(P + kr * ld + col, kr < K ? width - col : 0, P);
      }
      const int r = (tid >> 3) + p * C::RPP;
      const int k0 = ks * BK + ((tid & 7) ^ ((r >> 1) & 7)) * 8;
      return chunk_any(P + r * ld + k0, r < rows ? K - k0 : 0, P);
    };
    const KRange kr = split_range(nk, c.s, a.splits);
    const int k_in = inner ? min(kr.k1, nk - 1) : kr.k0;  // steps below it need no checks
    auto fetch = [&](int ks, Step& s) {
      if (ks >= kr.k1) return;
      if (ks < k_in) {
        fetch_inner(ks, s);
        return;
      }
#pragma unroll
      for (int p = 0; p < C::A_LOADS; ++p)
        s.a[p] = checked(AKM, A, a.lda, a_rows, c.m * C::BM, a.n, C::BM, p, ks);
#pragma unroll
      for (int p = 0; p < C::B_LOADS; ++p)
        s.b[p] = checked(BKM, Bt, a.ldb, b_rows, c.n * C::BN, a.k, C::BN, p, ks);
    };
    auto stash = [&](int st, const Step& r) {
      uint16_t* s = lds + st * C::STAGE;
#pragma unroll
      for (int p = 0; p < C::A_LOADS; ++p)
        *reinterpret_cast<uint4*>(s + (p * C::NT + tid) * 8) = r.a[p];
#pragma unroll
      for (int p = 0; p < C::B_LOADS; ++p)
        *reinterpret_cast<uint4*>(s + C::BM * BK + (p * C::NT + tid) * 8) = r.b[p];
    };
    f32x16_t acc[C::MI][C::NJ];
    zero_acc<C>(acc);
    auto multiply = [&](int st) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        bf16x8_t af[C::MI], bf[C::NJ];
#pragma unroll
        for (int i = 0; i < C::MI; ++i)
          af[i] = frag_a<C, AKM>(lds, st, wm * C::WM + i * 32, kk, lane);
#pragma unroll
        for (int i = 0; i < C::NJ; ++i)
          bf[i] = frag_b<C, BKM>(lds, st, wn * C::WN + i * 32, kk, lane);
#pragma unroll
        for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
          for (int nj = 0; nj < C::NJ; ++nj)
            acc[mi][nj] = mma16<TypeBf16, SWAP>(af[mi], bf[nj], acc[mi][nj]);
      }
    };
    // steps ks (stage st, its registers free) and ks + 1 (in `next`)
    auto step = [&](int ks, int st, Step& free, const Step& next) {
      fetch(ks + 2, free);
      multiply(st);
      if (ks + 1 < kr.k1) stash(st ^ 1, next);
      lds_barrier();
    };
    // the same where step ks + 2 needs no checks: no branch between a load and
    // its use, so the wait counts stay exact
    auto step_inner = [&](int ks, int st, Step& free, const Step& next) {
      fetch_inner(ks + 2, free);
      multiply(st);
      stash(st ^ 1, next);
      lds_barrier();
    };
    int ks = kr.k0;
    fetch(ks, s0);
    fetch(ks + 1, s1);
    if (ks < kr.k1) stash(0, s0);
    lds_barrier();
    for (; ks + 3 < k_in; ks += 2) {
      step_inner(ks, 0, s0, s1);
      step_inner(ks + 1, 1, s1, s0);
    }
    for (; ks < kr.k1; ks += 2) {
      step(ks, 0, s0, s1);
      if (ks + 1 < kr.k1) step(ks + 1, 1, s1, s0);
    }
    store_tile<C, MODE, RowPasses<C>>(a, c, wm, wn, lane, acc,
                                      reinterpret_cast<float*>(lds) + wave * RowPasses<C>::FLOATS);
    __syncthreads();
  }
}

// ---- 16-byte aligned operands --------------------------------------------------

// Operand rows, pitches and base addresses in whole 16-byte chunks: loads go
// straight into LDS.
//
// What bounds it, measured: 32 x 128 tiles the stream of weights (128 rows over
// 256 experts of 4096 x 7168: 858 us, 6.9 TB/s); 256 x 256 tiles the matrix
// cores and, per tile, the rows that pad a group to whole tiles and an output
// of 6 us that nothing overlaps (12288 rows, one group of 4096 x 7168: 1.27
// PFLOP/s; 24576 rows over 64 groups of 2816 x 2048: 0.72, 42% more rows
// multiplied than there are); the weight gradient its fp32 stores, 12 us a tile
// (8192 rows over 32 groups of 7168 x 2048: 541 us, 1.88 GB). Issuing the next
// tile's loads ahead of those stores gained 3% there and cost up to 9% where
// groups are short; two workgroups per CU of 128 x 128 tiles took 710 us.
template <class C, int MODE, bool PHASED>
__global__ __launch_bounds__(C::NT, C::MINW) void grouped_kernel(GArgs a) {
  constexpr bool AKM = MODE == kWgrad, BKM = MODE != kForward, SWAP = MODE != kWgrad;
  constexpr int kStageElems = PHASED || MODE == kWgrad ? 0 : C::NWAVES * RowPasses<C>::FLOATS * 2;
  __shared__ __attribute__((aligned(16))) uint16_t lds[C::LDS_ELEMS + kStageElems];
  __shared__ GroupTables gt;
  const int N = MODE == kForward ? a.n : a.k;
  const int tn = (N + C::BN - 1) / C::BN;
  build_group_tables(gt, a.offsets, a.G, a.rows, C::BM, tn);
  __shared__ int flag;
  const int tiles =
      (MODE == kWgrad ? a.G * ((a.n + C::BM - 1) / C::BM) * tn : gt.total) * a.splits;
  Tail tail{tiles, 1, a.tail_part, a.tail_count};
  int nb = gridDim.x;
  if (a.tail_part) {
    // all resident workgroups are launched, as the choice of this kernel assumed;
    // those without a unit end here, and the others are spread over the XCDs
    const int whole = tiles / nb * nb;
    const int nk = ((MODE == kForward ? a.k : a.n) + BK - 1) / BK;
    tail.splits =
        tail_splits(tiles - whole, nk, nb, kBigStep * C::BM / 256, C::BM * C::BN / 256);
    if (tail.splits > 1) tail.whole = whole;
    nb = min(nb, (tail.whole + (tiles - tail.whole) * tail.splits + 7) / 8 * 8);
    if (static_cast<int>(blockIdx.x) >= nb) return;
  }
  const int total = tail.whole + (tiles - tail.whole) * tail.splits;
  const int first = xcd_logical_block(blockIdx.x, nb);
  if (first >= total) return;
  auto locate = [&](int unit) {
    const Unit u = unit_of(tail, unit);
    GTile c = tile_of<MODE, C::BM, C::BN>(a, gt, u.tile);
    if (u.splits > 1) {
      c.s = u.s;
      c.splits = u.splits;
    }
    return c;
  };
  const uint32_t lda = static_cast<uint32_t>(a.lda) * 2u, ldb = static_cast<uint32_t>(a.ldb) * 2u;
  auto depth = [&](const GTile& c) { return MODE == kForward ? a.k : MODE == kDgrad ? a.n : c.rows; };
  auto range = [&](const GTile& c) {
    return split_range((depth(c) + BK - 1) / BK, c.s, c.splits);
  };
  auto next_ops = [&](int unit, Ops16<C>& op) {
    const GTile c = locate(unit);
    const KRange kr = range(c);
    // an empty range (an empty group, or fewer k-steps than splits) reads one
    // k-step of zeros
    op.nk = max(kr.k1 - kr.k0, 1);
    const int64_t k0 = int64_t(kr.k0) * BK;
    const int K = static_cast<int>(min(int64_t(depth(c)), int64_t(kr.k1) * BK) - k0);
    if constexpr (MODE == kWgrad) {
      // A dword that the resource's end cuts reads as zero, so an odd width ends
      // with the dword of its last value: rows start on 16 bytes, so the other
      // half of it is in the same aligned dword, and only feeds column n (or k),
      // which is not stored.
      kmajor_operand<C, C::BM>(op.ra, op.ao, op.base_a, op.left_a, op.step_a,
                               a.a + (c.row0 + k0) * a.lda, c.m * C::BM, lda,
                               span(K, lda, (a.n + 1) & ~1));
      kmajor_operand<C, C::BN>(op.rb, op.bo, op.base_b, op.left_b, op.step_b,
                               a.b + (c.row0 + k0) * a.ldb, c.n * C::BN, ldb,
                               span(K, ldb, (a.k + 1) & ~1));
    } else {
      const int left = c.rows - c.m * C::BM;
      kcontig_operand<C>(op.ra, op.ao, op.tail_a, a.a + (c.row0 + int64_t(c.m) * C::BM) * a.lda + k0,
                         left, lda, span(min(left, C::BM), lda, K), K);
      const uint16_t* W = a.b + int64_t(c.g) * a.n * a.k;
      if constexpr (MODE == kForward) {
        const int nleft = a.n - c.n * C::BN;
        kcontig_operand<C>(op.rb, op.bo, op.tail_b, W + int64_t(c.n) * C::BN * a.ldb + k0, nleft,
                           ldb, span(min(nleft, C::BN), ldb, K), K);
      } else {
        kmajor_operand<C, C::BN>(op.rb, op.bo, op.base_b, op.left_b, op.step_b, W + k0 * a.ldb,
                                 c.n * C::BN, ldb, span(K, ldb, a.k));
      }
    }
  };
  struct Epilogue {
    const GArgs& a;
    const Tail& tail;
    int* flag;
    decltype(locate)& at;
    decltype(range)& steps;
    __device__ int k_steps(int unit) const {
      const KRange r = steps(at(unit));
      return max(r.k1 - r.k0, 1);
    }
    __device__ void operator()(int unit, int wm, int wn, int lane, f32x16_t (&acc)[C::MI][C::NJ],
                               float* stage) const {
      GTile c = at(unit);
      if constexpr (PHASED && MODE != kWgrad) {
        if (!join_splits<C>(acc, tail, unit, unit_of(tail, unit), flag)) return;
        c.s = 0;
      }
      using P = std::conditional_t<PHASED, StagePasses<C>, RowPasses<C>>;
      store_tile<C, MODE, P>(a, c, wm, wn, lane, acc, stage);
    }
  } ep{a, tail, &flag, locate, range};
  if constexpr (PHASED)
    stream_phased<C, TypeBf16, AKM, BKM, SWAP>(lds, first, nb, total, next_ops, ep);
  else
    stream_ring<C, TypeBf16, AKM, BKM, SWAP>(lds, first, nb, total, next_ops, ep);
}

// Sums of the splits' partial outputs, in split order, eight columns of a row
// per thread. Rows [offsets[0], max offsets) exist (forward, dgrad), or all
// (offsets NULL).
struct FinishArgs {
  const float* part;
  const int32_t* offsets;
  void* out;
  int64_t rows, ldp, ldo, split_stride;
  int G, N, splits, out_f32, accumulate;
};
__global__ __launch_bounds__(256) void grouped_finish_kernel(FinishArgs a) {
  const int per = (a.N + 7) / 8;
  const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = id / per;
  const int c0 = static_cast<int>(id - row * per) * 8;
  if (a.offsets) {
    __shared__ int last[4];
    int end = 0;
    for (int g = threadIdx.x; g <= a.G; g += 256) end = max(end, a.offsets[g]);
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) end = max(end, wave_shfl_xor(end, k));
    if ((threadIdx.x & 63) == 0) last[threadIdx.x >> 6] = end;
    __syncthreads();
    end = max(max(last[0], last[1]), max(last[2], last[3]));
    if (row < max(a.offsets[0], 0) || row >= end) return;
  }
  if (row >= a.rows) return;
  const int cnt = min(a.N - c0, 8);
  float v[8] = {};
  const float* p = a.part + row * a.ldp + c0;
  for (int s = 0; s < a.splits; ++s, p += a.split_stride) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < cnt) v[j] += p[j];
  }
  const int64_t at = row * a.ldo + c0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < cnt) {
      if (a.out_f32) {
        float* o = static_cast<float*>(a.out) + at + j;
        *o = a.accumulate ? *o + v[j] : v[j];
      } else {
        static_cast<uint16_t*>(a.out)[at + j] = f32_to_bf16(v[j]);
      }
    }
}

// ---- choice of the kernel -------------------------------------------------------

using TileBig = Tile<256, 256, 128, 64, 2>;          // 8 waves, two-phase loop, 128 KB LDS
using TileFlat = Tile<192, 256, 96, 64, 2>;          // the same where these fill one round, 112 KB
using TileMid = Tile<128, 128, 64, 32, 3>;           // 8 waves
using TileDec = Tile<32, 128, 32, 64, 6, true>;      // 2 waves, weights streamed past L2

template <int MODE, class C>
int64_t tile_bound(const GArgs& a) {
  const int64_t tn = ((MODE == kForward ? a.n : a.k) + C::BN - 1) / C::BN;
  if (MODE == kWgrad) return int64_t(a.G) * ((a.n + C::BM - 1) / C::BM) * tn;
  const int64_t full = a.rows / C::BM + (a.rows < a.G ? a.rows : a.G);
  return full * tn;
}

enum Config { kBig, kFlat, kMid, kDec, kAny, kAnyLow, kAnyBig };

struct Choice {
  int config, splits;
  bool tail;            // share the last round's tiles
  int64_t ldp, stride;  // partial outputs
};
// Workspace of shared tiles: one partial tile per workgroup, one counter per tile.
constexpr int kTailSlots = 256;
constexpr size_t kTailPart = size_t(kTailSlots) * TileBig::BM * TileBig::BN * sizeof(float);
constexpr size_t kTailBytes = kTailPart + kTailSlots * sizeof(int32_t);

// Whether every row of both operands starts on a 16-byte chunk, and (rows along
// the contraction) ends on one.
bool chunked(const GroupedArgs& p) {
  if (p.mode == kForward) return p.k % 8 == 0 && p.ld_k % 8 == 0;
  if (p.mode == kDgrad) return p.n % 8 == 0 && p.k % 8 == 0 && p.ld_n % 8 == 0;
  return p.ld_n % 8 == 0 && p.ld_k % 8 == 0;
}

// Time model of a tile (microseconds), fitted to measured products: `busy` and
// `idle` per k-step with the GPU full or at most half full of tiles, `fixed` for
// a tile's first loads and its output (no wgrad: 0), `slots` tiles at a time.
struct TileCost {
  int config, bm, bn, slots;
  double busy, idle, fixed, fixed_wgrad;
};
constexpr TileCost kCosts[] = {
    {kBig, 256, 256, 256, 1.7, 1.05, 8.0, 12.0},
    {kFlat, 192, 256, 256, 1.46, 0.8, 8.0, 0.0},
    {kMid, 128, 128, 256, 0.65, 0.38, 4.0, 4.0},
    {kDec, 32, 128, 256, 0.6, 0.35, 3.0, 0.0},
    {kAny, 128, 128, 256, 0.95, 0.8, 5.0, 5.0},
    {kAnyLow, 64, 128, 256, 0.6, 0.6, 5.0, 0.0},
    {kAnyBig, 128, 256, 256, 1.45, 1.2, 8.0, 0.0},
};

// The rule: the tile and the number of splits with the least modelled time.
// Row counts per group live on the device, so the expected number of row tiles
// stands in for them: one per group while groups are smaller than a tile, else
// rows / BM and half a tile per group. What it decides, as measured (us):
//   x [128, 7168], 256 experts x 4096       32 x 128: 867, 128^2: 1004, 256^2: 1255
//   x [1000, 2048], 8 x 1408                128^2: 22, 32 x 128: 33, 256^2: 44
//   x [2048, 7168], 32 x 4096               128^2: 343, 256^2: 408, 32 x 128: 567
//   x [8192, 7168], 32 x 4096, Zipf loads   256^2: 621, 192 x 256: 671, 128^2: 729
//   x [5000, 2048], 8 x 2048                192 x 256: 51, 256^2: 59, 128^2: 68
//   x [3000, 4096], 1 x 4096                192 x 256: 101, 256^2: 102
//   x [30000, 2048], 100 x 1408, Zipf       256^2: 256, 192 x 256: 304
//   x [8192, 4095], 8 x 2048                128 x 256: 295, 128^2: 335 (any alignment)
//   x [2311, 613], 9 x 1407                 128^2: 26, 64 x 128: 31, 128 x 256: 32 (any)
//   dx of [2311, 1407], 9 x 613             64 x 128: 24, 128^2: 30 (any alignment)
//   dw of 8000 rows, 2 x 256 x 256          4 splits: 24, 1: 42 (128^2), 99 (256^2)
//   x [8, 4096], 1 x 2048                   4 splits: 18, 1: 26 (32 x 128)
// and where it is wrong, the tile it takes first:
//   x [1536, 7168], 1 x 1408                192 x 256, shared: 73, whole: 110; 128^2: 57
//   x [30000, 2048], 100 x 1408, even loads 256^2: 288, 192 x 256: 273
//   dx of [24576, 2816], 64 x 2048, Zipf    256^2: 397, 192 x 256: 373
// Splits add the finishing launch and the partial sums' traffic, so they pay
// only where few tiles leave most of the GPU idle for many k-steps.
Choice choose(const GroupedArgs& p, bool aligned) {
  const int64_t N = p.mode == kForward ? p.n : p.k;
  const double touched = static_cast<double>(p.rows < p.n_groups ? p.rows : p.n_groups);
  Choice best{};
  best.ldp = p.mode == kWgrad ? N : (N + 7) / 8 * 8;
  best.stride =
      ((p.mode == kWgrad ? int64_t(p.n_groups) * p.n : p.rows) * best.ldp + 63) / 64 * 64;
  double least = 0.0;
  for (const TileCost& t : kCosts) {
    if ((t.config >= kAny) == aligned || (t.fixed_wgrad == 0.0 && p.mode == kWgrad)) continue;
    const double nt = static_cast<double>((N + t.bn - 1) / t.bn);
    double tiles, depth;
    if (p.mode == kWgrad) {
      tiles = p.n_groups * nt * ((p.n + t.bm - 1) / t.bm);
      depth = static_cast<double>(p.rows) / p.n_groups;
    } else {
      const double mt = p.n_groups == 1 ? std::ceil(p.rows / static_cast<double>(t.bm))
                                        : p.rows / static_cast<double>(t.bm) + 0.5 * touched;
      tiles = nt * (mt > touched ? mt : touched);
      depth = p.mode == kForward ? p.k : p.n;
    }
    const double nk = std::ceil(depth / BK);
    for (int splits = 1; splits <= 16 && (splits == 1 || splits * 4 <= nk); splits *= 2) {
      const double units = tiles * splits;
      const double step = units <= t.slots / 2 ? t.idle : t.busy;
      // A tile of a long contraction in the last round is shared by the
      // workgroups that this round leaves idle; that takes a launch to clear the
      // counters, so it is left out where little can be won. With more than one
      // group the number of tiles is an estimate: half a round stands for what
      // the last one holds, a quarter where it is shared.
      const bool tail = t.config <= kFlat && p.mode != kWgrad && splits == 1 && nk >= 48.0;
      const double share = units / t.slots;
      double rounds = std::ceil(share), us = 0.0;
      if (p.mode != kWgrad && p.n_groups > 1) {
        if (share > 1.0) rounds = share + (tail ? 0.25 : 0.5);
      } else if (tail) {
        const float k_us = kBigStep * t.bm / 256, kb = t.bm * t.bn / 256.0f;
        const int rest = static_cast<int>(units) % t.slots, k = static_cast<int>(nk);
        const int s = tail_splits(rest, k, t.slots, k_us, kb);
        if (s > 1) {
          rounds = std::floor(share);
          us = 5.0 + (k + s - 1) / s * k_us + t.fixed + kb / 22.0 + s * kb / 30.0;
        }
      }
      us += rounds * (std::ceil(nk / splits) * step +
                      (p.mode == kWgrad ? t.fixed_wgrad : t.fixed));
      if (splits > 1) us += 6.0 + splits * best.stride * 8.0 / 1.5e6;
      if (!best.splits || us < least) {
        least = us;
        best.config = t.config;
        best.splits = splits;
        best.tail = tail;
      }
    }
  }
  return best;
}

template <class C, int MODE, bool PHASED>
void launch_fast(const GArgs& a, hipStream_t s) {
  // shared tiles: every workgroup that its workspace has room for
  const int64_t units = a.tail_part ? kTailSlots : tile_bound<MODE, C>(a) * a.splits;
  hipLaunchKernelGGL((grouped_kernel<C, MODE, PHASED>),
                     dim3(grid_of<grouped_kernel<C, MODE, PHASED>>(C::NT, units)), dim3(C::NT), 0, s,
                     a);
}

template <class C, int MODE>
void launch_any(const GArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(
      (grouped_any_kernel<C, MODE>),
      dim3(grid_of<grouped_any_kernel<C, MODE>>(C::NT, tile_bound<MODE, C>(a) * a.splits)),
      dim3(C::NT), 0, s, a);
}

template <int MODE>
void launch_config(const GArgs& a, int config, hipStream_t s) {
  if (config == kAny) {
    launch_any<TileAny, MODE>(a, s);
  } else if (config == kAnyLow) {
    if constexpr (MODE != kWgrad) launch_any<TileAnyLow, MODE>(a, s);
  } else if (config == kAnyBig) {
    if constexpr (MODE != kWgrad) launch_any<TileAnyBig, MODE>(a, s);
  } else if (config == kFlat) {
    if constexpr (MODE != kWgrad) launch_fast<TileFlat, MODE, true>(a, s);
  } else if (config == kMid) {
    launch_fast<TileMid, MODE, false>(a, s);
  } else if (config == kDec) {
    if constexpr (MODE != kWgrad) launch_fast<TileDec, MODE, false>(a, s);
  } else {
    launch_fast<TileBig, MODE, true>(a, s);
  }
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

size_t grouped_workspace(const GroupedArgs& p) {
  // the pointers' alignment is not known yet: enough for either kernel
  size_t bytes = 0;
  for (int aligned = 0; aligned <= chunked(p); ++aligned) {
    const Choice c = choose(p, aligned);
    const size_t b = c.splits > 1 ? size_t(c.splits) * c.stride * sizeof(float)
                     : c.tail     ? kTailBytes
                                  : 0;
    if (b > bytes) bytes = b;
  }
  return bytes;
}

hipError_t launch_grouped(const GroupedArgs& p, void* ws, hipStream_t s) {
  if (p.rows == 0 && p.mode != kWgrad) return hipSuccess;
  const Choice c = choose(p, chunked(p) && on16(p.a) && on16(p.b));
  GArgs a{};
  a.a = static_cast<const uint16_t*>(p.a);
  a.b = static_cast<const uint16_t*>(p.b);
  a.offsets = p.offsets;
  a.rows = p.rows;
  a.G = p.n_groups;
  a.n = p.n;
  a.k = p.k;
  a.lda = p.mode == kForward ? p.ld_k : p.ld_n;
  a.ldb = p.mode == kWgrad ? p.ld_k : p.k;
  a.splits = c.splits;
  const int64_t ldo = p.mode == kForward ? p.ld_n : p.mode == kDgrad ? p.ld_k : p.k;
  if (c.splits > 1) {
    a.out = ws;
    a.ldo = c.ldp;
    a.out_f32 = 1;
    a.split_stride = c.stride;
    a.vec = 1;
  } else {
    a.out = p.out;
    a.ldo = ldo;
    a.out_f32 = p.out_f32;
    a.accumulate = p.accumulate;
    a.vec = ldo % 8 == 0 && on16(p.out);
  }
  if (c.tail) {
    a.tail_part = static_cast<float*>(ws);
    a.tail_count = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kTailPart);
    const hipError_t e = launch_fill_i32(a.tail_count, kTailSlots, 0, s);
    if (e != hipSuccess) return e;
  }
  if (p.mode == kForward)
    launch_config<kForward>(a, c.config, s);
  else if (p.mode == kDgrad)
    launch_config<kDgrad>(a, c.config, s);
  else
    launch_config<kWgrad>(a, c.config, s);
  if (c.splits > 1) {
    FinishArgs f{};
    f.part = static_cast<const float*>(ws);
    f.offsets = p.mode == kWgrad ? nullptr : p.offsets;
    f.out = p.out;
    f.rows = p.mode == kWgrad ? int64_t(p.n_groups) * p.n : p.rows;
    f.ldp = c.ldp;
    f.ldo = ldo;
    f.split_stride = c.stride;
    f.G = p.n_groups;
    f.N = p.mode == kForward ? p.n : p.k;
    f.splits = c.splits;
    f.out_f32 = p.out_f32;
    f.accumulate = p.accumulate;
    const int64_t threads = f.rows * ((f.N + 7) / 8);
    hipLaunchKernelGGL(grouped_finish_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)),
                       dim3(256), 0, s, f);
  }
  return hipGetLastError();
}

}  // namespace dsmoe
