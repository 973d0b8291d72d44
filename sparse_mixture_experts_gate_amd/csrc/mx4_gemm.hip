// Products grouped by expert on microscaled 4-bit operands (definition in
// dsmoe_tokens.h): y = x W_g^T over ragged row groups.
//
// A block of 32 codes is 16 bytes, the 16-byte chunk of the 16-bit products'
// tiles: operands go straight into LDS in 128-byte rows (a k-step: 256 values),
// with the same swizzle, loaders and loops. A matrix instruction of 32 x 32 x 64
// takes one block per lane and its scale byte from a register's byte chosen by the
// instruction. The k order inside a step is ours to choose: lane half h takes
// chunks 4 h .. 4 h + 3, so the scale word [k / 128][row] of its half holds the
// bytes of its four sub-steps, and one 4-byte LDS read per 32 rows serves a k-step.
#include <cmath>

#include "device_common.h"
#include "gemm16_core.h"
#include "group_tables.h"
#include "internal.h"
#include "resident_grid.h"
#include "row_io.h"
#include "tile_schedule.h"

namespace dsmoe {

namespace {

constexpr int kStepBlocks = 8;  // blocks of a row per k-step
constexpr int kFp4 = 4;         // operand format of the scaled matrix instructions

struct MArgs {
  const uint8_t* xc;
  const uint8_t* wc;
  const uint8_t* xs;
  const uint8_t* ws;
  const int32_t* offsets;
  void* y;
  int64_t rows, ldy;
  int G, n;
  int kb;   // blocks of a row
  int kg;   // words of scales of a row
  int out_f32, vec;
};

// Scale words of a stage: [A half 0 | A half 1 | B half 0 | B half 1], rows adjacent,
// in pieces of 64 words, dealt over the waves.
template <class C>
struct Scales {
  static constexpr int WORDS = 2 * (C::BM + C::BN);
  static constexpr int PIECES = WORDS / 64;
  static constexpr int LOADS = (PIECES + C::NWAVES - 1) / C::NWAVES;
  static constexpr int STAGE = LOADS * C::NWAVES * 64;  // words, the last pieces unused
  static_assert(WORDS % 64 == 0 && (2 * C::BM) % 64 == 0, "a piece belongs to one operand");
};

template <class C>
struct MOps {
  i32x4_t ra, rb;
  i32x4_t rs[Scales<C>::LOADS];
  uint32_t ao[C::A_LOADS], bo[C::B_LOADS], so[Scales<C>::LOADS];
  uint32_t sstep[Scales<C>::LOADS];  // bytes between k-steps
  uint32_t tail_a, tail_b;
  int nk;
};

struct MTile {
  int g, m, n;
  int64_t row0;
  int rows;
};

template <class C>
__device__ __forceinline__ MTile tile_of(const MArgs& a, const GroupTables& t, int tile) {
  MTile c;
  const TileCoord tc = tile_coord_lds(t, a.G, 0, tile, C::BM);
  c.g = tc.g;
  c.row0 = tc.rbase;
  c.rows = tc.rows;
  const int tm = (tc.rows + C::BM - 1) / C::BM;
  super_tile(tc.n * tm + tc.m, tm, (a.n + C::BN - 1) / C::BN, c.m, c.n);
  return c;
}

__device__ __forceinline__ int64_t row_span(int rows, uint32_t ld) {
  return rows > 0 ? int64_t(rows) * ld : 0;
}

template <class C>
__device__ __forceinline__ void tile_ops(const MArgs& a, const MTile& c, int wave, MOps<C>& op) {
  using S = Scales<C>;
  const uint32_t ld = static_cast<uint32_t>(a.kb) * 16u;  // bytes of a row, of both operands
  const int left = c.rows - c.m * C::BM, nleft = a.n - c.n * C::BN;
  const int64_t row = c.row0 + int64_t(c.m) * C::BM;
  const int64_t col = int64_t(c.g) * a.n + int64_t(c.n) * C::BN;
  op.nk = (a.kb + kStepBlocks - 1) / kStepBlocks;
  // in units of 16 bits, 8 to a chunk
  kcontig_operand<C>(op.ra, op.ao, op.tail_a, a.xc + row * ld, left, ld,
                     row_span(min(left, C::BM), ld), a.kb * 8);
  kcontig_operand<C>(op.rb, op.bo, op.tail_b, a.wc + col * ld, nleft, ld,
                     row_span(min(nleft, C::BN), ld), a.kb * 8);
  // Scales past the last word of a row read as zeros: a group's own words end the
  // resource, so that no other group's bytes (a NaN) meet the zero codes there.
  // Rows past the operand's read other rows' words; their outputs are not stored.
  const i32x4_t rsa = rsrc4(a.xs, static_cast<uint32_t>(a.kg) * static_cast<uint32_t>(a.rows) * 4u);
  const i32x4_t rsb = rsrc4(a.ws + int64_t(c.g) * a.kg * a.n * 4,
                            static_cast<uint32_t>(a.kg) * static_cast<uint32_t>(a.n) * 4u);
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int j = 0; j < S::LOADS; ++j) {
    const int piece = j * C::NWAVES + wave;
    const bool is_a = piece * 64 < 2 * C::BM;
    const int i = piece * 64 + lane - (is_a ? 0 : 2 * C::BM);
    const int width = is_a ? C::BM : C::BN;
    const uint32_t half = static_cast<uint32_t>(i / width), r = static_cast<uint32_t>(i % width);
    const uint32_t plane = static_cast<uint32_t>(is_a ? a.rows : a.n) * 4u;
    const uint32_t r0 = static_cast<uint32_t>(is_a ? row : int64_t(c.n) * C::BN);
    op.rs[j] = is_a ? rsa : rsb;
    op.so[j] = piece < S::PIECES ? half * plane + (r0 + r) * 4u : kInvalidRow;
    op.sstep[j] = 2u * plane;
  }
}

// The issue side: walks the k-steps of a workgroup's tiles (first, first + nb, ...
// below total) and loads codes and scales into ring stages. Past the last step it
// loads that step again into stages nobody reads.
template <class C, class NextOps>
struct MLoader {
  using S = Scales<C>;
  MOps<C> op;
  NextOps& next_ops;
  uint32_t lds0, sc0;
  int ti, nb, total, ki, wave;
  bool more;
  static constexpr int NL = C::A_LOADS + C::B_LOADS + S::LOADS;

  __device__ MLoader(NextOps& n, uint32_t l0, uint32_t s0, int first, int nb_, int total_,
                     int wave_)
      : next_ops(n), lds0(l0), sc0(s0), ti(first), nb(nb_), total(total_), ki(0), wave(wave_),
        more(true) {
    next_ops(ti, op);
  }
  // load i of NL of the current k-step into stage st
  __device__ __forceinline__ void load(int st, int i) {
    const uint32_t base =
        __builtin_amdgcn_readfirstlane(lds0 + (st * C::STAGE + wave * 8 * BK) * 2);
    const uint32_t kn = static_cast<uint32_t>(ki) * (BK * 2);
    const bool last = ki == op.nk - 1;
    if (i < C::A_LOADS) {
      dma16(op.ra, (op.ao[i] + kn) | (last ? op.tail_a : 0u), base + i * C::RPP * BK * 2);
    } else if (i < C::A_LOADS + C::B_LOADS) {
      const int j = i - C::A_LOADS;
      const uint32_t v = (op.bo[j] + kn) | (last ? op.tail_b : 0u);
      const uint32_t at = base + C::BM * BK * 2 + j * C::RPP * BK * 2;
      if constexpr (C::B_NT)
        dma16_nt(op.rb, v, at);
      else
        dma16(op.rb, v, at);
    } else {
      const int j = i - C::A_LOADS - C::B_LOADS;
      const uint32_t at = __builtin_amdgcn_readfirstlane(
          sc0 + (st * S::STAGE + (j * C::NWAVES + wave) * 64) * 4);
      dma4(op.rs[j], op.so[j] + static_cast<uint32_t>(ki) * op.sstep[j], at);
    }
  }
  __device__ __forceinline__ void advance() {
    if (!more || ++ki < op.nk) return;
    ki = 0;
    ti += nb;
    if (ti < total) {
      next_ops(ti, op);
    } else {
      more = false;
      ki = op.nk - 1;
    }
  }
};

// 16 bytes (one block) of row l % 32 for sub-step kk: chunk 4 (l / 32) + kk.
template <class C>
__device__ __forceinline__ i32x4_t block_of(const uint16_t* lds, int st, bool b, int row, int kk,
                                            int lane) {
  const uint16_t* s = lds + st * C::STAGE + (b ? C::BM * BK : 0);
  return *reinterpret_cast<const i32x4_t*>(s + lds_off(row + (lane & 31), 4 * (lane >> 5) + kk));
}
// Scale word of row l % 32 for the lane's half of the step.
template <class C>
__device__ __forceinline__ int word_of(const uint32_t* sc, int st, bool b, int row, int lane) {
  const uint32_t* s = sc + st * Scales<C>::STAGE + (b ? 2 * C::BM : 0);
  return static_cast<int>(s[(lane >> 5) * (b ? C::BN : C::BM) + row + (lane & 31)]);
}

// c + b a with sub-step KK's bytes of the scale words; the W operand goes first,
// so c holds the transposed tile (lane l: row l % 32 of x's side).
template <int KK>
__device__ __forceinline__ f32x16_t mma4(i32x4_t a, i32x4_t b, f32x16_t c, int sa, int sb) {
  const i32x8_t A = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
  const i32x8_t B = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(B, A, c, kFp4, kFp4, KK, sb, KK, sa);
}

// Stores eight adjacent values of a row, of which `cnt` exist.
__device__ __forceinline__ void put8(const MArgs& a, int64_t at, int cnt, const uint32_t (&w)[4]) {
  uint16_t* p = static_cast<uint16_t*>(a.y) + at;
  if (a.vec && cnt >= 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < cnt) p[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
  }
}
__device__ __forceinline__ void put4(const MArgs& a, int64_t at, int cnt, const float (&v)[4]) {
  float* p = static_cast<float*>(a.y) + at;
  if (a.vec && cnt >= 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < cnt) p[j] = v[j];
  }
}

// Output of a finished tile, straight from registers, so that no barrier holds the
// other waves: a lane has columns 8 g + 4 h .. + 3 (g = 0 .. 3, h its half) of row l %
// 32. For bf16 the halves swap words, which leaves each lane 8 adjacent columns of
// its row, 16 bytes.
template <class C>
__device__ __forceinline__ void store_tile(const MArgs& a, const MTile& c, int wm, int wn, int lane,
                                           const f32x16_t (&acc)[C::MI][C::NJ]) {
  const int h = lane >> 5;
#pragma unroll
  for (int mi = 0; mi < C::MI; ++mi) {
    const int r = c.m * C::BM + wm * C::WM + mi * 32 + (lane & 31);
    const int64_t row = (c.row0 + r) * a.ldy;
#pragma unroll
    for (int nj = 0; nj < C::NJ; ++nj) {
      const int col0 = c.n * C::BN + wn * C::WN + nj * 32;
      const f32x16_t& x = acc[mi][nj];
      if (a.out_f32) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int col = col0 + 8 * g + 4 * h;
          const float v[4] = {x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]};
          if (r < c.rows && col < a.n) put4(a, row + col, a.n - col, v);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const auto s = __builtin_amdgcn_permlane32_swap(
                bf16_pair(x[8 * q + 2 * j], x[8 * q + 2 * j + 1]),
                bf16_pair(x[8 * q + 4 + 2 * j], x[8 * q + 4 + 2 * j + 1]), false, false);
            w[j] = s[0];
            w[2 + j] = s[1];
          }
          const int col = col0 + 16 * q + 8 * h;
          if (r < c.rows && col < a.n) put8(a, row + col, a.n - col, w);
        }
      }
    }
  }
}

// The k-loop: NST stages; the blocks of sub-step kk + 1 are read between the matrix
// instructions of sub-step kk. One barrier per k-step, before its last sub-step,
// whose blocks are already in registers: behind it the step's stage is free and is
// loaded with step k + NST at once, and step k + 1's loads, NST - 1 steps old, have
// landed. Waves are in step only there, so the two waves of a SIMD fill each
// other's gaps, and a wave that stores its tile holds no other up.
template <class C, class NextOps, class Epilogue>
__device__ __forceinline__ void mx4_ring(uint16_t* lds, uint32_t* sc, int first, int nb, int total,
                                         NextOps&& next_ops, Epilogue&& epilogue) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  using L = MLoader<C, std::remove_reference_t<NextOps>>;
  constexpr int NST = C::NST, NL = L::NL, INFLIGHT = NL * (NST - 2);
  constexpr int NR = C::MI + C::NJ, NM = C::MI * C::NJ;
  static_assert(INFLIGHT <= 63, "vmcnt range");
  L ld(next_ops, lds_addr(lds), lds_addr(sc), first, nb, total, wave);
  i32x4_t af[2][C::MI], bf[2][C::NJ];
  int sa[C::MI], sb[C::NJ], na[C::MI], nbs[C::NJ];
  f32x16_t acc[C::MI][C::NJ];
  auto rd = [&](int st, int kk, int buf, int i) {
    if (i < C::NJ)
      bf[buf][i] = block_of<C>(lds, st, true, wn * C::WN + i * 32, kk, lane);
    else
      af[buf][i - C::NJ] = block_of<C>(lds, st, false, wm * C::WM + (i - C::NJ) * 32, kk, lane);
  };
  auto rd_scales = [&](int st) {
#pragma unroll
    for (int i = 0; i < C::MI; ++i) na[i] = word_of<C>(sc, st, false, wm * C::WM + i * 32, lane);
#pragma unroll
    for (int i = 0; i < C::NJ; ++i) nbs[i] = word_of<C>(sc, st, true, wn * C::WN + i * 32, lane);
  };
  auto use_scales = [&] {
#pragma unroll
    for (int i = 0; i < C::MI; ++i) sa[i] = na[i];
#pragma unroll
    for (int i = 0; i < C::NJ; ++i) sb[i] = nbs[i];
  };
  auto sub = [&](auto kk_c, int st_rd, int st_dma) {
    constexpr int KK = decltype(kk_c)::value, buf = KK & 1;
    constexpr int RPS = (NR + NM - 1) / NM, LPS = (NL + NM - 1) / NM;
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      const int mi = i / C::NJ, nj = i % C::NJ;
      acc[mi][nj] = mma4<KK>(af[buf][mi], bf[buf][nj], acc[mi][nj], sa[mi], sb[nj]);
      // holds the instruction here (no code): selected out of this order, all blocks
      // of a k-step are live at once and spill
      asm volatile("" : "+v"(acc[mi][nj]));
#pragma unroll
      for (int q = 0; q < RPS; ++q)
        if (i * RPS + q < NR) rd(st_rd, (KK + 1) & 3, buf ^ 1, i * RPS + q);
      if constexpr (KK == 3) {
#pragma unroll
        for (int q = 0; q < LPS; ++q)
          if (i * LPS + q < NL) ld.load(st_dma, i * LPS + q);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int j = 0; j < NST; ++j) {
#pragma unroll
    for (int i = 0; i < NL; ++i) ld.load(j, i);
    ld.advance();
  }
  vm_wait<(INFLIGHT + NL < 63 ? INFLIGHT + NL : 63)>();
  lds_barrier();
  int st = 0;
#pragma unroll
  for (int i = 0; i < NR; ++i) rd(st, 0, 0, i);
  rd_scales(st);
  for (int tc = first; tc < total; tc += nb) {
    zero_acc<C>(acc);
    const int nkc = epilogue.k_steps();
    for (int kc = 0; kc < nkc; ++kc) {
      const int next = st == NST - 1 ? 0 : st + 1;
      use_scales();
      sub(std::integral_constant<int, 0>{}, st, 0);
      sub(std::integral_constant<int, 1>{}, st, 0);
      sub(std::integral_constant<int, 2>{}, st, 0);
      vm_wait<INFLIGHT>();
      lds_barrier();
      rd_scales(next);
      sub(std::integral_constant<int, 3>{}, next, st);
      ld.advance();
      st = next;
    }
    epilogue(tc, wm, wn, lane, acc);
  }
  vm_wait<0>();
}

template <class C>
__global__ __launch_bounds__(C::NT, C::MINW) void mx4_gemm_kernel(MArgs a) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[C::LDS_ELEMS];
  __shared__ uint32_t sc[C::NST * Scales<C>::STAGE];
  __shared__ GroupTables gt;
  build_group_tables(gt, a.offsets, a.G, a.rows, C::BM, (a.n + C::BN - 1) / C::BN);
  const int total = gt.total, nb = gridDim.x;
  const int first = xcd_logical_block(blockIdx.x, nb);
  if (first >= total) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  auto next_ops = [&](int tile, MOps<C>& op) { tile_ops<C>(a, tile_of<C>(a, gt, tile), wave, op); };
  struct Epilogue {
    const MArgs& a;
    const GroupTables& t;
    __device__ int k_steps() const { return (a.kb + kStepBlocks - 1) / kStepBlocks; }
    __device__ void operator()(int tile, int wm, int wn, int lane,
                               const f32x16_t (&acc)[C::MI][C::NJ]) const {
      store_tile<C>(a, tile_of<C>(a, t, tile), wm, wn, lane, acc);
    }
  } ep{a, gt};
  mx4_ring<C>(lds, sc, first, nb, total, next_ops, ep);
}

// ---- choice of the kernel -------------------------------------------------------

using TileBig = Tile<256, 256, 128, 64, 2>;      // 8 waves
using TileMid = Tile<128, 128, 64, 32, 3>;       // 8 waves
using TileDec = Tile<32, 128, 32, 64, 6, true>;  // 2 waves, weights streamed past L2

template <class C>
int64_t tile_bound(const MArgs& a) {
  const int64_t tn = (a.n + C::BN - 1) / C::BN;
  return (a.rows / C::BM + (a.rows < a.G ? a.rows : a.G)) * tn;
}

template <class C>
void launch(const MArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((mx4_gemm_kernel<C>), dim3(grid_of<mx4_gemm_kernel<C>>(C::NT, tile_bound<C>(a))),
                     dim3(C::NT), 0, s, a);
}

// Time model of a tile (microseconds): `busy` and `idle` per k-step with the GPU
// full or at most half full of tiles, `fixed` for a tile's first loads and its
// output.
struct TileCost {
  int bm, bn;
  double busy, idle, fixed;
};
constexpr TileCost kCosts[] = {
    {256, 256, 1.7, 1.05, 8.0}, {128, 128, 0.65, 0.38, 4.0}, {32, 128, 0.6, 0.35, 3.0}};

int choose(const MArgs& a) {
  const double touched = static_cast<double>(a.rows < a.G ? a.rows : a.G);
  const double nk = (a.kb + kStepBlocks - 1) / kStepBlocks;
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < 3; ++i) {
    const TileCost& t = kCosts[i];
    const double mt = a.G == 1 ? std::ceil(a.rows / static_cast<double>(t.bm))
                               : a.rows / static_cast<double>(t.bm) + 0.5 * touched;
    const double share = (a.n + t.bn - 1) / t.bn * (mt > touched ? mt : touched) / 256;
    double rounds = std::ceil(share);
    if (a.G > 1 && share > 1.0) rounds = share + 0.5;
    const double us = rounds * (nk * (share <= 0.5 ? t.idle : t.busy) + t.fixed);
    if (i == 0 || us < least) {
      least = us;
      best = i;
    }
  }
  return best;
}

}  // namespace

hipError_t launch_mx4_gemm(const Mx4GemmArgs& p, hipStream_t s) {
  if (p.rows == 0) return hipSuccess;
  MArgs a{};
  a.xc = p.xc;
  a.wc = p.wc;
  a.xs = p.xs;
  a.ws = p.wsc;
  a.offsets = p.offsets;
  a.y = p.y;
  a.rows = p.rows;
  a.ldy = p.ldy;
  a.G = p.G;
  a.n = p.n;
  a.kb = (p.k + 31) / 32;
  a.kg = (a.kb + 3) / 4;
  a.out_f32 = p.out_f32;
  a.vec = p.ldy % 8 == 0 && (reinterpret_cast<uintptr_t>(p.y) & 15) == 0;
  const int c = choose(a);
  if (c == 0)
    launch<TileBig>(a, s);
  else if (c == 1)
    launch<TileMid>(a, s);
  else
    launch<TileDec>(a, s);
  return hipGetLastError();
}

}  // namespace dsmoe
