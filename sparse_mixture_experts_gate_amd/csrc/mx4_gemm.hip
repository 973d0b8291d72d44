// Products grouped by expert on microscaled 4-bit operands (definition in
// dsmoe_tokens.h): y = x W_g^T over ragged row groups.
//
// A block of 32 codes is 16 bytes: operands go straight into LDS by 16-byte loads,
// rows of 8 blocks (a k-step of 256 values) in XOR-swizzled chunks. A matrix
// instruction of 32 x 32 x 64 takes one block per lane and its scale byte from a
// register's byte chosen by the instruction. The k order inside a step is ours to
// choose: lane half h takes chunks 4 h .. 4 h + 3, so the scale word [k / 128][row] of
// its half holds the bytes of its four sub-steps, and one 4-byte LDS read per 32 rows
// serves a k-step.
//
// What bounds it, measured. Large products no unit by itself: one group of 8192 rows,
// 4096 x 7168, takes 112 to 129 us, 3.7 to 4.3 PFLOP/s, at 1.9 GHz; the matrix
// instructions are busy for half of the cycles (alone, operands held in registers, they
// reach 6.4 PFLOP/s at 1.5 GHz), LDS reads for 22% (a CU reads 204 bytes a cycle and more),
// and zero codes take 87 us where random ones take 112. With the loads into LDS switched
// off the same loop takes 52% of the time: a k-step's 64 KB of loads and its matrix
// instructions take turns, as a ring of two stages has no more than one step in flight.
// Few rows: the stream of weights (128 rows over 256 experts of 4096 x 7168: 227 us, 6.9
// TB/s). Measured equal or slower on large products: waves in step per sub-step as in the
// 16-bit products' large tiles (four barriers more a step), k-steps of 128 values in four
// stages, loads of the lines three steps ahead into L2, waves without rows leaving out
// their matrix instructions, the last round's tiles cut into quarters, operands through
// registers three steps ahead into two stages (128 rows a tile, Zipf loads over 32
// groups: 226 against 199).
#include "device_common.h"
#include "gemm16_core.h"
#include "group_tables.h"
#include "internal.h"
#include "mx4_tiles.h"
#include "resident_grid.h"
#include "row_io.h"
#include "tile_schedule.h"

namespace dsmoe {

namespace {

constexpr int kFp4 = 4;  // operand format of the scaled matrix instructions

constexpr int kChunks = 8;          // blocks of a row per k-step, 16 bytes each
constexpr int kRow = kChunks * 16;  // bytes of a row of a stage
constexpr int kSubs = kChunks / 2;  // matrix instructions along a k-step

// BM x BN tile in waves of WM x WN (ALIKE waves on each), NST LDS stages in the load ring.
template <int BM_, int BN_, int WM_, int WN_, int NST_, bool B_NT_ = false, int ALIKE = 1>
struct MxTile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NST = NST_;
  static constexpr bool B_NT = B_NT_;  // weights streamed past L2
  static constexpr int WAVES_N = BN / WN, NWAVES = BM / WM * WAVES_N * ALIKE, NT = NWAVES * 64;
  static constexpr int MI = WM / 32, NJ = WN / 32;
  static constexpr int RPP = NT / kChunks;  // rows covered by one pass of 16-byte loads
  static constexpr int A_LOADS = BM / RPP, B_LOADS = BN / RPP;
  // scale words of a stage: [A half-steps][BM], then [B half-steps][BN]
  static constexpr int A_WORDS = 2 * BM, B_WORDS = 2 * BN;
  // waves that load A's words; the others B's, or all of them both
  static constexpr bool SHARED = BM == BN;
  static constexpr int S_LOADS = SHARED ? 1 : 2;
  static constexpr int A_LANES = A_WORDS / 4 / (SHARED ? NWAVES / 2 : NWAVES);
  static constexpr int B_LANES = B_WORDS / 4 / (SHARED ? NWAVES / 2 : NWAVES);
  static constexpr int CODES = (BM + BN) * kRow;
  static constexpr int STAGE = CODES + (A_WORDS + B_WORDS) * 4;  // bytes
  static constexpr int NL = A_LOADS + B_LOADS + S_LOADS;         // loads of a wave and step
  static_assert(BM % RPP == 0 && BN % RPP == 0 && RPP % 16 == 0, "whole passes, one swizzle");
  static_assert(A_LANES <= 64 && B_LANES <= 64 && STAGE % 16 == 0, "one load of a wave's words");
  static_assert(NST >= 2 && NL * (NST - 2) <= 63, "ring depth within the vmcnt range");
};

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
  int out_f32;
};

// Swizzled position of a row's chunk: 16 lanes that one 128-bit LDS access serves
// together read one chunk of 16 adjacent rows, which this spreads over all banks.
__device__ __forceinline__ int position(int row, int chunk) {
  return chunk ^ ((row >> 1) & 7);
}

template <class C>
struct MOps {
  i32x4_t ra, rb, rs[C::S_LOADS];
  uint32_t ao[C::A_LOADS], bo[C::B_LOADS], so[C::S_LOADS];
  uint32_t sstep[C::S_LOADS];  // bytes between k-steps
  uint32_t tail;               // sends chunks past a row's end out of range in the last step
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

template <class C>
__device__ __forceinline__ void tile_ops(const MArgs& a, const MTile& c, int wave, MOps<C>& op) {
  const uint32_t ld = static_cast<uint32_t>(a.kb) * 16u;  // bytes of a row, of both operands
  const int left = min(c.rows - c.m * C::BM, C::BM), nleft = min(a.n - c.n * C::BN, C::BN);
  const int64_t row = c.row0 + int64_t(c.m) * C::BM;
  const int64_t col = int64_t(c.g) * a.n + int64_t(c.n) * C::BN;
  op.nk = (a.kb + kChunks - 1) / kChunks;
  op.ra = rsrc4(a.xc + row * ld, static_cast<uint32_t>(left) * ld);
  op.rb = rsrc4(a.wc + col * ld, static_cast<uint32_t>(nleft) * ld);
  const int r0 = threadIdx.x / kChunks, chunk = position(r0, threadIdx.x % kChunks);
#pragma unroll
  for (int p = 0; p < C::A_LOADS; ++p) {
    const int r = r0 + p * C::RPP;
    op.ao[p] = (r < left ? static_cast<uint32_t>(r) * ld : kInvalidRow) + chunk * 16u;
  }
#pragma unroll
  for (int p = 0; p < C::B_LOADS; ++p) {
    const int r = r0 + p * C::RPP;
    op.bo[p] = (r < nleft ? static_cast<uint32_t>(r) * ld : kInvalidRow) + chunk * 16u;
  }
  op.tail = (op.nk - 1) * kChunks + chunk < a.kb ? 0u : kInvalidRow;
  // Scales past the last word of a row read as zeros: a group's own words end the
  // resource, so that no other group's bytes (a NaN) meet the zero codes there.
  // Rows past the operand's read other rows' words; their outputs are not stored.
  const uint32_t pa = static_cast<uint32_t>(a.rows) * 4u, pb = static_cast<uint32_t>(a.n) * 4u;
  const i32x4_t rsa = rsrc4(a.xs, static_cast<uint32_t>(a.kg) * pa);
  const i32x4_t rsb = rsrc4(a.ws + int64_t(c.g) * a.kg * a.n * 4, static_cast<uint32_t>(a.kg) * pb);
  const int lane = threadIdx.x & 63;
  // first word of this lane's four of an operand's, `w` waves with `lanes` of them
  auto word = [&](int w, int lanes, int width, uint32_t plane, uint32_t first) {
    const int i = (w * lanes + min(lane, lanes - 1)) * 4;
    return static_cast<uint32_t>(i / width) * plane +
           (first + static_cast<uint32_t>(i % width)) * 4u;
  };
  const uint32_t fa = static_cast<uint32_t>(row), fb = static_cast<uint32_t>(c.n) * C::BN;
  if constexpr (C::SHARED) {
    const bool is_a = wave < C::NWAVES / 2;
    op.rs[0] = is_a ? rsa : rsb;
    op.so[0] = is_a ? word(wave, C::A_LANES, C::BM, pa, fa)
                    : word(wave - C::NWAVES / 2, C::B_LANES, C::BN, pb, fb);
    op.sstep[0] = 2u * (is_a ? pa : pb);
  } else {
    op.rs[0] = rsa;
    op.so[0] = word(wave, C::A_LANES, C::BM, pa, fa);
    op.sstep[0] = 2u * pa;
    op.rs[C::S_LOADS - 1] = rsb;
    op.so[C::S_LOADS - 1] = word(wave, C::B_LANES, C::BN, pb, fb);
    op.sstep[C::S_LOADS - 1] = 2u * pb;
  }
}

// The issue side: walks the k-steps of a workgroup's tiles (first, first + nb, ...
// below total) and loads codes and scales into ring stages. Past the last step it
// loads that step again into stages nobody reads.
template <class C, class NextOps>
struct MLoader {
  MOps<C> op;
  NextOps& next_ops;
  uint32_t lds0;
  int ti, nb, total, ki, wave;
  bool more;

  __device__ MLoader(NextOps& n, uint32_t l0, int first, int nb_, int total_, int wave_)
      : next_ops(n), lds0(l0), ti(first), nb(nb_), total(total_), ki(0), wave(wave_), more(true) {
    next_ops(ti, op);
  }
  // load i of NL of the current k-step into stage st
  __device__ __forceinline__ void load(int st, int i) {
    const uint32_t stage = lds0 + st * C::STAGE;
    const uint32_t base = __builtin_amdgcn_readfirstlane(stage + wave * 1024);
    const uint32_t kn = static_cast<uint32_t>(ki) * kRow;
    const uint32_t tail = ki == op.nk - 1 ? op.tail : 0u;
    if (i < C::A_LOADS) {
      dma16(op.ra, (op.ao[i] + kn) | tail, base + i * C::RPP * kRow);
    } else if (i < C::A_LOADS + C::B_LOADS) {
      const int j = i - C::A_LOADS;
      const uint32_t at = base + (C::BM + j * C::RPP) * kRow;
      if constexpr (C::B_NT)
        dma16_nt(op.rb, (op.bo[j] + kn) | tail, at);
      else
        dma16(op.rb, (op.bo[j] + kn) | tail, at);
    } else {
      const int j = i - C::A_LOADS - C::B_LOADS;
      const uint32_t v = op.so[j] + static_cast<uint32_t>(ki) * op.sstep[j];
      const int lanes = j == 0 ? C::A_LANES : C::B_LANES;
      const uint32_t at = stage + C::CODES + wave * lanes * 16 + (j == 0 ? 0 : C::A_WORDS * 4);
      if (static_cast<int>(threadIdx.x & 63) < lanes)
        dma16(op.rs[j], v, __builtin_amdgcn_readfirstlane(at));
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

// 16 bytes (one block) of row l % 32 for sub-step kk: chunk SUBS (l / 32) + kk.
template <class C>
__device__ __forceinline__ i32x4_t block_of(const uint8_t* stage, bool b, int row, int kk,
                                            int lane) {
  const int r = row + (lane & 31), chunk = kSubs * (lane >> 5) + kk;
  return *reinterpret_cast<const i32x4_t*>(stage + (b ? C::BM * kRow : 0) + r * kRow +
                                           position(r, chunk) * 16);
}
// Scale bytes of row l % 32 for the lane's half of the step, sub-step kk's in byte kk.
template <class C>
__device__ __forceinline__ int word_of(const uint8_t* stage, bool b, int row, int lane) {
  const uint32_t* s =
      reinterpret_cast<const uint32_t*>(stage + C::CODES) + (b ? C::A_WORDS : 0);
  const int r = row + (lane & 31), h = lane >> 5;
  return static_cast<int>(s[h * (b ? C::BN : C::BM) + r]);
}

// c + b a with sub-step KK's bytes of the scale words; the W operand goes first,
// so c holds the transposed tile (lane l: row l % 32 of x's side).
template <int KK>
__device__ __forceinline__ f32x16_t mma4(i32x4_t a, i32x4_t b, f32x16_t c, int sa, int sb) {
  const i32x8_t A = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
  const i32x8_t B = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(B, A, c, kFp4, kFp4, KK, sb, KK, sa);
}

// Stores eight (bf16) or four adjacent values of a row, of which `cnt` > 0 exist; all of
// them where FULL. Rows start at any element, which 16-byte stores take (13151 x 256 rows,
// 39 groups of 953: 56 us in two-byte stores, 22 so).
template <bool FULL>
__device__ __forceinline__ void put8(uint16_t* p, int cnt, const uint32_t (&w)[4]) {
  const u32x4_any_t r = {w[0], w[1], w[2], w[3]};
  if (FULL || cnt >= 8)
    *reinterpret_cast<u32x4_any_t*>(p) = r;
  else
    store_end(p, r, cnt);
}
template <bool FULL>
__device__ __forceinline__ void put4(float* p, int cnt, const float (&v)[4]) {
  typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));
  if (FULL || cnt >= 4) {
    *reinterpret_cast<f32x4_any_t*>(p) = f32x4_any_t{v[0], v[1], v[2], v[3]};
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < cnt) p[j] = v[j];
  }
}

// A lane has columns 8 g + 4 h .. + 3 (g = 0 .. 3, h its half) of row l % 32. For bf16
// the halves swap words, which leaves each lane 8 adjacent columns of its row, 16
// bytes. FULL: every row and column exists.
template <class C, bool FULL>
__device__ __forceinline__ void store_part(const MArgs& a, const MTile& c, int wm, int wn, int lane,
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
          if (FULL || (r < c.rows && col < a.n))
            put4<FULL>(static_cast<float*>(a.y) + row + col, a.n - col, v);
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
          if (FULL || (r < c.rows && col < a.n))
            put8<FULL>(static_cast<uint16_t*>(a.y) + row + col, a.n - col, w);
        }
      }
    }
  }
}
// Output of a finished tile, straight from registers, so that no barrier holds the
// other waves.
template <class C>
__device__ __forceinline__ void store_tile(const MArgs& a, const MTile& c, int wm, int wn, int lane,
                                           const f32x16_t (&acc)[C::MI][C::NJ]) {
  if (c.m * C::BM + (wm + 1) * C::WM <= c.rows && c.n * C::BN + (wn + 1) * C::WN <= a.n)
    store_part<C, true>(a, c, wm, wn, lane, acc);
  else
    store_part<C, false>(a, c, wm, wn, lane, acc);
}

// The k-loop: NST stages; the blocks of sub-step kk + 1 are read between the matrix
// instructions of sub-step kk. One barrier per k-step, before its last sub-step,
// whose blocks are already in registers: behind it the step's stage is free for step
// k + NST, whose loads go out over the next four sub-steps (with two stages all in
// the first of them, since they are waited for after four), and step k + 1's loads
// have landed. Waves are in step only there, so the two waves of a SIMD fill each
// other's gaps, and a wave that stores its tile holds no other up.
constexpr int min_of(int a, int b) { return a < b ? a : b; }
template <class C, class NextOps, class Epilogue>
__device__ __forceinline__ void mx4_ring(uint8_t* lds, int first, int nb, int total,
                                         NextOps&& next_ops, Epilogue&& epilogue) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  constexpr int NST = C::NST, NL = C::NL, INFLIGHT = NL * (NST - 2), LAST = kSubs - 1;
  // sub-steps over which a step's loads are spread
  constexpr int SLOTS = NST > 2 ? kSubs : 1;
  constexpr int NR = C::MI + C::NJ, NM = C::MI * C::NJ;
  MLoader<C, std::remove_reference_t<NextOps>> ld(next_ops, lds_addr(lds), first, nb, total, wave);
  i32x4_t af[2][C::MI], bf[2][C::NJ];
  int sa[C::MI], sb[C::NJ], na[C::MI], nbs[C::NJ];
  f32x16_t acc[C::MI][C::NJ];
  auto rd = [&](int st, int kk, int buf, int i) {
    const uint8_t* s = lds + st * C::STAGE;
    if (i < C::NJ)
      bf[buf][i] = block_of<C>(s, true, wn * C::WN + i * 32, kk, lane);
    else
      af[buf][i - C::NJ] = block_of<C>(s, false, wm * C::WM + (i - C::NJ) * 32, kk, lane);
  };
  auto rd_scales = [&](int st) {
    const uint8_t* s = lds + st * C::STAGE;
#pragma unroll
    for (int i = 0; i < C::MI; ++i) na[i] = word_of<C>(s, false, wm * C::WM + i * 32, lane);
#pragma unroll
    for (int i = 0; i < C::NJ; ++i) nbs[i] = word_of<C>(s, true, wn * C::WN + i * 32, lane);
  };
  auto use_scales = [&] {
#pragma unroll
    for (int i = 0; i < C::MI; ++i) sa[i] = na[i];
#pragma unroll
    for (int i = 0; i < C::NJ; ++i) sb[i] = nbs[i];
  };
  auto sub = [&](auto kk_c, int st_rd, int st_dma) {
    constexpr int KK = decltype(kk_c)::value, buf = KK & 1, next = KK == LAST ? 0 : KK + 1;
    constexpr int RPS = (NR + NM - 1) / NM;
    constexpr int SLOT = KK == LAST ? 0 : KK + 1, L0 = min_of(NL * SLOT / SLOTS, NL),
                  L1 = min_of(NL * (SLOT + 1) / SLOTS, NL);
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      const int mi = i / C::NJ, nj = i % C::NJ;
      acc[mi][nj] = mma4<KK>(af[buf][mi], bf[buf][nj], acc[mi][nj], sa[mi], sb[nj]);
      // holds the instruction here (no code): selected out of this order, all blocks
      // of a k-step are live at once and spill
      asm volatile("" : "+v"(acc[mi][nj]));
#pragma unroll
      for (int q = 0; q < RPS; ++q)
        if (i * RPS + q < NR) rd(st_rd, next, buf ^ 1, i * RPS + q);
#pragma unroll
      for (int l = L0; l < L1; ++l)
        if ((l - L0) * NM / (L1 - L0) == i) ld.load(st_dma, l);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int j = 0; j < NST; ++j) {
#pragma unroll
    for (int i = 0; i < (j < NST - 1 ? NL : NL / SLOTS); ++i) ld.load(j, i);
    if (j < NST - 1) ld.advance();
  }
  vm_wait<INFLIGHT>();
  lds_barrier();
  int st = 0;
#pragma unroll
  for (int i = 0; i < NR; ++i) rd(st, 0, 0, i);
  rd_scales(st);
  for (int tc = first; tc < total; tc += nb) {
    zero_acc<C>(acc);
    const int nkc = epilogue.k_steps();
    for (int kc = 0; kc < nkc; ++kc) {
      const int next = st == NST - 1 ? 0 : st + 1, last = st == 0 ? NST - 1 : st - 1;
      use_scales();
      sub(std::integral_constant<int, 0>{}, st, last);
      sub(std::integral_constant<int, 1>{}, st, last);
      sub(std::integral_constant<int, 2>{}, st, last);
      ld.advance();
      vm_wait<INFLIGHT>();
      lds_barrier();
      rd_scales(next);
      sub(std::integral_constant<int, LAST>{}, next, st);
      st = next;
    }
    epilogue(tc, wm, wn, lane, acc);
  }
  vm_wait<0>();
}

// The k-loop of few tiles: 32 columns of weights a tile, so that four times as many CUs
// stream them. The four waves load a quarter each, all multiply the whole tile, each on
// its own matrix core and in the order of the other tiles (a row's sums are the same bits
// in every tile), and wave g ends with columns 8 g .. of each 32. One barrier per k-step:
// behind it the step's blocks are there and the stage before it is free. Latency-bound: a
// row of 7168 by 4096 x 7168 12 to 13 us (a launch and its 16 MB 5.6), of which the 112 matrix
// instructions one after the other are most: with the next step's blocks read ahead the
// same, split over the waves 8.9, which would make a row's sums depend on the tile.
template <class C, class NextOps, class Epilogue>
__device__ __forceinline__ void mx4_thin_ring(uint8_t* lds, int first, int nb, int total,
                                              NextOps&& next_ops, Epilogue&& epilogue) {
  static_assert(C::NWAVES == 4 && C::MI == 1 && C::NJ == 1, "one tile, a quarter a wave");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  MLoader<C, std::remove_reference_t<NextOps>> ld(next_ops, lds_addr(lds), first, nb, total, wave);
  auto load_step = [&](int st) {
#pragma unroll
    for (int i = 0; i < C::NL; ++i) ld.load(st, i);
    ld.advance();
  };
#pragma unroll
  for (int j = 0; j < C::NST - 1; ++j) load_step(j);
  int st = 0;
  for (int tc = first; tc < total; tc += nb) {
    f32x16_t acc = {};
    const int nkc = epilogue.k_steps();
    for (int kc = 0; kc < nkc; ++kc) {
      vm_wait<C::NL*(C::NST - 2)>();
      lds_barrier();
      load_step(st == 0 ? C::NST - 1 : st - 1);
      const uint8_t* s = lds + st * C::STAGE;
      const int sa = word_of<C>(s, false, 0, lane), sb = word_of<C>(s, true, 0, lane);
      i32x4_t a[kSubs], b[kSubs];
#pragma unroll
      for (int kk = 0; kk < kSubs; ++kk) {
        a[kk] = block_of<C>(s, false, 0, kk, lane);
        b[kk] = block_of<C>(s, true, 0, kk, lane);
      }
      acc = mma4<0>(a[0], b[0], acc, sa, sb);
      acc = mma4<1>(a[1], b[1], acc, sa, sb);
      acc = mma4<2>(a[2], b[2], acc, sa, sb);
      acc = mma4<3>(a[3], b[3], acc, sa, sb);
      st = st == C::NST - 1 ? 0 : st + 1;
    }
    epilogue(tc, wave, lane, acc);
  }
  vm_wait<0>();
}

// waves per SIMD the register budget is sized for
template <class C>
constexpr int kMinWaves = C::NWAVES >= 8 ? 2 : 1;

template <class C>
__global__ __launch_bounds__(C::NT, kMinWaves<C>) void mx4_gemm_kernel(MArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::NST * C::STAGE];
  __shared__ GroupTables gt;
  build_group_tables(gt, a.offsets, a.G, a.rows, C::BM, (a.n + C::BN - 1) / C::BN);
  // the grid is sized for the most tiles there can be: fewer are spread over all XCDs
  const int total = gt.total, nb = min(static_cast<int>(gridDim.x), (total + 7) / 8 * 8);
  if (static_cast<int>(blockIdx.x) >= nb) return;
  const int first = xcd_logical_block(blockIdx.x, nb);
  if (first >= total) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  auto next_ops = [&](int tile, MOps<C>& op) { tile_ops<C>(a, tile_of<C>(a, gt, tile), wave, op); };
  struct Epilogue {
    const MArgs& a;
    const GroupTables& t;
    __device__ int k_steps() const { return (a.kb + kChunks - 1) / kChunks; }
    __device__ void operator()(int tile, int wm, int wn, int lane,
                               const f32x16_t (&acc)[C::MI][C::NJ]) const {
      store_tile<C>(a, tile_of<C>(a, t, tile), wm, wn, lane, acc);
    }
  } ep{a, gt};
  mx4_ring<C>(lds, first, nb, total, next_ops, ep);
}

template <class C>
__global__ __launch_bounds__(C::NT) void mx4_thin_kernel(MArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::NST * C::STAGE];
  __shared__ GroupTables gt;
  build_group_tables(gt, a.offsets, a.G, a.rows, C::BM, (a.n + C::BN - 1) / C::BN);
  const int total = gt.total, nb = min(static_cast<int>(gridDim.x), (total + 7) / 8 * 8);
  if (static_cast<int>(blockIdx.x) >= nb) return;
  const int first = xcd_logical_block(blockIdx.x, nb);
  if (first >= total) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  auto next_ops = [&](int tile, MOps<C>& op) { tile_ops<C>(a, tile_of<C>(a, gt, tile), wave, op); };
  struct Epilogue {
    const MArgs& a;
    const GroupTables& t;
    __device__ int k_steps() const { return (a.kb + kChunks - 1) / kChunks; }
    // columns 8 g + 4 h .. + 3 of row l % 32
    __device__ void operator()(int tile, int g, int lane, const f32x16_t& acc) const {
      const MTile c = tile_of<C>(a, t, tile);
      const int r = c.m * C::BM + (lane & 31), col = c.n * C::BN + 8 * g + 4 * (lane >> 5);
      if (r >= c.rows || col >= a.n) return;
      const int64_t at = (c.row0 + r) * a.ldy + col;
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float lo = g & 1 ? +acc[4 + j] : +acc[j], hi = g & 1 ? +acc[12 + j] : +acc[8 + j];
        v[j] = g & 2 ? hi : lo;
      }
      if (a.out_f32) {
        put4<false>(static_cast<float*>(a.y) + at, a.n - col, v);
        return;
      }
      uint16_t* p = static_cast<uint16_t*>(a.y) + at;
      const u32x4_any_t w = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), 0, 0};
      if (a.n - col >= 4)
        *reinterpret_cast<u32x2_any2_t*>(p) = u32x2_any2_t{w[0], w[1]};
      else
        store_end(p, w, a.n - col);
    }
  } ep{a, gt};
  mx4_thin_ring<C>(lds, first, nb, total, next_ops, ep);
}

// ---- choice of the kernel -------------------------------------------------------

using TileBig = MxTile<256, 256, 128, 64, 2>;      // 8 waves
using TileWide = MxTile<128, 256, 64, 64, 3>;      // 8 waves
using TileFlat = MxTile<64, 256, 32, 64, 3>;       // 8 waves
using TileLow = MxTile<32, 128, 32, 32, 6, true>;  // 4 waves, weights streamed past L2
using TileThin = MxTile<32, 32, 32, 32, 4, true, 4>;  // the same, 4 waves alike

template <class C>
int64_t tile_bound(const MArgs& a) {
  const int64_t tn = (a.n + C::BN - 1) / C::BN;
  return (a.rows / C::BM + (a.rows < a.G ? a.rows : a.G)) * tn;
}

template <auto K, class C>
void launch(const MArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(K, dim3(grid_of<K>(C::NT, tile_bound<C>(a))), dim3(C::NT), 0, s, a);
}

template <class C>
constexpr bool sized(Mx4Tile t) {
  return C::BM == kCosts[t].bm && C::BN == kCosts[t].bn;
}
static_assert(sized<TileBig>(kTile256) && sized<TileWide>(kTile128) && sized<TileFlat>(kTile64) &&
                  sized<TileLow>(kTile32) && TileThin::BM == kThin && TileThin::BN == kThin,
              "the tiles that the rule weighs");

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
  switch (mx4_tile(p.rows, p.G, p.n, p.k)) {
    case kTile256:
      launch<mx4_gemm_kernel<TileBig>, TileBig>(a, s);
      break;
    case kTile128:
      launch<mx4_gemm_kernel<TileWide>, TileWide>(a, s);
      break;
    case kTile64:
      launch<mx4_gemm_kernel<TileFlat>, TileFlat>(a, s);
      break;
    case kTile32:
      launch<mx4_gemm_kernel<TileLow>, TileLow>(a, s);
      break;
    case kTileThin:
      launch<mx4_thin_kernel<TileThin>, TileThin>(a, s);
      break;
  }
  return hipGetLastError();
}

}  // namespace dsmoe
