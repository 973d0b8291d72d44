// Core of the 16-bit matrix products of the expert operators (bf16 or fp16
// operands, fp32 accumulation): tile shapes, one tile's operand streams and
// the two k-loops that run a workgroup's tiles.
//
// An operand is k-contiguous ([M, K] rows, the contraction along a row) or
// k-major ([K, M] rows, a k-step is 64 consecutive rows). Both go from memory
// straight into LDS (16-byte LDS-DMA loads) in the layouts of
// gemm_bf16_core.h: 128-byte rows with XOR-swizzled chunks, or 64 k rows read
// back by transpose reads.
#pragma once

#include <type_traits>

#include "gemm_bf16_core.h"

namespace dsmoe {
namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

// Operand types of the matrix cores; fragments travel as bf16x8_t (16 bytes).
struct TypeBf16 {
  __device__ static f32x16_t mfma(bf16x8_t a, bf16x8_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
struct TypeF16 {
  __device__ static f32x16_t mfma(bf16x8_t a, bf16x8_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
  }
};

// One tile's operands. `tail` masks (0, or the sign bit that sends an offset
// out of range) apply in the last k-step to chunks past the contraction of a
// k-contiguous operand. A k-major operand's resource is moved forward by
// `step` bytes every k-step (64-bit base: a group's rows may exceed 2^31
// bytes), with `left` bytes from it to the operand's end; rows past the end
// read as zeros in hardware.
template <class C>
struct Ops16 {
  i32x4_t ra, rb;
  uint32_t ao[C::A_LOADS], bo[C::B_LOADS];
  uint32_t tail_a, tail_b;
  uint64_t base_a, base_b;  // k-major only
  int64_t left_a, left_b;
  uint32_t step_a, step_b;
  int nk;
};

__device__ __forceinline__ uint32_t clamp_bytes(int64_t n) {
  return static_cast<uint32_t>(n < 0 ? 0 : n < 0x7fffffff ? n : 0x7fffffff);
}

// Rows of a k-contiguous operand: row r of the tile at base + r * ld_bytes,
// `rows` of them exist; K elements along a row.
template <class C, int LOADS>
__device__ __forceinline__ void kcontig_operand(i32x4_t& rs, uint32_t (&o)[LOADS], uint32_t& tail,
                                                const void* base, int rows, uint32_t ld_bytes,
                                                int64_t bytes, int K) {
  const int r0 = threadIdx.x >> 3, ch = threadIdx.x & 7;
  static_assert(C::RPP % 16 == 0, "a thread's logical chunk is the same in every pass");
#pragma unroll
  for (int p = 0; p < LOADS; ++p) {
    const int r = r0 + p * C::RPP;
    o[p] = r < rows ? static_cast<uint32_t>(r) * ld_bytes : kInvalidRow;
  }
  swizzle_rows<C>(o);
  const int chunk = ch ^ ((r0 >> 1) & 7);
  tail = ((K - 1) / BK * BK + chunk * 8 < K) ? 0u : kInvalidRow;
  rs = rsrc4(base, clamp_bytes(bytes));
}

// Columns col0 .. of a k-major operand whose first contraction row is at
// `base`; `bytes` from there to the end of its last row.
template <class C, int W, int LOADS>
__device__ __forceinline__ void kmajor_operand(i32x4_t& rs, uint32_t (&o)[LOADS], uint64_t& b,
                                               int64_t& left, uint32_t& step, const void* base,
                                               int col0, uint32_t ld_bytes, int64_t bytes) {
  static_assert(W >= 128, "the row swizzle of a k-major stage spans 16 chunks");
  kmajor_offsets<W, LOADS, C::NT>(o, col0, ld_bytes);
  b = reinterpret_cast<uint64_t>(base);
  left = bytes;
  step = BK * ld_bytes;
  rs = rsrc4(base, clamp_bytes(bytes));
}

// The issue side: walks the k-steps of a workgroup's tiles (first, first +
// nb, ... below total) and loads them into ring stages. Past the last step it
// loads that step again into stages nobody reads.
template <class C, bool AKM, bool BKM, class NextOps>
struct Loader {
  Ops16<C> op;
  NextOps& next_ops;
  uint32_t lds0;
  int ti, nb, total, ki, wave;
  bool more;
  static constexpr int NL = C::A_LOADS + C::B_LOADS;

  __device__ Loader(NextOps& n, uint32_t l0, int first, int nb_, int total_, int wave_)
      : next_ops(n), lds0(l0), ti(first), nb(nb_), total(total_), ki(0), wave(wave_), more(true) {
    next_ops(ti, op);
  }
  // load i of NL of the current k-step into stage st
  __device__ __forceinline__ void load(int st, int i) {
    const uint32_t base =
        __builtin_amdgcn_readfirstlane(lds0 + (st * C::STAGE + wave * 8 * BK) * 2);
    const uint32_t kn = static_cast<uint32_t>(ki) * (BK * 2);
    const bool last = ki == op.nk - 1;
    if (i < C::A_LOADS) {
      const uint32_t v = AKM ? op.ao[i] : ((op.ao[i] + kn) | (last ? op.tail_a : 0u));
      dma16(op.ra, v, base + i * C::RPP * BK * 2);
    } else {
      const int j = i - C::A_LOADS;
      const uint32_t v = BKM ? op.bo[j] : ((op.bo[j] + kn) | (last ? op.tail_b : 0u));
      const uint32_t at = base + C::BM * BK * 2 + j * C::RPP * BK * 2;
      if constexpr (C::B_NT)
        dma16_nt(op.rb, v, at);
      else
        dma16(op.rb, v, at);
    }
  }
  __device__ __forceinline__ void advance() {
    if (!more) return;
    if (++ki < op.nk) {
      if constexpr (AKM) {
        op.base_a += op.step_a;
        op.left_a -= op.step_a;
        op.ra = rsrc4(reinterpret_cast<const void*>(op.base_a), clamp_bytes(op.left_a));
      }
      if constexpr (BKM) {
        op.base_b += op.step_b;
        op.left_b -= op.step_b;
        op.rb = rsrc4(reinterpret_cast<const void*>(op.base_b), clamp_bytes(op.left_b));
      }
      return;
    }
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

// Fragment reads of sub-step kk (16 k) of a stage.
template <class C, bool AKM>
__device__ __forceinline__ bf16x8_t frag_a(const uint16_t* lds, int st, int row, int kk, int lane) {
  const uint16_t* s = lds + st * C::STAGE;
  if constexpr (AKM)
    return frag_kmajor<C::BM>(lds_addr(s), row, kk * 16, lane);
  else
    return *reinterpret_cast<const bf16x8_t*>(s + lds_off(row + (lane & 31), kk * 2 + (lane >> 5)));
}
template <class C, bool BKM>
__device__ __forceinline__ bf16x8_t frag_b(const uint16_t* lds, int st, int row, int kk, int lane) {
  const uint16_t* s = lds + st * C::STAGE + C::BM * BK;
  if constexpr (BKM)
    return frag_kmajor<C::BN>(lds_addr(s), row, kk * 16, lane);
  else
    return *reinterpret_cast<const bf16x8_t*>(s + lds_off(row + (lane & 31), kk * 2 + (lane >> 5)));
}

// acc (+)= the product of two fragments. SWAP: the B fragment goes first and
// acc holds the transposed tile (lane l: row l % 32 of A's side, four runs of
// four adjacent columns); without it lane l holds column l % 32 and rows
// acc_row(l, r).
template <class T, bool SWAP>
__device__ __forceinline__ f32x16_t mma16(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return SWAP ? T::mfma(b, a, c) : T::mfma(a, b, c);
}

// Output through LDS: the fragments' layout gives a lane 4 adjacent columns of
// its row, which as stores would be 16-byte pieces of 32 rows. 32 rows of PJ of
// a wave's 32-column parts at a time pass through its part of LDS (fp32, 16-byte
// chunks XOR-swizzled with the row, free of bank conflicts both ways), and come
// back as 8 adjacent columns of one row per lane: with 64 columns whole 128-byte
// lines for 16-bit outputs.
template <class C, int PJ = C::NJ>
struct RowPasses {
  static_assert(C::NJ % PJ == 0, "whole parts");
  static constexpr int COLS = PJ * 32;
  static constexpr int CPR = COLS / 4;             // chunks of a row
  static constexpr int LPR = COLS / 8;             // lanes of a row
  static constexpr int RPP = 64 / LPR;             // rows of a pass
  static constexpr int N = 32 / RPP;               // passes over 32 rows
  static constexpr int PARTS = C::NJ / PJ;         // column parts of a wave
  static constexpr int FLOATS = 32 * COLS;         // LDS floats per wave

  // row (0..31) and first column (within the part's) of this lane in pass p
  __device__ static int row(int p, int lane) { return p * RPP + lane / LPR; }
  __device__ static int col(int lane) { return (lane % LPR) * 8; }

  __device__ static void put(float* stage, int lane, const f32x16_t (&acc)[C::NJ], int part = 0) {
    const int r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int nj = 0; nj < PJ; ++nj)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = (nj * 8 + 2 * g + h) ^ (r & (CPR - 1));
        const f32x16_t& x = acc[part * PJ + nj];
        const f32x4_t v = {x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]};
        *reinterpret_cast<f32x4_t*>(stage + r * COLS + c * 4) = v;
      }
  }
  __device__ static void get(const float* stage, int lane, int p, float (&v)[8]) {
    const int r = row(p, lane), c = (lane % LPR) * 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4_t x =
          *reinterpret_cast<const f32x4_t*>(stage + r * COLS + ((c + i) ^ (r & (CPR - 1))) * 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = x[j];
    }
  }
};
// Passes that fit the waves' parts of one ring stage (8 waves).
template <class C>
using StagePasses =
    RowPasses<C, (C::NWAVES * 32 * C::WN * 4 <= C::STAGE * 2 ? C::NJ : C::NJ / 2)>;

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// ---- tiles of the last round, split along the contraction
//
// Tiles run in rounds of one per workgroup, and the last round's may be few. The
// first `whole` tiles run whole; each of the others is shared by `splits`
// workgroups, whose fp32 partial tiles meet in memory: the last to arrive adds
// them in split order (so the sum does not depend on who is last).
struct Tail {
  int whole, splits;
  float* part;     // [(unit - whole)][BM * BN]
  int32_t* count;  // [tile - whole], zero before and after
};
struct Unit {
  int tile, s, splits;
};
__device__ __forceinline__ Unit unit_of(const Tail& t, int unit) {
  if (unit < t.whole) return {unit, 0, 1};
  const int v = unit - t.whole, q = v / t.splits;
  return {t.whole + q, v - q * t.splits, t.splits};
}
// k-steps [k0, k1) of split s.
struct KRange {
  int k0, k1;
};
__device__ __forceinline__ KRange split_range(int nk, int s, int splits) {
  return {static_cast<int>(int64_t(nk) * s / splits),
          static_cast<int>(int64_t(nk) * (s + 1) / splits)};
}
// Number of splits for `rest` tiles of nk k-steps on `slots` workgroups, by time
// in microseconds: `step` per k-step, and to share a tile its partial sums'
// way to memory and back, `kb` KB at the measured 22 (out) and 30 (in) KB/us of
// one CU.
inline __host__ __device__ int tail_splits(int rest, int nk, int slots, float step, float kb) {
  if (rest <= 0) return 1;
  int best = 1;
  float least = nk * step;
  for (int s = 2; s <= slots / rest && s <= 8 && s <= nk; ++s) {
    const float us = (nk + s - 1) / s * step + kb * (1.0f / 22.0f + s * (1.0f / 30.0f));
    if (us < least) {
      least = us;
      best = s;
    }
  }
  return best;
}
// Called by all threads of the workgroup at a unit's end. True where acc holds
// the tile's sum. `flag`: an int in LDS.
//
// The workgroups may run on different XCDs, whose L2s are not coherent with each
// other: partial sums are written through to memory and read from it (device
// scope, the sc1 bit), so waiting for the stores is all the ordering there is to
// do. Fences around plain stores write back and invalidate a whole L2 each: an
// update of 1408 x 2816 took 888 us with them, 329 so.
constexpr int kDevice = 16;  // sc1
template <class C>
__device__ __forceinline__ bool join_splits(f32x16_t (&acc)[C::MI][C::NJ], const Tail& t, int unit,
                                            const Unit& u, int* flag) {
  if (u.splits == 1) return true;
  constexpr int BYTES = C::BM * C::BN * 4;
  // the thread's 16-byte pieces at i * NT * 16 (a scalar offset: addresses in
  // vector registers would push the k-loop's out)
  auto rsrc = [&](int v) {
    return __builtin_amdgcn_make_buffer_rsrc(
        reinterpret_cast<char*>(t.part) + int64_t(v) * BYTES, 0, BYTES, 0x00020000);
  };
  const int off = threadIdx.x * 16;
  const auto mine = rsrc(unit - t.whole);
#pragma unroll
  for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
    for (int nj = 0; nj < C::NJ; ++nj)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4_t v = {acc[mi][nj][4 * q], acc[mi][nj][4 * q + 1], acc[mi][nj][4 * q + 2],
                           acc[mi][nj][4 * q + 3]};
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), mine, off,
                                               ((mi * C::NJ + nj) * 4 + q) * C::NT * 16, kDevice);
      }
  vm_wait<0>();  // the wave's partial sums have reached memory before the count
  lds_barrier();
  if (threadIdx.x == 0) *flag = atomicAdd(t.count + (u.tile - t.whole), 1);
  lds_barrier();
  if (*flag != u.splits - 1) return false;
  zero_acc<C>(acc);
  for (int s = 0; s < u.splits; ++s) {
    const auto other = rsrc(unit - t.whole - u.s + s);
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
      for (int nj = 0; nj < C::NJ; ++nj)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4_t v = __builtin_bit_cast(
              f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                           other, off, ((mi * C::NJ + nj) * 4 + q) * C::NT * 16, kDevice));
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[mi][nj][4 * q + j] += v[j];
        }
  }
  if (threadIdx.x == 0) t.count[u.tile - t.whole] = 0;
  return true;
}

// Ring loop for small tiles: NST stages, loads NST - 1 k-steps ahead, the
// fragments of sub-step kk + 1 read between the MFMAs of sub-step kk, one
// barrier per k-step (before its last sub-step, whose fragments are already
// in registers). LDS: C::LDS_ELEMS for the ring, then the waves' output stages.
template <class C, class T, bool AKM, bool BKM, bool SWAP, class NextOps, class Epilogue>
__device__ __forceinline__ void stream_ring(uint16_t* lds, int first, int nb, int total,
                                            NextOps&& next_ops, Epilogue&& epilogue) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  constexpr int NST = C::NST, NL = C::A_LOADS + C::B_LOADS, INFLIGHT = NL * (NST - 2);
  constexpr int NR = C::MI + C::NJ, NM = C::MI * C::NJ;
  static_assert(INFLIGHT <= 63, "vmcnt range");
  Loader<C, AKM, BKM, std::remove_reference_t<NextOps>> ld(next_ops, lds_addr(lds), first, nb,
                                                            total, wave);
  bf16x8_t af[2][C::MI], bfr[2][C::NJ];
  auto rd = [&](int st, int kk, int buf, int i) {
    if (i < C::NJ)
      bfr[buf][i] = frag_b<C, BKM>(lds, st, wn * C::WN + i * 32, kk, lane);
    else
      af[buf][i - C::NJ] = frag_a<C, AKM>(lds, st, wm * C::WM + (i - C::NJ) * 32, kk, lane);
  };
  f32x16_t acc[C::MI][C::NJ];
  auto sub = [&](int buf, int st_rd, int kk_rd, bool dma, int st_dma) {
    constexpr int RPS = (NR + NM - 1) / NM, LPS = (NL + NM - 1) / NM;
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      const int mi = i / C::NJ, nj = i % C::NJ;
      acc[mi][nj] = mma16<T, SWAP>(af[buf][mi], bfr[buf][nj], acc[mi][nj]);
#pragma unroll
      for (int q = 0; q < RPS; ++q)
        if (i * RPS + q < NR) rd(st_rd, kk_rd, buf ^ 1, i * RPS + q);
      if (dma) {
#pragma unroll
        for (int q = 0; q < LPS; ++q)
          if (i * LPS + q < NL) ld.load(st_dma, i * LPS + q);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int j = 0; j < NST - 1; ++j) {
#pragma unroll
    for (int i = 0; i < NL; ++i) ld.load(j, i);
    ld.advance();
  }
  vm_wait<INFLIGHT>();
  lds_barrier();
  int st = 0, sti = NST - 1;
#pragma unroll
  for (int i = 0; i < NR; ++i) rd(st, 0, 0, i);
  for (int tc = first; tc < total; tc += nb) {
    zero_acc<C>(acc);
    const int nkc = epilogue.k_steps(tc);
    for (int kc = 0; kc < nkc; ++kc) {
      sub(0, st, 1, true, sti);
      ld.advance();
      sub(1, st, 2, false, 0);
      sub(0, st, 3, false, 0);
      vm_wait<INFLIGHT>();
      lds_barrier();
      st = st == NST - 1 ? 0 : st + 1;
      sti = sti == NST - 1 ? 0 : sti + 1;
      sub(1, st, 0, false, 0);
    }
    epilogue(tc, wm, wn, lane, acc,
             reinterpret_cast<float*>(lds + C::LDS_ELEMS) + wave * RowPasses<C>::FLOATS);
  }
  vm_wait<0>();
}

// Two-phase loop for 256 x 256 tiles in 8 waves: the waves of one half
// multiply (8 MFMAs) while those of the other half read the next sub-step's
// fragments and issue loads, then they swap, so each SIMD's matrix core has
// work in every phase. Two stages of 64 KB: the loads of step k + 1 go out in
// the first two memory phases of step k, or the first three where B's
// transposing reads make these longer (12288 rows, 4096 x 7168, input gradient:
// 654 us with two, 647 with three; 24576 rows over 64 groups of 2816 x 2048: 413
// and 397; forward of the first: 579 and 586), and are waited for in its last.
//
// Rows of a tile past its data are multiplied all the same: leaving out waves
// whose part of the tile is empty took as long (the loads set the pace there),
// and a branch per 32-row part twice as long (the accumulators were copied).
//
// The halves fall into step again for a tile's epilogue: staggered, each half
// would wait at a barrier for the other's stores.
//
// Why the stages are safe: within a tile the second half runs one phase behind
// (its extra barrier before the k-loop; the first half's after it). A stage is read in the
// memory phases of its step, each of which ends with lgkmcnt(0) before its
// barrier. Step k + 1's loads overwrite the stage of step k - 1; the first
// half issues them after the barrier that ends the second half's last memory
// phase of step k - 1. Every wave waits for its own loads in its last memory
// phase of step k, and the first half's first read of step k + 1 comes one
// barrier after the second half's wait. The output stages lie in the stage of
// the tile's last step, which every wave has read when the halves are in step;
// the barrier after the epilogue keeps the next loads out of it until then.
template <class C, class T, bool AKM, bool BKM, bool SWAP, class NextOps, class Epilogue>
__device__ __forceinline__ void stream_phased(uint16_t* lds, int first, int nb, int total,
                                              NextOps&& next_ops, Epilogue&& epilogue) {
  static_assert(C::NWAVES == 8 && C::NST == 2, "two halves of four waves, two stages");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  constexpr int NL = C::A_LOADS + C::B_LOADS;
  constexpr int PARTS = BKM && !AKM ? 3 : 2, PER = (NL + PARTS - 1) / PARTS;
  Loader<C, AKM, BKM, std::remove_reference_t<NextOps>> ld(next_ops, lds_addr(lds), first, nb,
                                                            total, wave);
  bf16x8_t af[C::MI], bfr[C::NJ];
  f32x16_t acc[C::MI][C::NJ];
#pragma unroll
  for (int i = 0; i < NL; ++i) ld.load(0, i);
  ld.advance();
  vm_wait<0>();
  lds_barrier();
  int st = 0;
  for (int tc = first; tc < total; tc += nb) {
    zero_acc<C>(acc);
    const int nkc = epilogue.k_steps(tc);
    if (wave >= 4) __builtin_amdgcn_s_barrier();
    for (int kc = 0; kc < nkc; ++kc) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
        for (int i = 0; i < C::NJ; ++i)
          bfr[i] = frag_b<C, BKM>(lds, st, wn * C::WN + i * 32, kk, lane);
#pragma unroll
        for (int i = 0; i < C::MI; ++i)
          af[i] = frag_a<C, AKM>(lds, st, wm * C::WM + i * 32, kk, lane);
        if (kk < PARTS) {
#pragma unroll
          for (int i = kk * PER; i < (kk + 1) * PER && i < NL; ++i) ld.load(st ^ 1, i);
          if (kk == PARTS - 1) ld.advance();
        }
        if (kk == 3) vm_wait<0>();
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
          for (int nj = 0; nj < C::NJ; ++nj)
            acc[mi][nj] = mma16<T, SWAP>(af[mi], bfr[nj], acc[mi][nj]);
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
      }
      st ^= 1;
    }
    if (wave < 4) __builtin_amdgcn_s_barrier();
    // the stage just read is free until the next tile's first loads
    static_assert(8 * StagePasses<C>::FLOATS * 4 <= C::STAGE * 2, "output stages fit");
    epilogue(tc, wm, wn, lane, acc,
             reinterpret_cast<float*>(lds + (st ^ 1) * C::STAGE) + wave * StagePasses<C>::FLOATS);
    lds_barrier();
  }
  vm_wait<0>();
}

}  // namespace
}  // namespace dsmoe
