// Tokens sorted by expert (definition in dsmoe_tokens.h): a stable counting sort
// of the (token, slot) pairs, and the rows moved to their places.
//
// Rows are bytes here: a token's row is read once and written to its K places, 16
// bytes per lane of a group of LANES lanes. Few pairs take one launch: every
// group counts the pairs before its own over all selections (from L2). More pairs
// take three: places within chunks of 1024 pairs, a scan of the chunks' counts,
// then the rows.
#include "device_common.h"
#include "internal.h"
#include "row_io.h"

namespace dsmoe {

namespace {

constexpr int kMaxExperts = 512, kMaxK = 64;
constexpr int kChunk = 1024;  // pairs whose places one workgroup finds

typedef uint32_t u32x4_any1_t __attribute__((ext_vector_type(4), aligned(1)));

struct MoveArgs {
  const int32_t* idx;
  int32_t* offsets;
  int32_t* perm;
  int32_t* inv;
  const uint8_t* x;   // NULL: sort only
  const uint8_t* x2;  // second rows (tile scales) or NULL
  uint8_t* xp;
  uint8_t* xp2;
  int64_t t0, T;  // tokens t0 .. T - 1 of this launch's groups
  int64_t pairs, rows, ldt, ldp;
  int row_bytes, row2_bytes;  // (below 2^31: d * 4 is)
  int E, K;
  bool stream;
  // the sort's tables (many pairs)
  const int32_t* base;   // [chunks][E] place of a chunk's first pair of an expert
  const uint16_t* rank;  // [pairs] place of a pair among its chunk's of its expert
};

// Copies one row to the places that exist, by LANES lanes; lane k of a wave holds slot
// k's in `at`. The whole wave sweeps on or ends: places come out of lanes that may hold
// no piece of the row.
template <int LANES, bool STREAM>
__device__ __forceinline__ void move_row(const uint8_t* src, uint8_t* dst, int bytes, int64_t ldp,
                                         int32_t at, int K, int lane) {
  constexpr int CH = 4;  // 16-byte pieces of a lane in flight
  const int whole = bytes / 16;
  int w0 = __builtin_amdgcn_readfirstlane(lane >> 6) * 64;
  for (int c0 = lane; w0 < whole; w0 += CH * LANES, c0 += CH * LANES) {
    u32x4_any1_t v[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (c0 + i * LANES < whole)
        v[i] = *reinterpret_cast<const u32x4_any1_t*>(src + (c0 + i * LANES) * 16);
    for (int k = 0; k < K; ++k) {
      const int p = __builtin_amdgcn_readlane(at, k);
      if (p < 0) continue;
      uint8_t* d = dst + p * ldp;
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (c0 + i * LANES < whole) {
          auto* q = reinterpret_cast<u32x4_any1_t*>(d + (c0 + i * LANES) * 16);
          if constexpr (STREAM)
            __builtin_nontemporal_store(v[i], q);
          else
            *q = v[i];
        }
    }
  }
  const int tail = bytes - whole * 16;
  if (tail == 0) return;
  const uint8_t v = lane < tail ? src[whole * 16 + lane] : 0;
  for (int k = 0; k < K; ++k) {
    const int p = __builtin_amdgcn_readlane(at, k);
    if (p >= 0 && lane < tail) dst[p * ldp + whole * 16 + lane] = v;
  }
}

template <int LANES>
__device__ __forceinline__ void move_token(const MoveArgs& a, int64_t t, const int32_t* pos,
                                           int lane) {
  if (!a.x) return;
  const int32_t at = (lane & 63) < a.K ? pos[lane & 63] : -1;
  const uint8_t* x = a.x + t * a.ldt;
  if (a.stream)
    move_row<LANES, true>(x, a.xp, a.row_bytes, a.ldp, at, a.K, lane);
  else
    move_row<LANES, false>(x, a.xp, a.row_bytes, a.ldp, at, a.K, lane);
  if (a.x2)
    move_row<LANES, false>(a.x2 + t * a.row2_bytes, a.xp2, a.row2_bytes, a.row2_bytes, at, a.K,
                           lane);
}

// Sum over the wave, the same for all lanes.
__device__ __forceinline__ int wave_sum_int(int v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += wave_shfl_xor(v, m);
  return v;
}

// Few pairs: block t < T places and moves token t's row; block T writes offsets
// and the end of perm. Latency-bound (a launch, selections from L2, the row): 64 tokens
// to 8 of 256 experts 6.8 us with rows of 2048 bf16 values, 6.7 with 64.
constexpr int kFewThreads = 256, kFewK = 8;
constexpr int kFewLoads = 4;  // selections of a thread in flight
__global__ __launch_bounds__(kFewThreads) void dispatch_few_kernel(MoveArgs a) {
  const int tid = threadIdx.x;
  const int n = static_cast<int>(a.pairs), E = a.E, K = a.K;
  if (blockIdx.x == a.T) {
    __shared__ int32_t count[kMaxExperts];
    for (int e = tid; e < kMaxExperts; e += kFewThreads) count[e] = 0;
    __syncthreads();
    for (int q = tid; q < n; q += kFewThreads) {
      const int e = a.idx[q];
      if (static_cast<uint32_t>(e) < static_cast<uint32_t>(E)) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    if (tid < 64) {  // eight experts per lane, then over the lanes
      int c[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = sum += count[8 * tid + j];
      int p = sum;
#pragma unroll
      for (int s = 1; s < 64; s <<= 1) {
        const int o = __shfl_up(p, s, 64);
        if (tid >= s) p += o;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) count[8 * tid + j] = p - sum + c[j];
    }
    __syncthreads();
    const int rows = static_cast<int>(a.rows);
    for (int e = tid; e <= E; e += kFewThreads) a.offsets[e] = e ? min(count[e - 1], rows) : 0;
    for (int r = count[E - 1] + tid; r < rows; r += kFewThreads) a.perm[r] = -1;
    return;
  }
  __shared__ int32_t pos[kFewK];
  __shared__ int32_t part[kFewThreads / 64][kFewK];
  const int t = blockIdx.x;
  int ex[kFewK], before[kFewK] = {};
#pragma unroll
  for (int j = 0; j < kFewK; ++j) {
    const int e = j < K ? a.idx[t * K + j] : -1;
    ex[j] = static_cast<uint32_t>(e) < static_cast<uint32_t>(E) ? e : -1;
  }
  for (int q0 = tid; q0 < n; q0 += kFewLoads * kFewThreads) {
    int e[kFewLoads];
#pragma unroll
    for (int i = 0; i < kFewLoads; ++i) {
      const int q = q0 + i * kFewThreads;
      e[i] = q < n ? a.idx[q] : -1;
    }
#pragma unroll
    for (int i = 0; i < kFewLoads; ++i) {
      const int q = q0 + i * kFewThreads;
      if (static_cast<uint32_t>(e[i]) < static_cast<uint32_t>(E)) {
#pragma unroll
        for (int j = 0; j < kFewK; ++j)
          before[j] += e[i] < ex[j] || (e[i] == ex[j] && q < t * K + j);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kFewK; ++j) {
    const int s = wave_sum_int(before[j]);
    if ((tid & 63) == 0) part[tid >> 6][j] = s;
  }
  __syncthreads();
  if (tid < K) {
    int p = part[0][tid];
#pragma unroll
    for (int w = 1; w < kFewThreads / 64; ++w) p += part[w][tid];
    const int e = a.idx[t * K + tid];
    if (static_cast<uint32_t>(e) >= static_cast<uint32_t>(E) || p >= a.rows) p = -1;
    pos[tid] = p;
    a.inv[t * K + tid] = p;
    if (p >= 0) a.perm[p] = t;
  }
  __syncthreads();
  move_token<kFewThreads>(a, t, pos, tid);
}

// Many pairs, first launch: block c finds for the pairs of chunk c how many
// earlier ones of the chunk have the same expert, and counts the chunk's pairs by
// expert. Lanes of a wave with the same expert find each other bit by bit: no atomics,
// so the order is the definition's.
__global__ __launch_bounds__(kChunk) void rank_kernel(const int32_t* idx, int64_t pairs, int E,
                                                      int32_t* count, uint16_t* rank) {
  constexpr int WAVES = kChunk / 64;
  __shared__ uint16_t seen[WAVES][kMaxExperts];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < WAVES * kMaxExperts / 2; i += kChunk)
    reinterpret_cast<uint32_t*>(&seen[0][0])[i] = 0;
  const int64_t p = int64_t(blockIdx.x) * kChunk + tid;
  const int e = p < pairs ? idx[p] : -1;
  const bool there = static_cast<uint32_t>(e) < static_cast<uint32_t>(E);
  uint64_t same = __ballot(there);
#pragma unroll
  for (int b = 0; b < 9; ++b) {
    const uint64_t has = __ballot((e >> b) & 1);
    same &= (e >> b) & 1 ? has : ~has;
  }
  const int before = __popcll(same & ((uint64_t(1) << lane) - 1));
  __syncthreads();
  if (there && before == 0) seen[wave][e] = static_cast<uint16_t>(__popcll(same));
  __syncthreads();
  if (tid < E) {
    int run = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const int c = seen[w][tid];
      seen[w][tid] = static_cast<uint16_t>(run);
      run += c;
    }
    count[int64_t(blockIdx.x) * E + tid] = run;
  }
  __syncthreads();
  if (there) rank[p] = static_cast<uint16_t>(seen[wave][e] + before);
}

// Second launch, one block: the chunks' counts become the places of their first
// pairs. Threads of a column (expert) take a run of PER chunks each, whose counts stay
// in registers (PER 0: runs of any length, read twice). Latency-bound: one block, so that
// nothing but its own barriers stands between counts and places; sorting 8192 x 8 pairs
// over 256 experts takes 10 us in all, 32768 x 8 21.
template <int PER>
__global__ __launch_bounds__(1024) void scan_kernel(int32_t* count, int chunks, int E, int cols,
                                                    int64_t rows, int32_t* offsets) {
  __shared__ int32_t part[1024];
  __shared__ __attribute__((aligned(16))) int32_t first[kMaxExperts + 4];
  const int tid = threadIdx.x, runs = 1024 / cols;  // cols: a power of two, at least E
  const int e = tid & (cols - 1), run = tid / cols;
  const int per = PER ? PER : (chunks + runs - 1) / runs, c0 = min(run * per, chunks),
            c1 = e < E ? min(c0 + per, chunks) : 0;
  int32_t* col = count + e;
  constexpr int N = PER ? PER : 8;  // loads in flight
  int32_t n[N];
  auto read = [&](int c) {
#pragma unroll
    for (int i = 0; i < N; ++i) n[i] = c + i < c1 ? col[int64_t(c + i) * E] : 0;
  };
  int sum = 0;
  for (int c = c0; c < (PER ? c0 + 1 : c1); c += N) {
    read(c);
#pragma unroll
    for (int i = 0; i < N; ++i) sum += n[i];
  }
  part[tid] = sum;
  if (tid < kMaxExperts) first[tid] = 0;
  __syncthreads();
  int at = 0;  // pairs of this expert in the runs before this thread's
  if (e < E) {
    int all = 0;
#pragma unroll 4
    for (int r = 0; r < runs; ++r) {
      const int v = part[r * cols + e];
      at += r < run ? v : 0;
      all += v;
    }
    if (run == 0) first[e] = all;
  }
  __syncthreads();
  if (tid < 64) {  // scan of the experts' pairs, eight experts per lane
    int4 lo = reinterpret_cast<const int4*>(first)[2 * tid];
    int4 hi = reinterpret_cast<const int4*>(first)[2 * tid + 1];
    const int v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    int all = 0, c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = all;
      all += v[j];
    }
    int p = all;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int o = __shfl_up(p, s, 64);
      if (tid >= s) p += o;
    }
    p -= all;
    reinterpret_cast<int4*>(first)[2 * tid] = make_int4(p + c[0], p + c[1], p + c[2], p + c[3]);
    reinterpret_cast<int4*>(first)[2 * tid + 1] = make_int4(p + c[4], p + c[5], p + c[6], p + c[7]);
    if (tid == 63) first[kMaxExperts] = p + all;
  }
  __syncthreads();
  for (int i = tid; i <= E; i += 1024)
    offsets[i] = static_cast<int32_t>(min(int64_t(first[i]), rows));
  if (e >= E) return;
  at += first[e];
  for (int c = c0; c < (PER ? c0 + 1 : c1); c += N) {
    if (!PER) read(c);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c + i < c1) {
        col[int64_t(c + i) * E] = at;
        at += n[i];
      }
  }
}

// Third launch: a group of LANES lanes per token. Bound by stores: 8192 E4M3 rows of 7168
// to 8 experts each, 58 MB read and 485 written, 96 us, 5.7 TB/s, 22 KB/us for each CU; a
// workgroup per place that reads its row instead took 160, as rows then come out of the
// caches eight times.
template <int LANES>
__global__ __launch_bounds__(256) void move_kernel(MoveArgs a) {
  constexpr int GROUPS = 256 / LANES;
  __shared__ int32_t places[GROUPS][kMaxK];
  const int lane = threadIdx.x & (LANES - 1), group = threadIdx.x / LANES;
  const int64_t t = a.t0 + int64_t(blockIdx.x) * GROUPS + group;
  const bool real = t < a.T;
  if (real && lane < a.K) {
    const int64_t p = t * a.K + lane;
    const int e = a.idx[p];
    int32_t at = -1;
    if (static_cast<uint32_t>(e) < static_cast<uint32_t>(a.E)) {
      at = a.base[p / kChunk * a.E + e] + a.rank[p];
      if (at >= a.rows) at = -1;
    }
    places[group][lane] = at;
    a.inv[p] = at;
    if (at >= 0) a.perm[at] = static_cast<int32_t>(t);
    // places behind the last pair
    if (p < a.rows && p >= a.offsets[a.E]) a.perm[p] = -1;
  }
  __syncthreads();
  if (real) move_token<LANES>(a, t, places[group], lane);
}

// The same without rows: a thread per pair.
__global__ __launch_bounds__(256) void place_kernel(MoveArgs a) {
  const int64_t p = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (p >= a.pairs) return;
  const int e = a.idx[p];
  int32_t at = -1;
  if (static_cast<uint32_t>(e) < static_cast<uint32_t>(a.E)) {
    at = a.base[p / kChunk * a.E + e] + a.rank[p];
    if (at >= a.rows) at = -1;
  }
  a.inv[p] = at;
  if (at >= 0) a.perm[at] = static_cast<int32_t>(p / a.K);
  if (p < a.rows && p >= a.offsets[a.E]) a.perm[p] = -1;
}

// No pairs at all.
__global__ __launch_bounds__(256) void no_pairs_kernel(int32_t* offsets, int E) {
  for (int e = threadIdx.x; e <= E; e += 256) offsets[e] = 0;
}

// Whether the pairs are few: every token's group reads all selections. Measured with
// rows of 2048 bf16 values over 256 experts, one launch / three (us, replayed graphs):
//   T x K  64 x 8    6.8 /  9.3     256 x 8   9.7 / 10.2     512 x 8  13.9 / 11.5
//                                   512 x 4   9.3 /  9.8    1024 x 4  14.7 / 11.6
//                                  1024 x 1   7.9 /  9.1    2048 x 1  13.5 / 10.2
// More than eight slots would read them again for every eight (64 x 16: 12.2 / 10.6).
bool few(int64_t T, int K) { return K <= kFewK && T <= 1024 && T * K <= 2048; }

int64_t chunks_of(int64_t pairs) { return (pairs + kChunk - 1) / kChunk; }

}  // namespace

size_t dispatch_workspace(int64_t T, int K, int E) {
  if (few(T, K)) return 0;
  const int64_t pairs = T * K;
  return static_cast<size_t>((chunks_of(pairs) * E * 4 + 15) / 16 * 16 + pairs * 2);
}

hipError_t launch_dispatch(const DispatchArgs& p, void* ws, hipStream_t s) {
  const int64_t pairs = p.T * p.K;
  if (pairs == 0) {
    hipLaunchKernelGGL(no_pairs_kernel, dim3(1), dim3(256), 0, s, p.offsets, p.E);
    return hipGetLastError();
  }
  MoveArgs a{};
  a.idx = p.idx;
  a.offsets = p.offsets;
  a.perm = p.perm;
  a.inv = p.inv;
  a.x = p.x;
  a.x2 = p.x2;
  a.xp = p.xp;
  a.xp2 = p.xp2;
  a.T = p.T;
  a.pairs = pairs;
  a.rows = p.rows;
  a.row_bytes = static_cast<int>(p.row_bytes);
  a.row2_bytes = static_cast<int>(p.row2_bytes);
  a.ldt = p.ldt;
  a.ldp = p.ldp;
  a.E = p.E;
  a.K = p.K;
  a.stream = p.rows * p.row_bytes >= kFarBytes;
  if (few(p.T, p.K)) {
    hipLaunchKernelGGL(dispatch_few_kernel, dim3(static_cast<unsigned>(p.T + 1)), dim3(kFewThreads),
                       0, s, a);
    return hipGetLastError();
  }
  const int64_t chunks = chunks_of(pairs);
  int32_t* count = static_cast<int32_t*>(ws);
  uint16_t* rank = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) +
                                               (chunks * p.E * 4 + 15) / 16 * 16);
  a.base = count;
  a.rank = rank;
  int cols = 64;
  while (cols < p.E) cols *= 2;
  hipLaunchKernelGGL(rank_kernel, dim3(static_cast<unsigned>(chunks)), dim3(kChunk), 0, s, p.idx,
                     pairs, p.E, count, rank);
  const int runs = 1024 / cols;
  auto scan = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(1), dim3(1024), 0, s, count, static_cast<int>(chunks), p.E, cols,
                       p.rows, p.offsets);
  };
  // (the whole sort in us, scan_kernel<4> / <16> / <0>: 4096 x 8 pairs over 64 experts
  // 8.7 / 9.5 / 9.3; 8192 x 8 over 256 - / 10.2 / 11.3)
  if (chunks <= 4 * runs)
    scan(scan_kernel<4>);
  else if (chunks <= 16 * runs)
    scan(scan_kernel<16>);
  else
    scan(scan_kernel<0>);
  if (!p.x) {
    hipLaunchKernelGGL(place_kernel, dim3(static_cast<unsigned>((pairs + 255) / 256)), dim3(256), 0,
                       s, a);
    return hipGetLastError();
  }
  // a wave takes rows that its lanes hold in one piece each: 8192 tokens to 8 experts,
  // rows of 256 bytes 14 us (a block per token 18), of 1 KB 21 (22), of 2 KB 33 (33),
  // of 8 KB, 4096 tokens, 67 (61)
  const bool narrow = p.row_bytes <= 1024;
  const int64_t per = kMaxBlocks * (narrow ? 4 : 1);
  for (int64_t t = 0; t < p.T; t += per) {
    a.t0 = t;
    const int64_t n = p.T - t < per ? p.T - t : per;
    a.T = t + n;
    if (narrow)
      hipLaunchKernelGGL(move_kernel<64>, dim3(static_cast<unsigned>((n + 3) / 4)), dim3(256), 0, s,
                         a);
    else
      hipLaunchKernelGGL(move_kernel<256>, dim3(static_cast<unsigned>(n)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace dsmoe
