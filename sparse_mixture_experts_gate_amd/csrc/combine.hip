// Sorted rows back to their tokens with weights, and the gradients of that
// (definitions in dsmoe_tokens.h).
//
// Memory-bound: a group of LANES lanes owns a token, 8 adjacent values per lane
// and chunk; its places and weights are wave-uniform, and the rows of up to eight
// places are in flight together. 8192 x 8 rows of 7168 bf16 values: 205 us, 1.06 GB at
// 5.2 TB/s; the gradients 398 us, 2.0 GB at 5.0. Few tokens: latency; gradients of 64 x 8
// rows of 4096 by 256 lanes a token 8.7 us, with one place's row at a time 9.9.
#include "device_common.h"
#include "internal.h"
#include "row_io.h"

namespace dsmoe {

namespace {

constexpr int kMaxK = 64;

struct TokArgs {
  const void* yp;
  const int32_t* inv;
  const float* w;
  const void* base;  // forward: base; backward: dy
  void* y;           // forward: y; backward: dy_perm
  float* dw;
  int64_t t0, T, rows, ldt, ldp;
  int K, d;
  bool stream;
};

// A token's places: lane k holds slot k's place and weight, `mask` the slots that
// have one.
struct Places {
  int32_t at;
  float w;
  uint64_t mask;
};
__device__ __forceinline__ Places places_of(const TokArgs& a, int64_t t, int lane) {
  Places p{-1, 0.0f, 0};
  if (lane < a.K) {
    p.at = a.inv[t * a.K + lane];
    p.w = a.w ? a.w[t * a.K + lane] : 1.0f;
  }
  p.mask = __ballot(p.at >= 0 && p.at < a.rows);
  return p;
}
__device__ __forceinline__ int next_slot(uint64_t& m) {
  const int k = __builtin_ctzll(m);
  m &= m - 1;
  return k;
}

// A token row's chunk that is loaded before those of its places and put in order behind
// their loads; in front of them, its wait would stand before theirs. With inputs that no
// cache holds, a return of 4096 x 8 rows of 7168 bf16 values, one in eight here, takes 43.0
// us that way and 41.8 so, of 4096 x 6 rows of 2048 30.2 and 28.6, of 8192 x 4 rows of 1408,
// half of them here, 24.5 and 20.4, the gradients of these 31.0 and 29.8; other gradients,
// fp32 rows and few tokens the same within 2%.
template <class T>
struct Early {
  typename RawOf<T>::type raw;
  bool waits = false;
  __device__ __forceinline__ void load(const void* row, int64_t at, int i0, int d) {
    raw = load8(static_cast<const T*>(row) + at, i0, d);
    waits = true;
  }
  __device__ __forceinline__ void get(float (&v)[VEC], int cnt) {
    if (waits) unpack(raw, v, cnt);
    waits = false;
  }
};

// acc += w row over the next N slots, all loads first.
template <class T, int N>
__device__ __forceinline__ void add_rows(const TokArgs& a, const Places& p, uint64_t& m, int i0,
                                         Early<T>& base, float (&acc)[VEC]) {
  typename RawOf<T>::type r[N];
  float w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int k = next_slot(m);
    const int64_t at = __builtin_amdgcn_readlane(p.at, k);
    w[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(p.w), k));
    r[i] = load8(static_cast<const T*>(a.yp) + at * a.ldp, i0, a.d);
  }
  base.get(acc, a.d - i0);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float v[VEC];
    unpack(r[i], v, a.d - i0);
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc[j] = __builtin_fmaf(w[i], v[j], acc[j]);
  }
}

// Threads of a workgroup whose groups of LANES lanes own a token each.
template <int LANES>
constexpr int kThreads = LANES < 256 ? 256 : LANES;

template <class T, int LANES>
__global__ __launch_bounds__(kThreads<LANES>) void token_combine_kernel(TokArgs a) {
  constexpr int GROUPS = kThreads<LANES> / LANES;
  const int lane = threadIdx.x & (LANES - 1);
  const int64_t t = a.t0 + int64_t(blockIdx.x) * GROUPS + threadIdx.x / LANES;
  if (t >= a.T) return;  // whole waves
  const Places p = places_of(a, t, threadIdx.x & 63);
  // The whole wave sweeps on or ends, since places come out of lanes that may hold no
  // values: lanes past the row take its last chunk along and store nothing.
  const int last = (a.d - 1) & ~(VEC - 1);
  for (int s0 = __builtin_amdgcn_readfirstlane(lane >> 6) * 64 * VEC; s0 < a.d;
       s0 += LANES * VEC) {
    const int i0 = min(s0 + static_cast<int>(threadIdx.x & 63) * VEC, last);
    __builtin_assume(i0 < a.d);
    float acc[VEC] = {};
    Early<T> base;
    if (a.base) base.load(a.base, t * a.ldt, i0, a.d);
    uint64_t m = p.mask;
    int left = __popcll(m);
    for (; left >= 8; left -= 8) add_rows<T, 8>(a, p, m, i0, base, acc);
    if (left & 4) add_rows<T, 4>(a, p, m, i0, base, acc);
    if (left & 2) add_rows<T, 2>(a, p, m, i0, base, acc);
    if (left & 1) add_rows<T, 1>(a, p, m, i0, base, acc);
    base.get(acc, a.d - i0);
    if (s0 + static_cast<int>(threadIdx.x & 63) * VEC < a.d)
      store8(static_cast<T*>(a.y) + t * a.ldt + i0, acc, a.d - i0, a.stream);
  }
}

// The gradients of the next N slots for the chunk of dy that a lane holds, all loads
// first; lane k of each wave adds the wave's part of <dy, row> to slot k's `sum`.
template <class T, int N>
__device__ __forceinline__ void grad_rows(const TokArgs& a, const Places& p, uint64_t& m, int i0,
                                          Early<T>& dy, float (&g)[VEC], float& sum) {
  typename RawOf<T>::type r[N];
  int64_t at[N];
  float w[N];
  int k[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    k[i] = next_slot(m);
    at[i] = __builtin_amdgcn_readlane(p.at, k[i]) * a.ldp;
    w[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(p.w), k[i]));
    if (a.dw) r[i] = load8(static_cast<const T*>(a.yp) + at[i], i0, a.d);
  }
  dy.get(g, a.d - i0);
  if (a.dw) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float v[VEC], dot = 0.0f;
      unpack(r[i], v, a.d - i0);
#pragma unroll
      for (int j = 0; j < VEC; ++j) dot = __builtin_fmaf(v[j], g[j], dot);
      dot = wave_sum(dot);
      if (static_cast<int>(threadIdx.x & 63) == k[i]) sum += dot;
    }
  }
  if (a.y && i0 < a.d) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = w[i] * g[j];
      store8(static_cast<T*>(a.y) + at[i] + i0, o, a.d - i0, a.stream);
    }
  }
}

// A chunk of dy's row stays in a lane's registers for all places; longer rows take
// several sweeps over them. A wave's part of slot k's <dy, row> is lane k's; the waves'
// are added through LDS in wave order.
template <class T, int LANES>
__global__ __launch_bounds__(kThreads<LANES>) void token_combine_bwd_kernel(TokArgs a) {
  constexpr int GROUPS = kThreads<LANES> / LANES, WAVES = LANES / 64;
  __shared__ float part[GROUPS][WAVES][kMaxK];
  const int lane = threadIdx.x & (LANES - 1), group = threadIdx.x / LANES;
  const int wave = lane >> 6;
  const int64_t t = a.t0 + int64_t(blockIdx.x) * GROUPS + group;
  const bool real = t < a.T;
  if (real) {
    const Places p = places_of(a, t, threadIdx.x & 63);
    float sum = 0.0f;
    for (int s0 = 0; s0 < a.d; s0 += LANES * VEC) {
      const int i0 = s0 + lane * VEC;
      float g[VEC];
      Early<T> dy;
      dy.load(a.base, t * a.ldt, i0, a.d);
      uint64_t m = p.mask;
      int left = __popcll(m);
      for (; left >= 8; left -= 8) grad_rows<T, 8>(a, p, m, i0, dy, g, sum);
      for (; left >= 4; left -= 4) grad_rows<T, 4>(a, p, m, i0, dy, g, sum);
      for (; left >= 2; left -= 2) grad_rows<T, 2>(a, p, m, i0, dy, g, sum);
      for (; left >= 1; --left) grad_rows<T, 1>(a, p, m, i0, dy, g, sum);
    }
    part[group][wave][threadIdx.x & 63] = sum;
  }
  if (!a.dw) return;
  __syncthreads();
  if (real && lane < a.K) {
    // 1024 lanes are four sweeps of 256 side by side: added as those are one after the
    // other, dweight is the same bits however many tokens there are
    constexpr int FIRST = WAVES < 4 ? WAVES : 4;
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < FIRST; ++w) {
      float q = part[group][w][lane];
#pragma unroll
      for (int j = w + 4; j < WAVES; j += 4) q += part[group][j][lane];
      s = w ? s + q : q;
    }
    a.dw[t * a.K + lane] = s;
  }
}

template <class T, int LANES>
void launch_with(TokArgs a, bool backward, hipStream_t s) {
  constexpr int GROUPS = kThreads<LANES> / LANES;
  // (work items of a launch are counted in 32 bits)
  const int64_t T_ = a.T, per = kMaxBlocks * 256 / kThreads<LANES> * GROUPS;
  for (int64_t t = 0; t < T_; t += per) {
    const int64_t n = T_ - t < per ? T_ - t : per;
    a.t0 = t;
    a.T = t + n;
    const dim3 grid(static_cast<unsigned>((n + GROUPS - 1) / GROUPS)), threads(kThreads<LANES>);
    if (backward)
      hipLaunchKernelGGL((token_combine_bwd_kernel<T, LANES>), grid, threads, 0, s, a);
    else
      hipLaunchKernelGGL((token_combine_kernel<T, LANES>), grid, threads, 0, s, a);
  }
}

template <class T>
void launch(const CombineArgs& p, bool backward, hipStream_t s) {
  TokArgs a{p.yp, p.inv, p.w, p.base, p.y, p.dw, 0, p.T, p.rows, p.ldt, p.ldp, p.K, p.d, false};
  a.stream = (backward ? p.rows : p.T) * p.d * int64_t(sizeof(T)) >= kFarBytes;
  // a wave takes rows that its lanes hold in one chunk each: 4096 tokens of 8 places,
  // rows of 256 bf16 values 5.0 us and 10.3 backward (a block of 256 per token 6.1 and 19.1),
  // of 512 6.6 and 13.0 (7.5, 17.4), of 1024 13.9 and 24.4 (13.9, 24.9); 64 tokens of 1024
  // 4.7 and 8.0 (3.6, 5.6).
  // Longer rows that 1024 lanes hold, of no more tokens than CUs, take those: 64 tokens of
  // 4096 4.2 and 7.1 (256 lanes 4.9 and 8.7), of 7168 5.3 and 7.9 (7.3, 14.4), 256 of 7168
  // 6.2 and 12.1 (8.5, 18.5), 512 of 4096 6.8 and 17.0 (7.2, 15.8); 64 of 2048 3.7 and 6.8
  // (3.8, 5.7).
  if (p.d <= 512)
    launch_with<T, 64>(a, backward, s);
  else if (p.d > 2048 && p.d <= 8192 && p.T <= 256)
    launch_with<T, 1024>(a, backward, s);
  else
    launch_with<T, 256>(a, backward, s);
}

}  // namespace

hipError_t launch_token_combine(const CombineArgs& p, hipStream_t s) {
  p.bf16 ? launch<uint16_t>(p, false, s) : launch<float>(p, false, s);
  return hipGetLastError();
}

hipError_t launch_token_combine_backward(const CombineArgs& p, hipStream_t s) {
  p.bf16 ? launch<uint16_t>(p, true, s) : launch<float>(p, true, s);
  return hipGetLastError();
}

}  // namespace dsmoe
