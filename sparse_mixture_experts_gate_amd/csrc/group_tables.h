// Tile tables of products grouped by expert, built on the device from the row
// offsets by every workgroup for itself. In an anonymous namespace, so each
// translation unit gets its own copy.
#pragma once

#include "tile_schedule.h"

namespace dsmoe {
namespace {

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

}  // namespace
}  // namespace dsmoe
