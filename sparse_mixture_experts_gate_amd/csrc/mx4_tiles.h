// Which tile a product on 4-bit operands takes: host arithmetic only, so that a test can
// ask it without a GPU.
#pragma once

#include <cmath>
#include <cstdint>

namespace dsmoe {
namespace {

// Time model of a tile (microseconds), fitted to measured products, per k-step: `one`
// and `many` with the GPU full of tiles of one group, or of more, whose weights come
// from memory; `idle` with it at most half full; `fixed` for a tile's first loads and
// its output.
struct TileCost {
  int bm, bn;
  double one, many, idle, fixed;
};
constexpr TileCost kCosts[] = {{256, 256, 1.76, 1.76, 1.22, 7.0},
                               {128, 256, 0.97, 1.15, 0.7, 3.5},
                               {64, 256, 0.7, 0.95, 0.36, 1.8},
                               {32, 128, 0.34, 0.38, 0.21, 1.1}};

// The rule: 32 x 32 tiles while they are no more than the CUs, else the tile with the
// least modelled time. Row counts per group live on the device, so the expected number
// of row tiles stands in for them: at least one per group with rows, else rows / BM and
// half a tile per group; with more than one group half a round more than the tiles fill.
// Measured (us, replayed graphs, 256 / 128 / 64 / 32 rows / 32 x 32; *: what the rule takes):
//   x [1, 7168], 1 x 4096                     41 / 24 / 20 / 14.6 / 13.2*
//   x [16, 4096], 1 x 4096                    27 / 17 / 14 / 11.4 / 10.3*
//   x [16, 7168], 2 x 4096                    42 / 24 / 21 / 15.4 / 14.2*
//   x [64, 2048], 32 x 256                    18 / 12 / 10.8 / 9.9 / 8.5*
//   x [128, 7168], 1 x 4096                   42 / 26 / 21 / 15.5* / 17.1
//   x [128, 7168], 256 x 4096                356 / 286 / 286 / 245* / 291
//   x [128, 7168], 128 of 256 groups x 4096  406 / 324 / 325 / 277* / 331 (32 rows, weights
//                                            through the caches: 325)
//   x [1024, 7168], 1 x 4096                  46 / 30 / 27* / 52 / 85
//   x [2048, 2048], 64 x 2816                 48 / 38 / 37* / 45 / 69
//   x [2048, 4096], 1 x 4096                  33 / 27* / 30 / 59 / 97
//   x [1024, 4096], 16 x 4096                 33 / 29* / 34 / 44 / 68
//   x [2048, 7168], 32 x 4096                118 / 99* / 111 / 154 / 243
//   x [4096, 7168], 32 x 4096                130 / 132* / 150 / 236 / 421
//   x [8192, 7168], 32 x 4096                195 / 180* / 242 / 430 / 818
//   x [8192, 7168], 32 x 4096, Zipf loads    191 / 182* / 242 / 432 / 811
//   x [8192, 7168], 1 x 4096                 129* / 130 / 167 / 375 / 720
//   x [24576, 2048], 64 x 2816               129* / 129 / 163 / 296 / 515
//   x [28240, 843], 5 x 1497                  57* / 61 / 71 / 154 / 246
// and where it is wrong:
//   x [6, 2048], 6 x 1408                     18 / 12 / 10.8 / 9.2* / 8.3
//   x [8, 2048], 8 x 2816                     18 / 12 / 10.9* / 9.8 / 10.5
//   x [8, 7168], 8 x 4096                     43 / 26 / 23* / 21 / 26
//   x [512, 2048], 8 x 1408                   18 / 13.5 / 11.9* / 10.1 / 12.9
//   x [800, 4096], 2 x 4096                   31 / 21* / 18 / 34 / 51
//   x [2048, 7168], 32 x 4096, Zipf loads    154 / 119* / 108 / 151 / 248
enum Mx4Tile { kTile256, kTile128, kTile64, kTile32, kTileThin };
constexpr int kThin = 32;  // rows and columns of kTileThin

inline Mx4Tile mx4_tile(int64_t rows, int groups, int n, int k) {
  const double touched = static_cast<double>(rows < groups ? rows : groups);
  auto row_tiles = [&](int bm) {
    const double mt = groups == 1 ? std::ceil(rows / static_cast<double>(bm))
                                  : rows / static_cast<double>(bm) + 0.5 * touched;
    return mt > touched ? mt : touched;
  };
  if ((n + kThin - 1) / kThin * row_tiles(kThin) <= 256) return kTileThin;
  const double nk = (k + 255) / 256;
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < 4; ++i) {
    const TileCost& t = kCosts[i];
    const double share = (n + t.bn - 1) / t.bn * row_tiles(t.bm) / 256;
    const double rounds = groups == 1 ? std::ceil(share) : share > 0.5 ? share + 0.5 : 1.0;
    const double step = share <= 0.5 ? t.idle : groups == 1 ? t.one : t.many;
    const double us = rounds * (nk * step + t.fixed);
    if (i == 0 || us < least) {
      least = us;
      best = i;
    }
  }
  return static_cast<Mx4Tile>(best);
}

}  // namespace
}  // namespace dsmoe
