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
// Measured (us, 256 / 128 / 64 / 32 rows):
//   x [16, 4096], 1 x 4096                    25 / 15 / 13 / 10
//   x [512, 2048], 8 x 1408                   17 / 12 / 10 / 8
//   x [1024, 7168], 1 x 4096                  47 / 30 / 26 / 48
//   x [2048, 4096], 1 x 4096                  35 / 26 / 31 / 58
//   x [1024, 4096], 16 x 4096                 34 / 39 / 36 / 42
//   x [2048, 2048], 64 x 2816                 59 / 41 / 37 / 41
//   x [4096, 7168], 32 x 4096                174 / 125 / 168 / 221
//   x [8192, 7168], 1 x 4096                 119 / 129 / 173 / 361
//   x [8192, 7168], 32 x 4096, Zipf loads    195 / 199 / 245 / 424
//   x [24576, 2048], 64 x 2816               119 / 122 / 158 / 271
//   x [128, 7168], 128 of 256 groups x 4096   32 rows: 276 (weights through the caches
//                                            325), 64: 328
// 32 x 32 against 32 x 128:
//   x [1, 7168], 1 x 4096, 128 tiles         11.8 / 13.4
//   x [16, 7168], 2 x 4096, 256 tiles        12.5 / 15.4
//   x [64, 2048], 32 x 256, 256 tiles         6.9 / 7.8
//   x [6, 2048], 6 x 1408, 264 tiles          7.5 / 7.8
//   x [128, 7168], 1 x 4096, 512 tiles       14.8 / 15.0
//   x [8, 2048], 8 x 2816, 704 tiles          9.5 / 8.8
// and where it is wrong, the tile it takes first:
//   x [2048, 7168], 32 x 4096                 128 rows: 124, 64: 109
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
