// Grid of a persistent launch.
#pragma once

#include "internal.h"
#include "per_device.h"

namespace dsmoe {
namespace {

// Workgroups of a persistent launch of kernel K: the resident ones of the
// current device, or no more than the tiles there can be (whole XCD rounds).
template <auto K>
unsigned grid_of(int threads, int64_t tiles) {
  static PerDevice resident;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) dev = -1;
  const int res = resident.get(dev, [&] {
    int nb = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&nb, K, threads, 0) != hipSuccess || nb < 1)
      nb = 1;
    return (device_cu_count() * nb + 7) / 8 * 8;
  });
  const int64_t t = tiles < 1 ? 8 : (tiles + 7) / 8 * 8;
  return static_cast<unsigned>(t < res ? t : res);
}

}  // namespace
}  // namespace dsmoe
