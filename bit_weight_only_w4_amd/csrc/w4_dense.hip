// Dense products: the launch and its instantiations (kernel in w4_dense.h).
#include <algorithm>

#include "w4_dense.h"

namespace w4 {

namespace {

// The tiles, largest first: waves along M and N, 32-row tiles of a wave along M and N, and how many workgroups a CU
// holds (LDS: four stages).
struct Tile {
  int wm, wn, mt, nt, fit;
};
constexpr Tile kTiles[] = {{2, 4, 4, 2, 1}, {2, 2, 2, 2, 2}, {2, 2, 1, 2, 3}, {1, 2, 1, 2, 4}};
constexpr int kTileCount = 4;

struct DensePlan {
  int tile;
  uint32_t splits, per;
};

// Tile and splits by an estimate in clocks.  A step of a tile takes the matrix cores TM TN / 64 clocks and (TM + TN) 64
// bytes through the caches, at about 48 bytes a clock and CU (what three stages in flight carry over the memory's
// latency); a CU's workgroups share both.  Each round of workgroups pays its start and end; a split K
// pays for writing and reading its sums.
DensePlan plan_dense(bool gated, int64_t m, int64_t n, int64_t pitch) {
  const int64_t cus = device_cu_count(), steps = (pitch + 127) / 128;
  const int64_t width = gated ? 2 * n : n;
  DensePlan best{0, 1, (uint32_t)steps};
  double least = 0;
  for (int i = 0; i < kTileCount; ++i) {
    const Tile& t = kTiles[i];
    const int64_t tm = 32 * t.mt * t.wm, tn = 32 * t.nt * t.wn;
    const int64_t tiles = ((m + tm - 1) / tm) * ((width + tn - 1) / tn);
    const double step = std::max(tm * tn / 32.0, (tm + tn) * 128 / 48.0);
    for (int64_t s = 1; s <= 32 && s * 4 <= std::max<int64_t>(steps, 4); ++s) {
      const int64_t per = (steps + s - 1) / s;
      if ((s - 1) * per >= steps) continue;  // an empty split
      const int64_t on_cu = (tiles * s + cus - 1) / cus;  // workgroups of the busiest CU
      const double lonely = std::max(step, 1300.0 / std::min<int64_t>(on_cu, t.fit));  // the copies' latency over three steps
      double clocks = on_cu * per * lonely + (double)((on_cu + t.fit - 1) / t.fit) * 4000 + on_cu * tm * tn / 24.0;
      if (s > 1) clocks += 7000 + (double)s * m * width * 8 / 1600;
      if (least == 0 || clocks < least) {
        least = clocks;
        best = DensePlan{i, (uint32_t)s, (uint32_t)per};
      }
    }
  }
  return best;
}

template <int TYPE, bool GATED>
hipError_t dense_pick(int tile, const DenseArgs& a, hipStream_t s) {
  switch (tile) {
    case 0: return dense_launch<TYPE, GATED, 2, 4, 4, 2, 2>(a, s);
    case 1: return dense_launch<TYPE, GATED, 2, 2, 2, 2, 2>(a, s);
    case 2: return dense_launch<TYPE, GATED, 2, 2, 1, 2, 2>(a, s);
    default: return dense_launch<TYPE, GATED, 1, 2, 1, 2, 2>(a, s);
  }
}

}  // namespace

size_t dense_bytes(bool gated, int64_t m, int64_t n, int64_t pitch) {
  const DensePlan p = plan_dense(gated, m, n, pitch);
  return p.splits > 1 ? (size_t)p.splits * (size_t)m * (size_t)(gated ? 2 * n : n) * 4 : 0;
}

hipError_t launch_dense(int type, bool gated, const DenseArgs& args, hipStream_t s) {
  DenseArgs a = args;
  const DensePlan p = plan_dense(gated, a.m, a.n, a.pitch);
  a.splits = p.splits;
  a.per = p.per;
  if (p.splits == 1) a.partial = nullptr;
  a.wide = a.n % 8 == 0 && ((uintptr_t)a.out | (uintptr_t)a.products) % 16 == 0;
  if (type == kDenseF16)
    return gated ? dense_pick<kDenseF16, true>(p.tile, a, s) : dense_pick<kDenseF16, false>(p.tile, a, s);
  if (type == kDenseBF16) return gated ? hipErrorInvalidValue : dense_pick<kDenseBF16, false>(p.tile, a, s);
  return gated ? dense_pick<kDenseI8, true>(p.tile, a, s) : dense_pick<kDenseI8, false>(p.tile, a, s);
}

}  // namespace w4
