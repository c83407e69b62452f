// Dense products: the launch and its instantiations (kernel in w4_dense.h).
#include <algorithm>

#include "w4_dense.h"

namespace w4 {

namespace {

// The tiles, largest first: waves along M and N, 32-row tiles of a wave along M and N, stages; how many workgroups of it
// a CU holds (LDS), and what was measured (MI355X, over twelve shapes of 1 to 4096 rows, fp16 and int8): microseconds
// a step of 128 bytes when alone on a CU and when the CU is full, and a round's start and end.
struct Tile {
  int tm, tn, fit;
  double alone, full, ends;
};
constexpr Tile kTiles[] = {{256, 256, 1, 1.85, 1.85, 5}, {128, 256, 1, 0.95, 0.95, 4.5}, {64, 128, 2, 0.34, 0.72, 3},
                           {32, 128, 2, 0.33, 0.60, 3}};
constexpr int kTileCount = 4;

struct DensePlan {
  int tile;
  uint32_t splits, per;
  uint32_t tiles, rest;  // tiles in all, and how many of the last are covered with 64 x 128 tiles by a second launch
};
constexpr int kRestTile = 2;

// Tile and K splits by an estimate in microseconds: rounds of workgroups over the CUs, each operand's bytes at 5.5 TB/s
// where that takes longer, and for a split the second kernel and its sums' way through memory.  Against the best of
// 4 tiles and 1 to 20 splits it is within 7% on those shapes (64 x 128 tiles for 40 x 28672 x 8192 int8: 36 us, its
// weights at 6.5 TB/s; 128 x 256 for 1000 x 17920 x 1536 fp16: 78 us, 256 x 256 there 87; five splits of 256 x 256
// for 2048 x 1536 x 17920 fp16: 129 us, unsplit 128 x 256 tiles 262).  Where a last round of large tiles would leave
// most CUs idle, its tiles are covered by smaller ones in a second launch.
DensePlan plan_dense(bool gated, int64_t m, int64_t n, int64_t pitch) {
  const int64_t cus = device_cu_count(), steps = (pitch + 127) / 128;
  const int64_t width = gated ? 2 * n : n;
  DensePlan best{0, 1, (uint32_t)steps, 0, 0};
  double least = 0;
  for (int i = 0; i < kTileCount; ++i) {
    const Tile& t = kTiles[i];
    const int64_t tiles = ((m + t.tm - 1) / t.tm) * ((width + t.tn - 1) / t.tn);
    for (int64_t s = 1; s <= 20 && s * 4 <= std::max<int64_t>(steps, 4); ++s) {
      const int64_t per = (steps + s - 1) / s;
      if ((s - 1) * per >= steps) continue;  // an empty split
      const int64_t rounds = (tiles * s + cus * t.fit - 1) / (cus * t.fit);
      const double work = rounds * (per * (tiles * s <= cus ? t.alone : t.full) + t.ends);
      const double bytes = (double)(m + width) * pitch / 5.5e6;
      auto offer = [&](double w, int64_t rest) {
        double us = std::max(w, bytes) + 0.1 * std::min(w, bytes);
        if (s > 1) us += 3 + (double)s * m * width * 8 / 5e6;
        if (least == 0 || us < least) {
          least = us;
          best = DensePlan{i, (uint32_t)s, (uint32_t)per, (uint32_t)tiles, (uint32_t)rest};
        }
      };
      offer(work, 0);
      const int64_t rest = tiles % cus;
      if (t.fit == 1 && s == 1 && tiles > cus && rest) {
        const Tile& r = kTiles[kRestTile];
        const int64_t small = rest * (t.tm / r.tm) * (t.tn / r.tn);
        offer(tiles / cus * (per * t.alone + t.ends) + 2 + (small + cus * r.fit - 1) / (cus * r.fit) *
                  (per * (small <= cus ? r.alone : r.full) + r.ends),
              rest);
      }
    }
  }
  return best;
}

template <int TYPE, bool GATED>
hipError_t dense_tiles(int tile, const DenseArgs& a, uint32_t tile0, uint32_t count, int of, hipStream_t s) {
  const uint32_t bm = kTiles[of].tm, bn = kTiles[of].tn / (GATED ? 2 : 1);
  switch (tile) {
    case 0: return dense_launch<TYPE, GATED, 2, 4, 4, 2, 2>(a, tile0, count, bm, bn, s);
    case 1: return dense_launch<TYPE, GATED, 2, 4, 2, 2, 3>(a, tile0, count, bm, bn, s);
    case 2: return dense_launch<TYPE, GATED, 2, 2, 1, 2, 3>(a, tile0, count, bm, bn, s);
    default: return dense_launch<TYPE, GATED, 1, 2, 1, 2, 4>(a, tile0, count, bm, bn, s);
  }
}

template <int TYPE, bool GATED>
hipError_t dense_run(const DensePlan& p, const DenseArgs& a, hipStream_t s) {
  hipError_t e = dense_tiles<TYPE, GATED>(p.tile, a, 0, p.tiles - p.rest, p.tile, s);
  if (e == hipSuccess && p.rest) e = dense_tiles<TYPE, GATED>(kRestTile, a, p.tiles - p.rest, p.rest, p.tile, s);
  if (e == hipSuccess && p.splits > 1) e = dense_sum<TYPE, GATED>(a, s);
  return e;
}

}  // namespace

size_t dense_bytes(bool gated, int64_t m, int64_t n, int64_t pitch) {
  const DensePlan p = plan_dense(gated, m, n, pitch);
  return p.splits > 1 ? (size_t)p.splits * (size_t)m * (size_t)(gated ? 2 * n : n) * 4 : 0;
}

hipError_t launch_dense(int type, bool gated, const DenseArgs& args, hipStream_t s) {
  DenseArgs a = args;
  const DensePlan p = plan_dense(gated, a.m, a.n, a.pitch);
  if ((uint64_t)p.tiles * 8 >= ((uint64_t)1 << 31)) return hipErrorInvalidValue;
  a.splits = p.splits;
  a.per = p.per;
  if (p.splits == 1) a.partial = nullptr;
  a.wide = a.n % 8 == 0 && ((uintptr_t)a.out | (uintptr_t)a.products) % 16 == 0;
  if (type == kDenseF16)
    return gated ? dense_run<kDenseF16, true>(p, a, s) : dense_run<kDenseF16, false>(p, a, s);
  if (type == kDenseBF16) return gated ? hipErrorInvalidValue : dense_run<kDenseBF16, false>(p, a, s);
  return gated ? dense_run<kDenseI8, true>(p, a, s) : dense_run<kDenseI8, false>(p, a, s);
}

}  // namespace w4
