// Dense products: the launch and its instantiations (kernel in w4_dense.h).
#include <algorithm>

#include "w4_dense.h"

namespace w4 {

// Tile and K splits by an estimate in microseconds: rounds of workgroups over the CUs, each operand's bytes at 5.5 TB/s
// where that takes longer, and for a split the second kernel and its sums' way through memory.  Against the best of
// 4 tiles and 1 to 20 splits it is within 7% on those shapes (64 x 128 tiles for 40 x 28672 x 8192 int8: 36 us, its
// weights at 6.5 TB/s; 128 x 256 for 1000 x 17920 x 1536 fp16: 78 us, 256 x 256 there 87; five splits of 256 x 256
// for 2048 x 1536 x 17920 fp16: 129 us, unsplit 128 x 256 tiles 262).  Where a last round of large tiles would leave
// most CUs idle, its tiles are covered by smaller ones in a second launch.
//
// Four bits: decoding makes a step of the largest tile take 1.1 (MXFP4), 1.19 (FP4, INT4) or 1.3 (NF4) times as long, of
// the others, whose rows of B meet fewer of A, 1.18 times that (160 and 256 tokens of 1536 -> 8960 to 8192 -> 28672).
// Decoding columns: 1.07 (FP4, INT4), 1.1 (MXFP4) or 1.25 (NF4), 1.12 times that for 128 x 256, 2.2 and 1.62 for 64 x 128
// (4096 x 2048 weights, 256 and 2048 tokens: a step of 64 x 128 tiles alone 0.71 to 1.07 us, of full CUs 1.14 to 1.5).
// Measured with weights of one term; of two, a step of second terms takes longer than one of first terms, which together
// makes NF4 of 256 x 256 tiles 1.02, columns of 128 x 256 1.35 (FP4) and 1.63 (NF4).
DensePlan plan_dense(bool gated, int64_t m, int64_t n, int64_t pitch, int packed, int terms) {
  const bool columns = packed >= 0 && !gated;
  const double slow = packed < 0         ? 1.0
                      : packed == kNF4   ? columns ? 1.25 : 1.3
                      : packed == kMXFP4 ? 1.1
                                         : columns ? 1.07 : 1.19;
  const int64_t cus = device_cu_count(), steps = (pitch + 127) / 128 * terms;
  const int64_t width = gated ? 2 * n : n;
  DensePlan best{0, 0, 1, (uint32_t)steps, 0, 0};
  double least = 0;
  for (int i = 0; i < (packed < 0 ? kTileCount : kTileCount - 1); ++i) {
    auto tile_of = [&](int j) {
      Tile t = kTiles[j];
      const double f = packed < 0 || j == 0 ? slow : columns ? 1.12 * slow : 1.18 * slow;
      t.alone *= columns && j == 2 ? 2.2 * slow : f;
      t.full *= columns && j == 2 ? 1.62 * slow : f;
      if (columns) t.ends += 3;  // the first steps are decoded before there is anything to multiply
      return t;
    };
    const Tile t = tile_of(i);
    const int64_t tiles = ((m + t.tm - 1) / t.tm) * ((width + t.tn - 1) / t.tn);
    for (int64_t s = 1; s <= 20 && s * 4 <= std::max<int64_t>(steps, 4); ++s) {
      const int64_t per = (steps / terms + s - 1) / s * terms;
      if ((s - 1) * per >= steps) continue;  // an empty split
      const int64_t rounds = (tiles * s + cus * t.fit - 1) / (cus * t.fit);
      const double work = rounds * (per * (tiles * s <= cus ? t.alone : t.full) + t.ends);
      const double bytes = ((double)m + (packed < 0 ? terms : 0.3125) * width) * pitch / 5.5e6;
      auto offer = [&](double w, int64_t rest) {
        double us = std::max(w, bytes) + 0.1 * std::min(w, bytes);
        if (s > 1) us += 3 + (double)s * m * width * 8 / 5e6;
        if (least == 0 || us < least) {
          least = us;
          best = DensePlan{us, i, (uint32_t)s, (uint32_t)per, (uint32_t)tiles, (uint32_t)rest};
        }
      };
      offer(work, 0);
      const int64_t rest = tiles % cus;
      if (t.fit == 1 && s == 1 && tiles > cus && rest) {
        const Tile r = tile_of(kRestTile);
        const int64_t small = rest * (t.tm / r.tm) * (t.tn / r.tn);
        offer(tiles / cus * (per * t.alone + t.ends) + 2 + (small + cus * r.fit - 1) / (cus * r.fit) *
                  (per * (small <= cus ? r.alone : r.full) + r.ends),
              rest);
      }
    }
  }
  return best;
}

bool dense_prepare(const DensePlan& p, DenseArgs* a) {
  if ((uint64_t)p.tiles * 8 >= ((uint64_t)1 << 31)) return false;
  a->splits = p.splits;
  a->per = p.per;
  if (p.splits == 1) a->partial = nullptr;
  a->wide = a->n % 8 == 0 && ((uintptr_t)a->out | (uintptr_t)a->products) % 16 == 0;
  return true;
}

double dense_us(bool gated, int64_t m, int64_t n, int64_t pitch, int packed, int terms) {
  return plan_dense(gated, m, n, pitch, packed, terms).us;
}

size_t dense_bytes(bool gated, int64_t m, int64_t n, int64_t pitch, int packed, int terms) {
  const DensePlan p = plan_dense(gated, m, n, pitch, packed, terms);
  return p.splits > 1 ? (size_t)p.splits * (size_t)m * (size_t)(gated ? 2 * n : n) * 4 : 0;
}

hipError_t launch_dense(int type, bool gated, const DenseArgs& args, hipStream_t s) {
  DenseArgs a = args;
  const DensePlan p = plan_dense(gated, a.m, a.n, a.pitch, -1, (int)a.terms);
  if (!dense_prepare(p, &a)) return hipErrorInvalidValue;
  if (type == kDenseF16)
    return gated ? dense_run<kDenseF16, true, -1>(p, a, s) : dense_run<kDenseF16, false, -1>(p, a, s);
  if (type == kDenseBF16) return gated ? hipErrorInvalidValue : dense_run<kDenseBF16, false, -1>(p, a, s);
  return gated ? dense_run<kDenseI8, true, -1>(p, a, s) : dense_run<kDenseI8, false, -1>(p, a, s);
}

}  // namespace w4
