// Dense products: the launch and its instantiations (kernel in w4_dense.h).
#include "w4_dense.h"

namespace w4 {

namespace {

template <int TYPE, bool GATED>
hipError_t dense_pick(const DenseArgs& a, hipStream_t s) {
  const auto tiles = [&](uint32_t tm, uint32_t tn) {
    const uint32_t cn = GATED ? tn / 2 : tn;
    return (int64_t)((a.m + tm - 1) / tm) * ((a.n + cn - 1) / cn);
  };
  const int64_t cus = device_cu_count();
  if (a.m > 32 && tiles(256, 256) >= cus) return dense_launch<TYPE, GATED, 2, 4, 4, 2>(a, s);
  if (a.m > 32) return dense_launch<TYPE, GATED, 2, 2, 2, 2>(a, s);
  return dense_launch<TYPE, GATED, 1, 2, 1, 2>(a, s);
}

}  // namespace

hipError_t launch_dense(int type, bool gated, const DenseArgs& args, hipStream_t s) {
  DenseArgs a = args;
  a.wide = a.n % 8 == 0 && ((uintptr_t)a.out | (uintptr_t)a.products) % 16 == 0;
  if (type == kDenseF16) return gated ? dense_pick<kDenseF16, true>(a, s) : dense_pick<kDenseF16, false>(a, s);
  if (type == kDenseBF16) return gated ? hipErrorInvalidValue : dense_pick<kDenseBF16, false>(a, s);
  return gated ? dense_pick<kDenseI8, true>(a, s) : dense_pick<kDenseI8, false>(a, s);
}

}  // namespace w4
