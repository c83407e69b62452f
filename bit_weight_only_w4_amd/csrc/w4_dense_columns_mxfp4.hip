// The dense product with columns of MXFP4 weights decoded on chip (w4_dense.h).
#include "w4_dense.h"

namespace w4 {

hipError_t launch_dense_columns_mxfp4(int type, const DenseArgs& args, hipStream_t s) {
  DenseArgs a = args;
  const DensePlan p = plan_dense(false, a.m, a.n, a.pitch, kMXFP4, 1);
  if (!dense_prepare(p, &a)) return hipErrorInvalidValue;
  return type == kDenseF16 ? dense_run<kDenseF16, false, kMXFP4>(p, a, s) : dense_run<kDenseBF16, false, kMXFP4>(p, a, s);
}

}  // namespace w4
