// The dense product with columns of FP4 weights decoded on chip (w4_dense.h).
#include "w4_dense.h"

namespace w4 {

hipError_t launch_dense_columns_fp4(const DenseArgs& args, hipStream_t s) {
  DenseArgs a = args;
  const DensePlan p = plan_dense(false, a.m, a.n, a.pitch, kFP4, dense_terms(kFP4));
  return dense_prepare(p, &a) ? dense_run<kDenseF16, false, kFP4>(p, a, s) : hipErrorInvalidValue;
}

}  // namespace w4
