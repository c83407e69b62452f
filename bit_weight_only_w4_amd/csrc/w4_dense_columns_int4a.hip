// The dense product with columns of asymmetric INT4 weights decoded on chip (w4_dense.h).
#include "w4_dense.h"

namespace w4 {

hipError_t launch_dense_columns_int4a(const DenseArgs& args, hipStream_t s) {
  DenseArgs a = args;
  const DensePlan p = plan_dense(false, a.m, a.n, a.pitch, kINT4A, dense_terms(kINT4A));
  return dense_prepare(p, &a) ? dense_run<kDenseF16, false, kINT4A>(p, a, s) : hipErrorInvalidValue;
}

}  // namespace w4
