// The dense gated product over MXFP4 weights decoded on chip (w4_dense.h).
#include "w4_dense.h"

namespace w4 {

hipError_t launch_dense_mxfp4(const DenseArgs& args, hipStream_t s) {
  DenseArgs a = args;
  const DensePlan p = plan_dense(true, a.m, a.n, a.pitch, kMXFP4, dense_terms(kMXFP4));
  return dense_prepare(p, &a) ? dense_run<kDenseF16, true, kMXFP4>(p, a, s) : hipErrorInvalidValue;
}

}  // namespace w4
