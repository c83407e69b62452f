// The dense gated product over NF4 weights decoded on chip (w4_dense.h).
#include "w4_dense.h"

namespace w4 {

hipError_t launch_dense_nf4(const DenseArgs& args, hipStream_t s) {
  DenseArgs a = args;
  const DensePlan p = plan_dense(true, a.m, a.n, a.pitch, kNF4, dense_terms(kNF4));
  return dense_prepare(p, &a) ? dense_run<kDenseF16, true, kNF4>(p, a, s) : hipErrorInvalidValue;
}

}  // namespace w4
