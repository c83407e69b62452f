// Instantiation of the fused GEMV for one weight x activation format (mxfp4_bf16), one member
// per launch.
#include "w4_gemv_impl.h"

namespace w4 {
hipError_t launch_gemv_mxfp4_bf16(int b, const GemvArgs& a, int groups, const GemvPlan& p,
                                hipStream_t s) {
  return launch_fx<kMXFP4, kBF16, false>(b, a, groups, p, s);
}
}  // namespace w4
