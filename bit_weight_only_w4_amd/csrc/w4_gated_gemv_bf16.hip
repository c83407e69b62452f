// Gated launches of the fused GEMV (kernel in w4_gemv_impl.h): instantiations for bf16 tokens.
#include "w4_gemv_impl.h"
#include "w4_ffn.h"

namespace w4 {

hipError_t launch_gated_gemv_bf16(int weight, const GemvGatedArgs& a, const GemvPlan& p, hipStream_t s) {
  switch (weight) {
    case kNF4: return launch_gated_b<kNF4, kBF16, 1>(a, p, s);
    case kINT4: return launch_gated_b<kINT4, kBF16, 1>(a, p, s);
    case kFP4: return launch_gated_b<kFP4, kBF16, 1>(a, p, s);
    case kINT4A: return launch_gated_b<kINT4A, kBF16, 1>(a, p, s);
    default: return launch_gated_b<kMXFP4, kBF16, 1>(a, p, s);
  }
}

}  // namespace w4
