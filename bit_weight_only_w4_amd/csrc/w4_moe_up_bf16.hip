// Instantiations of the expert products' up direction for bf16 activations.
#include "w4_moe_impl.h"

namespace w4 {
hipError_t launch_moe_up_bf16(int weight, int kw, const MoeArgs& a, hipStream_t s) {
  return launch_moe_weight<kUp, kBF16, 1>(weight, kw, a, s);
}
hipError_t launch_moe_pair_bf16(int weight, int kw, const MoeArgs& a, uint32_t tokens, hipStream_t s) {
  return launch_moe_pair_weight<kBF16>(weight, kw, a, tokens, s);
}
}  // namespace w4
