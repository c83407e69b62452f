// Instantiations of the expert products of many tokens, down direction (h is bf16 planes for every format).
#include "w4_moe_wide_impl.h"

namespace w4 {
hipError_t launch_moe_wide_down(int weight, const MoeArgs& a, hipStream_t s) {
  return launch_moe_wide_weight<kDown, kBF16>(weight, a, s);
}
}  // namespace w4
