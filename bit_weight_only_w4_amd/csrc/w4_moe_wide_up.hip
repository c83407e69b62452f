// Instantiations of the expert products of many tokens, up direction.
#include "w4_moe_wide_impl.h"

namespace w4 {
hipError_t launch_moe_wide_up(int weight, int xtype, const MoeArgs& a, hipStream_t s) {
  return xtype == kF16 ? launch_moe_wide_weight<kUp, kF16>(weight, a, s)
                       : launch_moe_wide_weight<kUp, kBF16>(weight, a, s);
}
}  // namespace w4
