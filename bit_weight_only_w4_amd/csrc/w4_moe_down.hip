// Instantiations of the expert products' down direction (h is bf16 planes for every format).
#include "w4_moe_impl.h"

namespace w4 {
hipError_t launch_moe_down(int weight, int kw, int tiles, const MoeArgs& a, uint32_t slots, hipStream_t s) {
  return tiles == 1 ? launch_moe_weight<kDown, kBF16, 1>(weight, kw, a, slots, s)
                    : launch_moe_weight<kDown, kBF16, 3>(weight, kw, a, slots, s);
}
}  // namespace w4
