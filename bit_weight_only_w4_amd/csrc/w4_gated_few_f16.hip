// Gated block for a few tokens (kernel in w4_gated_few.h): instantiations for f16 tokens.
#include "w4_gated_few.h"

namespace w4 {

hipError_t launch_gated_few_f16(int weight, const GatedFewArgs& a, hipStream_t s) { return few_dispatch<kF16>(weight, a, s); }

}  // namespace w4
