// Input gradient for a few tokens (kernel in w4_grad_few.h): instantiations for bf16 gradients.
#include "w4_grad_few.h"

namespace w4 {

hipError_t launch_grad_few_bf16(int weight, const GradFewArgs& a, uint32_t splits, hipStream_t s) {
  return grad_few_dispatch<kBF16>(weight, a, splits, s);
}

}  // namespace w4
