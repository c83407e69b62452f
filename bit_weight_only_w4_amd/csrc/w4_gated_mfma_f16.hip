// Gated launches of the MFMA kernel (w4_mfma_impl.h): instantiations for fp16 tokens.
#include "w4_mfma_impl.h"

namespace w4 {

hipError_t mfma_dispatch_gated_f16(int op, int weight, const MfmaGatedArgs& a, int tiles, int kw, int lds, int grid,
                                   int slices, int* out, hipStream_t s) {
  return gated_dispatch<kF16>(op, weight, a, tiles, kw, lds, grid, slices, out, s);
}

}  // namespace w4
