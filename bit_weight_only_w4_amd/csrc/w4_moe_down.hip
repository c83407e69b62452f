// Instantiations of the expert products' down direction (h is bf16 planes for every format).
#include "w4_moe_impl.h"

namespace w4 {
hipError_t launch_moe_down(int weight, int kw, int tiles, const MoeArgs& a, hipStream_t s) {
  return tiles == 1 ? launch_moe_weight<kDown, kBF16, 1>(weight, kw, a, s)
                    : launch_moe_weight<kDown, kBF16, 3>(weight, kw, a, s);
}

namespace {
template <int FMT>
hipError_t token_kw(int kw, const MoeArgs& a, uint32_t tokens, hipStream_t s) {
  switch (kw) {
    case 1: return launch_moe_token_one<FMT, 1>(a, tokens, s);
    case 2: return launch_moe_token_one<FMT, 2>(a, tokens, s);
    case 4: return launch_moe_token_one<FMT, 4>(a, tokens, s);
    case 8: return launch_moe_token_one<FMT, 8>(a, tokens, s);
  }
  return hipErrorInvalidValue;
}
}  // namespace

hipError_t launch_moe_token(int weight, int kw, const MoeArgs& a, uint32_t tokens, hipStream_t s) {
  switch (weight) {
    case kNF4: return token_kw<kNF4>(kw, a, tokens, s);
    case kINT4: return token_kw<kINT4>(kw, a, tokens, s);
    case kFP4: return token_kw<kFP4>(kw, a, tokens, s);
    case kINT4A: return token_kw<kINT4A>(kw, a, tokens, s);
    case kMXFP4: return token_kw<kMXFP4>(kw, a, tokens, s);
  }
  return hipErrorInvalidValue;
}
}  // namespace w4
