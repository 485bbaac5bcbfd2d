// Products x^T . da: the gradient of one weight, or of the gated pair's two.
#include "product.hpp"

namespace fff {

template <typename E>
static hipError_t run(const Product& p, void* workspace, hipStream_t st) {
  if (p.pair == kPairTwo) return run_linear<E, kProductTN, kPairTwo>(p, workspace, st);
  return run_linear<E, kProductTN, kSingle>(p, workspace, st);
}

hipError_t run_tn(const Product& p, void* workspace, hipStream_t st) {
  return p.bf16 ? run<uint16_t>(p, workspace, st) : run<float>(p, workspace, st);
}

}  // namespace fff
