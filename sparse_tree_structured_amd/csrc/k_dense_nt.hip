// Products da . W^T: the gradient of x, of one weight or of the gated pair's two.
#include "product.hpp"

namespace fff {

template <ProductPair PAIR>
static hipError_t run(const Product& p, void* workspace, hipStream_t st) {
  if (p.bf16)  // dx is of the layer's type
    return run_with<uint16_t, kProductNT, PAIR>(p, LinearEpilogue<uint16_t, uint16_t>{p.e}, workspace, st);
  return run_with<float, kProductNT, PAIR>(p, LinearEpilogue<float, float>{p.e}, workspace, st);
}

hipError_t run_nt(const Product& p, void* workspace, hipStream_t st) {
  return p.pair == kPairSum ? run<kPairSum>(p, workspace, st) : run<kSingle>(p, workspace, st);
}

}  // namespace fff
