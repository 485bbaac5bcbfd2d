// Products x . W: the linear layer and the gated pair.
#include "product.hpp"

namespace fff {

template <typename E>
static hipError_t run(const Product& p, void* workspace, hipStream_t st) {
  if (p.pair == kPairColumns)
    return run_with<E, kProductNN, kPairColumns>(p, GatedEpilogue<E>{p.e}, workspace, st);
  return run_linear<E, kProductNN, kSingle>(p, workspace, st);
}

hipError_t run_nn(const Product& p, void* workspace, hipStream_t st) {
  return p.bf16 ? run<uint16_t>(p, workspace, st) : run<float>(p, workspace, st);
}

}  // namespace fff
