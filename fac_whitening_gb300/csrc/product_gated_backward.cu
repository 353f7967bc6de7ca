// The gated backward product's kernels (product.cuh).
#include "product.cuh"

namespace gift {
namespace product {
cudaError_t launch_gated_backward(const Launch &L, bool bf16, bool vec, const Params &P, const CUtensorMap *maps,
                                  const IoMaps &io, int pairs, bool after) {
  return launch_typed<GATED_BACKWARD, true>(L, bf16, vec, P, maps, io, pairs, after);
}
}  // namespace product
}  // namespace gift
