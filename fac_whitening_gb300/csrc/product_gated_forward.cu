// The gated forward product's kernels (product.cuh).
#include "product.cuh"

namespace gift {
namespace product {
cudaError_t launch_gated_forward(const Launch &L, bool bf16, bool vec, const Params &P, const CUtensorMap *maps,
                                 const IoMaps &io, int pairs, bool after) {
  return launch_typed<GATED_FORWARD, false>(L, bf16, vec, P, maps, io, pairs, after);
}
}  // namespace product
}  // namespace gift
