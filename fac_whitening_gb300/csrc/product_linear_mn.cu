// The linear product's kernels (product.cuh): the input gradient's.
#include "product.cuh"

namespace gift {
namespace product {
cudaError_t launch_linear_mn(const Launch &L, bool bf16, bool vec, const Params &P, const CUtensorMap *maps, const IoMaps &io, int pairs,
                             bool after) {
  return launch_typed<LINEAR, true>(L, bf16, vec, P, maps, io, pairs, after);
}
}  // namespace product
}  // namespace gift
