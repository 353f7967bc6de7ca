// The linear forward product's and the input gradient's kernels, whole and in slices of k (product.cuh).
#include "product.cuh"

namespace gift {
namespace product {
cudaError_t launch_linear(const Launch &L, bool bf16, bool vec, const Params &P, const CUtensorMap *maps, int pairs,
                          bool after) {
  return launch_typed<LINEAR>(L, bf16, vec, P, maps, pairs, after);
}
cudaError_t launch_slices(const Launch &L, const Params &P, const CUtensorMap *maps, int pairs, bool after) {
  return launch<SLICE, float, true>(L, P, maps, pairs, after);
}
}  // namespace product
}  // namespace gift
