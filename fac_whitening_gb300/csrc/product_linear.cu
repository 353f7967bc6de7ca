// The linear product's kernels (product.cuh): the forward product, and the choice of B's layout.
#include "product.cuh"

namespace gift {
namespace product {
cudaError_t launch_linear(const Launch &L, bool bf16, bool vec, bool mn, const Params &P, const CUtensorMap *maps,
                          const IoMaps &io, int pairs, bool after) {
  return mn ? launch_linear_mn(L, bf16, vec, P, maps, io, pairs, after)
            : launch_typed<LINEAR, false>(L, bf16, vec, P, maps, io, pairs, after);
}
}  // namespace product
}  // namespace gift
