// The linear products' kernels in slices of k (product.cuh).
#include "product.cuh"

namespace gift {
namespace product {
cudaError_t launch_slices(const Launch &L, bool bf16, bool mn, const Params &P, const CUtensorMap *maps, const IoMaps &io, int pairs,
                          bool after) {
  if (bf16)
    return mn ? launch<SLICE, __nv_bfloat16, true, true>(L, P, maps, io, pairs, after)
              : launch<SLICE, __nv_bfloat16, true, false>(L, P, maps, io, pairs, after);
  return mn ? launch<SLICE, float, true, true>(L, P, maps, io, pairs, after)
            : launch<SLICE, float, true, false>(L, P, maps, io, pairs, after);
}
}  // namespace product
}  // namespace gift
