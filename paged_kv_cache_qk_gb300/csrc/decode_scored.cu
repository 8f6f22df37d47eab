// Launch of the decode kernel (decode_kernel.cuh) whose scores follow rules.
#include "decode_kernel.cuh"

namespace pkvqk {

cudaError_t launch_paged_decode_scored(const DecodePlan& p, const CUtensorMap& kmap,
                                       const CUtensorMap& vmap, const DecodeArgs& a,
                                       int grid_ctas, cudaStream_t stream) {
  return launch_decode<true>(p, kmap, vmap, a, grid_ctas, stream);
}

}  // namespace pkvqk
