// Launches of the multi-query attention kernel (prefill_kernel.cuh) whose scores follow rules.
#include "prefill_launch.cuh"

namespace pkvqk {

cudaError_t launch_paged_prefill_scored(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                        const PrefillArgs& a, cudaStream_t stream) {
  // a cap too wide for one reference takes the kernel that also adds a bias, of 0
  const bool cap = a.rules.cap > 0.f, bias = a.rules.slopes != nullptr;
  if (cap && !bias && a.rules.cap <= kBoundedCap)
    return launch_format<0, kRuleIntervals | kRuleCap | kRuleBounded>(kmap, vmap, a, stream);
  if (cap) return launch_format<0, kRuleIntervals | kRuleCap | kRuleBias>(kmap, vmap, a, stream);
  if (bias) return launch_format<0, kRuleIntervals | kRuleBias>(kmap, vmap, a, stream);
  return launch_format<0, kRuleIntervals>(kmap, vmap, a, stream);
}

}  // namespace pkvqk
