// Launches of the multi-query attention kernel whose scores follow rules
// (prefill_scored_kernel.cuh).
#include "prefill_order.h"
#include "prefill_scored_kernel.cuh"

#include <algorithm>
#include <cstring>

namespace pkvqk {

namespace {

template <int kRules>
cudaError_t launch_rules(const CUtensorMap& kmap, const CUtensorMap& vmap,
                         const PrefillArgs& args, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_set{0};
  const auto kern = scored_prefill_kernel<kRules>;
  const cudaError_t e = set_smem_limit_once(kern, kScoredSmemBytes, smem_set);
  if (e != cudaSuccess) return e;
  PrefillArgs a = args;
  CUtensorMap qmap;
  std::memset(&qmap, 0, sizeof(qmap));
  // Every sequence's last row tiles first, where row tiles differ in their keys: packed
  // prompts, and chunks of at least half the longest span (fresh 4 x 2048 tokens 107 -> 86
  // us).  Else the row tiles of a sequence together, which share its keys.
  const long long gx = static_cast<long long>(a.m_tiles) * a.num_kv_heads * a.num_splits;
  a.mt_major = row_tile_major(a.cu_seqlens_q != nullptr || 2ll * a.q_len >= a.longest, gx,
                              a.batch) ? 1 : 0;
  dim3 grid(static_cast<unsigned>(gx), a.batch);
  if (a.mt_major && a.cu_seqlens_q != nullptr && a.batch <= kPackedBatch) {
    // at most this many row tiles of all sequences hold rows
    const long long tiles = (a.total_q * a.group + (2ll * kM - 1) * a.batch) / (2 * kM);
    a.mt_major = kPackedMajor;
    grid = dim3(static_cast<unsigned>(std::min<long long>(
        tiles * a.num_kv_heads * a.num_splits, gx * a.batch)));
  }
  a.group_shift = -1;
  if (a.group > 0 && (a.group & (a.group - 1)) == 0)
    for (int s = 0; s < 31; ++s)
      if ((1 << s) == a.group) a.group_shift = s;
  a.q_tma = encode_rows_map(&qmap, a.q, a.total_q, a.num_q_heads, a.q_stride_h * 2,
                            a.q_stride_t * 2, a.group) ? 1 : 0;
  return launch_pdl(kern, grid, dim3(kThreads), kScoredSmemBytes, stream, kmap, vmap, qmap, a);
}

}  // namespace

cudaError_t launch_paged_prefill_scored(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                        const PrefillArgs& a, cudaStream_t stream) {
  // a cap too wide for one reference takes the kernel that also adds a bias, of 0
  const bool cap = a.rules.cap > 0.f, bias = a.rules.slopes != nullptr;
  if (cap && !bias && a.rules.cap <= kBoundedCap)
    return launch_rules<kRuleIntervals | kRuleCap | kRuleBounded>(kmap, vmap, a, stream);
  if (cap) return launch_rules<kRuleIntervals | kRuleCap | kRuleBias>(kmap, vmap, a, stream);
  if (bias) return launch_rules<kRuleIntervals | kRuleBias>(kmap, vmap, a, stream);
  return launch_rules<kRuleIntervals>(kmap, vmap, a, stream);
}

}  // namespace pkvqk
