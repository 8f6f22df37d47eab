// Launch of the multi-query attention kernel (prefill_kernel.cuh), for a cache format and
// the score rules it is built for.
#pragma once

#include "prefill_kernel.cuh"
#include "prefill_order.h"

#include <cstring>

namespace pkvqk {

namespace {

template <int kFormat, int kRules = 0>
cudaError_t launch_format(const CUtensorMap& kmap, const CUtensorMap& vmap,
                          const PrefillArgs& args, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_set{0};
  const auto kern = paged_prefill_kernel<kFormat, kRules>;
  const cudaError_t e = set_smem_limit_once(kern, kSmemBytes<kFormat>, smem_set);
  if (e != cudaSuccess) return e;
  PrefillArgs a = args;
  CUtensorMap qmap, omap;
  std::memset(&qmap, 0, sizeof(qmap));
  std::memset(&omap, 0, sizeof(omap));
  // Every sequence's last row tiles first, where row tiles differ in their keys: fresh
  // varlen prompts, and over an 8-bit cache chunks of at least half the longest
  // sequence (fresh 4 x 2048 tokens 106 -> 90 us, 1 x 4096 103 -> 69, 3 x 1500 after 700
  // 86 -> 70, 8 x 1024 after 1024 238 -> 228).  Else the row tiles of a sequence
  // together: 8 x 512 after 0 to 6144, 4 kv heads, 215 us against 238.
  const long long gx = static_cast<long long>(a.m_tiles) * a.num_kv_heads * a.num_splits;
  // Under score rules as over an 8-bit cache.
  const bool mostly_new = (kFormat != 0 || kRules != 0) && 2ll * a.q_len >= a.longest;
  a.mt_major = row_tile_major(a.cu_seqlens_q != nullptr || mostly_new, gx, a.batch) ? 1 : 0;
  a.group_shift = -1;
  if (a.group > 0 && (a.group & (a.group - 1)) == 0)
    for (int s = 0; s < 31; ++s)
      if ((1 << s) == a.group) a.group_shift = s;
  a.q_tma = 0;                                 // 8-bit: Q is loaded and turned into f16
  if constexpr (kFormat == 0)
    a.q_tma = encode_rows_map(&qmap, a.q, a.total_q, a.num_q_heads, a.q_stride_h * 2,
                              a.q_stride_t * 2, a.group) ? 1 : 0;
  a.o_tma = (a.num_splits == 1 &&
             encode_rows_map(&omap, a.out, a.total_q, a.num_q_heads, kHeadDim * 2,
                             static_cast<long long>(a.num_q_heads) * kHeadDim * 2, a.group))
                ? 1 : 0;
  return launch_pdl(kern, dim3(static_cast<unsigned>(gx), a.batch),
                    dim3(kThreads), kSmemBytes<kFormat>, stream, kmap, vmap, qmap, omap, a);
}

}  // namespace

}  // namespace pkvqk
