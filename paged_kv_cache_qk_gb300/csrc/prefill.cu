// Host side of the multi-query attention kernel (prefill_kernel.cuh): row-tile
// tensor maps of q and out, and the launches, for bf16 and 8-bit caches.
#include "prefill_kernel.cuh"
#include "prefill_order.h"

#include <cudaTypedefs.h>

#include <cstring>
#include <mutex>

namespace pkvqk {

namespace {

// cuTensorMapEncodeTiled through the runtime's driver entry point, looked up
// once; nullptr if the driver does not provide it.
PFN_cuTensorMapEncodeTiled_v12000 row_map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 3-D view (128 dims, heads, tokens) of q or out, strides in bytes, with a box
// of (64 dims, group heads, 128 / group tokens) and 128-byte swizzle: one box
// is one 64-dim half of a 128-row tile in the packed row order
// r = t * group + h % group, laid out as the MMA operand (and the output
// staging) expects.  False where the layout does not allow such a box (group
// not a power of two up to 128, base or strides not multiples of 16 bytes).
bool encode_rows_map(CUtensorMap* map, const void* base, long long tokens, int heads,
                     long long stride_h, long long stride_t, int group) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = row_map_encoder();
  if (encode == nullptr || base == nullptr || tokens < 1 || group < 1 || group > 128 ||
      (group & (group - 1)) != 0 || heads < group)
    return false;
  if (reinterpret_cast<uintptr_t>(base) % 16 != 0 || stride_h % 16 != 0 || stride_t % 16 != 0 ||
      stride_h <= 0 || stride_t <= 0)
    return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(heads),
                        static_cast<cuuint64_t>(tokens)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride_h), static_cast<cuuint64_t>(stride_t)};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(kM / group)};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
                box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int prefill_smem_bytes() { return kSmemBytes<0>; }

namespace {

template <int kFormat>
cudaError_t launch_format(const CUtensorMap& kmap, const CUtensorMap& vmap,
                          const PrefillArgs& args, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_set{0};
  const auto kern = paged_prefill_kernel<kFormat>;
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
  const bool mostly_new = kFormat != 0 && 2ll * a.q_len >= a.longest;
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

cudaError_t launch_paged_prefill(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                 const PrefillArgs& args, cudaStream_t stream) {
  return launch_format<0>(kmap, vmap, args, stream);
}

cudaError_t launch_paged_prefill_q8(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                    const PrefillArgs& args, int format, cudaStream_t stream) {
  return format == kFormatE4m3 ? launch_format<kFormatE4m3>(kmap, vmap, args, stream)
                               : launch_format<kFormatInt8>(kmap, vmap, args, stream);
}

}  // namespace pkvqk
