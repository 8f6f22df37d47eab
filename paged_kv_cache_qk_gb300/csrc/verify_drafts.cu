// Verdict on drafted tokens: which of a sequence's drafts the target model keeps, and
// the token that follows them.
//
// For sequence b with n drafts x_i, target rows p_i (i <= n) and draft rows q_i (i < n),
// given uniforms u:  draft i is kept while u_i q_i(x_i) < p_i(x_i); j is the first that
// is not (n if all are).  The next token is drawn from w = max(p_j - q_j, 0), from p_n
// where all drafts are kept, and from p_j where w vanishes: the smallest v with
//     w(0) + .. + w(v) > u_K (w(0) + .. + w(V - 1)).
// Kept and drawn this way the tokens are distributed as the target's own.
//
// What decides a border must not depend on the order of a sum: u_i q_i(x_i) is formed
// in float64, where it is exact, and weights are summed as integers, multiples of
// 2^-44 (exact for every fp32 probability of 2^-20 and more, off by at most 2^-45
// below; the sum of 2^20 - 1 weights of at most 1 fits 64 bits).
//
// A sequence is a cluster of CTAs.  Each finds j by itself (one warp: two dependent
// gathers), then sums its slice of the vocabulary, a contiguous part a warp, and
// pushes the sum into every CTA of the cluster; after one cluster barrier the CTA, and
// in it the warp, that holds the crossing walks its part once more (L2 holds it) and
// writes the token.  Only the one row of p and of q that j names is read: the bytes
// that bound the call.
#include "device_common.cuh"
#include "kernels.h"

#include <cuda_fp16.h>

namespace pkvqk {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 2;
constexpr int kMaxCluster = 16;
constexpr int kDepth = 4;                      // vectors of p (and of q) in flight a lane
constexpr float kOne = 17592186044416.f;       // 2^44: weight 1

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }

// A probability as a multiple of 2^-44: NaN and below 0 count as 0, above 1 as 1.
__device__ __forceinline__ unsigned long long fixed(float x) {
  return __float2ull_rn(fminf(fmaxf(x, 0.f), 1.f) * kOne);
}

// 16 bytes of a row (kVec: it starts on a 16-byte boundary), or one value.
template <typename T, bool kVec>
struct Loaded {
  static constexpr int kCount = kVec ? 16 / static_cast<int>(sizeof(T)) : 1;
  union {
    uint4 raw;
    T t[kCount];
  };

  __device__ __forceinline__ Loaded() {}
  // elements at .. at + kCount - 1 of row; those from end on are 0
  __device__ __forceinline__ void load(const T* row, int at, int end) {
    if (kVec && at + kCount <= end) {
      raw = *reinterpret_cast<const uint4*>(row + at);
    } else {
#pragma unroll
      for (int i = 0; i < kCount; ++i) t[i] = at + i < end ? row[at + i] : T(0.f);
    }
  }
  __device__ __forceinline__ float operator[](int i) const { return as_float(t[i]); }
};

// What the token is drawn from: p less `less` (a row of q, or one token's whole weight).
template <typename T>
struct Weights {
  const T* p;
  const T* q;                                  // or nullptr
  int token;                                   // weighs nothing; -1: none

  template <bool kVec>
  __device__ __forceinline__ unsigned long long weigh(const Loaded<T, kVec>& a,
                                                      const Loaded<T, kVec>& b, int at, int i,
                                                      bool& bad) const {
    bad = bad || !(a[i] >= 0.f);
    unsigned long long w = fixed(a[i]);
    if (q != nullptr) {
      bad = bad || !(b[i] >= 0.f);
      const unsigned long long less = fixed(b[i]);
      w = w > less ? w - less : 0ull;
    }
    return at + i == token ? 0ull : w;
  }
};

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// This warp's sum of the weights of [begin, end).
template <typename T, bool kVec>
__device__ __forceinline__ unsigned long long sum_part(const Weights<T>& w, int begin, int end,
                                                       bool& bad) {
  using Vec = Loaded<T, kVec>;
  constexpr int kStep = 32 * Vec::kCount;
  const int lane = threadIdx.x & 31;
  unsigned long long sum = 0;
  for (int at = begin + lane * Vec::kCount; at < end; at += kDepth * kStep) {
    Vec a[kDepth], b[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) a[d].load(w.p, at + d * kStep, end);
    if (w.q != nullptr) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) b[d].load(w.q, at + d * kStep, end);
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
#pragma unroll
      for (int i = 0; i < Vec::kCount; ++i) sum += w.weigh(a[d], b[d], at + d * kStep, i, bad);
  }
  return warp_sum(sum);
}

// The first element of [begin, end) at which `before` and the weights so far pass t
// (one warp, all lanes; the caller knows that there is one).
template <typename T, bool kVec>
__device__ __forceinline__ int find_in_part(const Weights<T>& w, int begin, int end,
                                            unsigned long long before, unsigned long long t) {
  using Vec = Loaded<T, kVec>;
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (int from = begin; from < end; from += 32 * Vec::kCount) {
    const int at = from + lane * Vec::kCount;
    Vec a, b;
    a.load(w.p, at, end);
    if (w.q != nullptr) b.load(w.q, at, end);
    unsigned long long mine = 0;
#pragma unroll
    for (int i = 0; i < Vec::kCount; ++i) mine += w.weigh(a, b, at, i, bad);
    unsigned long long upto = mine;            // inclusive scan over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long n = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += n;
    }
    const unsigned passed = __ballot_sync(0xffffffffu, before + upto > t);
    if (passed != 0) {
      int found = 0;
      if (lane == __ffs(passed) - 1) {
        unsigned long long run = before + upto - mine;
        bool done = false;
#pragma unroll
        for (int i = 0; i < Vec::kCount; ++i) {
          run += w.weigh(a, b, at, i, bad);
          if (!done && run > t) {
            found = at + i;
            done = true;
          }
        }
      }
      return __shfl_sync(0xffffffffu, found, __ffs(passed) - 1);
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return -1;
}

// How many drafts are kept (one warp, all lanes).
template <typename T>
__device__ __forceinline__ int kept_drafts(const VerifyArgs& a, int b, int n, bool& bad_token) {
  const int lane = threadIdx.x & 31;
  const T* p = static_cast<const T*>(a.target) + b * a.target_stride_b;
  const T* q = static_cast<const T*>(a.draft) + b * a.draft_stride_b;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    bool keep = false, known = true;
    if (i < n) {
      const int x = a.draft_tokens[static_cast<int64_t>(b) * a.max_drafts + i];
      const float u = a.uniforms[static_cast<int64_t>(b) * (a.max_drafts + 1) + i];
      known = x >= 0 && x < a.vocab;
      if (known) {
        const float px = as_float(p[i * a.target_stride_t + x]);
        const float qx = a.draft != nullptr ? as_float(q[i * a.draft_stride_t + x]) : 1.f;
        keep = static_cast<double>(u) * qx < px;
      }
    }
    const unsigned refused = __ballot_sync(0xffffffffu, !keep);
    if (refused != 0) {
      const int first = __ffs(refused) - 1;
      bad_token = __shfl_sync(0xffffffffu, static_cast<int>(!known), first) != 0;
      return min(n, i0 + first);
    }
  }
  return n;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// v into the same shared variable of the cluster's CTA `rank`
__device__ __forceinline__ void push(unsigned long long* to, uint32_t rank, unsigned long long v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(to)), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) verify_drafts_kernel(const VerifyArgs a) {
  __shared__ unsigned long long warp_sums[kWarps];
  __shared__ unsigned long long cta_sums[2][kMaxCluster];   // [round][rank]
  __shared__ int s_kept, s_bad_token;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
  const int b = blockIdx.y;
  cluster_arrive();                            // this CTA's shared memory is there

  pdl_launch_dependents();
  pdl_wait();
  int n = a.max_drafts;
  if (a.draft_lens != nullptr) n = max(0, min(n, a.draft_lens[b]));
  if (warp == 0) {
    bool bad_token = false;
    const int j = kept_drafts<T>(a, b, n, bad_token);
    if (lane == 0) {
      s_kept = j;
      s_bad_token = bad_token;
    }
  }
  cluster_wait();
  __syncthreads();
  const int j = s_kept;
  const bool refused = j < n;
  const int64_t draft_row = static_cast<int64_t>(b) * a.max_drafts;

  Weights<T> w;
  w.p = static_cast<const T*>(a.target) + b * a.target_stride_b + j * a.target_stride_t;
  w.q = refused && a.draft != nullptr
            ? static_cast<const T*>(a.draft) + b * a.draft_stride_b + j * a.draft_stride_t
            : nullptr;
  w.token = refused && a.draft == nullptr ? a.draft_tokens[draft_row + j] : -1;

  // slices of whole 16-byte pieces
  constexpr int kPiece = 16 / static_cast<int>(sizeof(T));
  const int pieces = (a.vocab + kPiece - 1) / kPiece;
  const int per_warp = (pieces + ranks * kWarps - 1) / (ranks * kWarps) * kPiece;
  const int part = rank * kWarps + warp;
  const int begin = static_cast<int>(min(static_cast<long long>(a.vocab),
                                         static_cast<long long>(part) * per_warp));
  const int end = min(a.vocab, begin + per_warp);

  unsigned long long total = 0, before = 0;
  bool bad = false;
  for (int round = 0; round < 2; ++round) {
    const unsigned long long mine = sum_part<T, kVec>(w, begin, end, bad);
    if (lane == 0) warp_sums[warp] = mine;
    __syncthreads();
    if (warp == 0) {
      const unsigned long long cta = warp_sum(lane < kWarps ? warp_sums[lane] : 0ull);
      if (lane < ranks) push(&cta_sums[round][rank], lane, cta);
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    total = before = 0;
    for (int r = 0; r < ranks; ++r) {
      const unsigned long long s = cta_sums[round][r];
      total += s;
      if (r < rank) before += s;
    }
    // the same total in every CTA: all go round again, or none
    if (total != 0 || !refused) break;
    w.q = nullptr;                             // nothing is left of p less q: p itself
    w.token = -1;
  }
  if (bad) report(a.status_flags, kFlagBadValue);

  int32_t* tokens = a.tokens + static_cast<int64_t>(b) * (a.max_drafts + 1);
  if (total != 0) {
    float u = a.uniforms[static_cast<int64_t>(b) * (a.max_drafts + 1) + a.max_drafts];
    u = fminf(fmaxf(u, 0.f), 1.f);             // NaN: 0
    const double at = static_cast<double>(u) * static_cast<double>(total);
    const unsigned long long t =
        at >= static_cast<double>(total) ? total - 1 : min(total - 1, static_cast<unsigned long long>(at));
    for (int k = 0; k < warp; ++k) before += warp_sums[k];
    if (t >= before && t - before < warp_sums[warp]) {
      const int v = find_in_part<T, kVec>(w, begin, end, before, t);
      if (lane == 0) tokens[j] = v;
    }
  } else if (rank == 0 && threadIdx.x == 0) {
    tokens[j] = -1;
    report(a.status_flags, kFlagBadValue);
  }
  if (rank == 0) {
    for (int i = threadIdx.x; i <= a.max_drafts; i += kThreads)
      if (i != j) tokens[i] = i < j ? a.draft_tokens[draft_row + i] : -1;
    if (threadIdx.x == 0) {
      a.num_accepted[b] = j;
      if (a.kept_lens != nullptr) a.kept_lens[b] = a.seq_lens[b] - (n - j);
      if (s_bad_token) report(a.status_flags, kFlagBadToken);
    }
  }
}

template <typename T, bool kVec>
cudaError_t launch_one(const VerifyArgs& a, int cluster, cudaStream_t stream) {
  const auto kern = verify_drafts_kernel<T, kVec>;
  if (cluster > 8) {
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = set_once(
        [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); },
        allowed);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster, a.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename T>
cudaError_t launch_type(const VerifyArgs& a, int cluster, cudaStream_t stream) {
  // 16-byte loads where every row starts on a 16-byte boundary
  constexpr int kPiece = 16 / static_cast<int>(sizeof(T));
  bool vec = reinterpret_cast<uintptr_t>(a.target) % 16 == 0 && a.target_stride_b % kPiece == 0 &&
             a.target_stride_t % kPiece == 0;
  if (a.draft != nullptr)
    vec = vec && reinterpret_cast<uintptr_t>(a.draft) % 16 == 0 &&
          a.draft_stride_b % kPiece == 0 && a.draft_stride_t % kPiece == 0;
  return vec ? launch_one<T, true>(a, cluster, stream) : launch_one<T, false>(a, cluster, stream);
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs& a, int type, int sm_count,
                                 cudaStream_t stream) {
  if (a.batch == 0) return cudaSuccess;
  // CTAs a sequence: as many as keep one wave of resident CTAs and leave a CTA 1024
  // tokens or more
  int cluster = kMaxCluster;
  while (cluster > 1 && (static_cast<long long>(a.batch) * cluster > static_cast<long long>(kCtasPerSm) * sm_count ||
                         a.vocab / cluster < 1024))
    cluster >>= 1;
  switch (type) {
    case kProbFp32: return launch_type<float>(a, cluster, stream);
    case kProbBf16: return launch_type<__nv_bfloat16>(a, cluster, stream);
    case kProbFp16: return launch_type<__half>(a, cluster, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkvqk
