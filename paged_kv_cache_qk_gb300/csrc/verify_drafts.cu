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
// below; the sum of 2^20 - 1 weights of at most 1 fits 64 bits), and their sum is multiplied
// by u_K in integers too (part_of).
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

#include <type_traits>

namespace pkvqk {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 4;
constexpr int kMaxCluster = 16;
constexpr int kDepth = 4;                      // loads of p (and of q) in flight a lane
constexpr int kGroups = 64;                    // sums kept a warp, of equal runs of its part

// A value's bits, and value i of words that hold them one after another.
template <typename T>
__device__ __forceinline__ uint32_t bits_at(const T* p) {
  if constexpr (sizeof(T) == 4) return *reinterpret_cast<const uint32_t*>(p);
  else return *reinterpret_cast<const uint16_t*>(p);
}
template <typename T>
__device__ __forceinline__ float value_in(const uint32_t* words, int i) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(words[i]);
  } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    return (i & 1) ? bf16hi(words[i >> 1]) : bf16lo(words[i >> 1]);
  } else {
    return __half2float(__ushort_as_half(static_cast<uint16_t>(words[i >> 1] >> (16 * (i & 1)))));
  }
}
template <typename T>
__device__ __forceinline__ float value_at(const T* p) {
  const uint32_t w = bits_at(p);
  return value_in<T>(&w, 0);
}

// A probability as a multiple of 2^-44, in two parts of fp32 and integer instructions
// (float to 64-bit integer runs at a small fraction of their rate: 64 sequences over 131072
// tokens took 50 us with it): x 2^22 rounded to a whole number h, the low bits of
// x 2^22 + 2^23, and what is left, x - h 2^-22 (exact), times 2^44 rounded to a whole number
// l, |l| <= 2^21, the low bits above 3 * 2^22.  The value is h 2^22 + l; the magic
// numbers' own bits stay in h and l until sums are formed.  NaN and below 0 count as 0,
// above 1 as 1.
struct Fixed {
  uint32_t h, l;
};
constexpr float kMagicH = 8388608.f, kMagicL = 12582912.f;
constexpr uint32_t kBitsH = 0x4b000000u, kBitsL = 0x4b400000u;

__device__ __forceinline__ Fixed fixed(float x) {
  const float s = __saturatef(x);
  const float h = fmaf(s, 4194304.f, kMagicH);
  const float rest = fmaf(kMagicH - h, 2.384185791015625e-07f, s);     // 2^-22
  return {__float_as_uint(h), __float_as_uint(fmaf(rest, 17592186044416.f, kMagicL))};
}

// 16 bytes of a row (kVec: it starts on a 16-byte boundary), or one value.
template <typename T, bool kVec>
struct Loaded {
  static constexpr int kCount = kVec ? 16 / static_cast<int>(sizeof(T)) : 1;
  uint32_t words[kVec ? 4 : 1];

  // elements at .. at + kCount - 1 of row
  __device__ __forceinline__ void load(const T* row, int at) {
    if constexpr (kVec) {
      const uint4 u = *reinterpret_cast<const uint4*>(row + at);
      words[0] = u.x;
      words[1] = u.y;
      words[2] = u.z;
      words[3] = u.w;
    } else {
      words[0] = bits_at(row + at);
    }
  }
  // the same; those from end on are 0
  __device__ __forceinline__ void load(const T* row, int at, int end) {
    if constexpr (kVec) {
      if (at + kCount <= end) {
        load(row, at);
      } else {
        constexpr int kEach = 4 / static_cast<int>(sizeof(T));       // values a word
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          words[k] = 0;
#pragma unroll
          for (int i = 0; i < kEach; ++i)
            if (at + k * kEach + i < end) words[k] |= bits_at(row + at + k * kEach + i) << (16 * i);
        }
      }
    } else {
      words[0] = at < end ? bits_at(row + at) : 0u;
    }
  }
  __device__ __forceinline__ float operator[](int i) const { return value_in<T>(words, i); }
};

// What the token is drawn from: p less `less` (a row of q, or one token's whole weight).
template <typename T>
struct Weights {
  const T* p;
  const T* q;                                  // or nullptr
  int token;                                   // weighs nothing; -1: none

  // Adds the weight of value i of a (and b) to h 2^22 + l (up to 512 weights: 32 bits each).
  template <bool kVec, bool kBoth>
  __device__ __forceinline__ void weigh(const Loaded<T, kVec>& a, const Loaded<T, kVec>& b, int at,
                                        int i, uint32_t& h, int32_t& l, bool& bad) const {
    const float x = a[i];
    bad = bad || !(x >= 0.f);
    const Fixed f = fixed(x);
    if (kBoth) {
      const float y = b[i];
      bad = bad || !(y >= 0.f);
      const Fixed less = fixed(y);
      // rounding keeps the order: above 0 only where x > y
      if (__saturatef(x) > __saturatef(y)) {
        h += f.h - less.h;
        l += static_cast<int32_t>(f.l - less.l);
      }
    } else if (at + i != token) {
      h += f.h - kBitsH;
      l += static_cast<int32_t>(f.l - kBitsL);
    }
  }
};

__device__ __forceinline__ unsigned long long joined(uint32_t h, int32_t l) {
  return (static_cast<unsigned long long>(h) << 22) + static_cast<long long>(l);
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The parts of two probabilities of [0, 1] at once (fixed, in packed instructions).
__device__ __forceinline__ void fixed2(float x0, float x1, uint32_t (&h)[2], uint32_t (&l)[2]) {
  const uint64_t x = pack2(x0, x1);
  const uint64_t hi = fma2(x, pack2(4194304.f, 4194304.f), pack2(kMagicH, kMagicH));
  // x - (hi - 2^23) 2^-22, each step exact
  const uint64_t whole = add2(hi, pack2(-kMagicH, -kMagicH));
  const uint64_t rest = fma2(whole, pack2(-2.384185791015625e-07f, -2.384185791015625e-07f), x);
  const uint64_t lo = fma2(rest, pack2(17592186044416.f, 17592186044416.f),
                           pack2(kMagicL, kMagicL));
  float f0, f1;
  unpack2(hi, f0, f1);
  h[0] = __float_as_uint(f0);
  h[1] = __float_as_uint(f1);
  unpack2(lo, f0, f1);
  l[0] = __float_as_uint(f0);
  l[1] = __float_as_uint(f1);
}

// Largest value by its bits, which order as whole numbers; negative ones and NaN come last.
template <typename T>
__device__ __forceinline__ uint32_t largest(uint32_t m, uint32_t word) {
  if constexpr (sizeof(T) == 4) return max(m, word);
  else return __vmaxu2(m, word);
}
// whether it (of both halves, for 16-bit types) is at most 1
template <typename T>
__device__ __forceinline__ bool at_most_one(uint32_t m) {
  constexpr uint32_t kOne = sizeof(T) == 4 ? 0x3f800000u
                            : std::is_same<T, __nv_bfloat16>::value ? 0x3f80u
                                                                    : 0x3c00u;
  if constexpr (sizeof(T) == 4) return m <= kOne;
  else return (m & 0xffffu) <= kOne && (m >> 16) <= kOne;
}

// This warp's sum of the weights of [begin, end), run by run: sums[g] holds the g-th run of
// `run` values, a multiple of what the warp takes in one step.  A lane's values of a step
// that all lie in [0, 1], none of them the token without weight, go in packed
// instructions; others one by one.
template <typename T, bool kVec, bool kBoth>
__device__ __forceinline__ unsigned long long sum_part(const Weights<T>& w, int begin, int end,
                                                       int run, unsigned long long* sums,
                                                       bool& bad) {
  using Vec = Loaded<T, kVec>;
  constexpr int kStep = 32 * Vec::kCount;
  constexpr int kWords = sizeof(Vec) / 4;
  const int lane = threadIdx.x & 31;
  unsigned long long total = 0;
  for (int from = begin, g = 0; from < end; from += run, ++g) {
    const int to = min(end, from + run);
    const bool holds_token = !kBoth && w.token >= from && w.token < to;
    unsigned long long sum = 0;
    for (int at = from + lane * Vec::kCount; at < to; at += kDepth * kStep) {
      Vec a[kDepth], b[kDepth];
      if (at + (kDepth - 1) * kStep + Vec::kCount <= to) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) a[d].load(w.p, at + d * kStep);
        if (kBoth) {
#pragma unroll
          for (int d = 0; d < kDepth; ++d) b[d].load(w.q, at + d * kStep);
        }
      } else {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) a[d].load(w.p, at + d * kStep, to);
        if (kBoth) {
#pragma unroll
          for (int d = 0; d < kDepth; ++d) b[d].load(w.q, at + d * kStep, to);
        }
      }
      uint32_t most = 0;
#pragma unroll
      for (int d = 0; d < kDepth; ++d)
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
          most = largest<T>(most, a[d].words[k]);
          if (kBoth) most = largest<T>(most, b[d].words[k]);
        }
      uint32_t h = 0;
      int32_t l = 0;
      if (at_most_one<T>(most) && !holds_token) {
        constexpr int kValues = kDepth * Vec::kCount;
#pragma unroll
        for (int e = 0; e < kValues; e += 2) {
          const float x0 = a[e / Vec::kCount][e % Vec::kCount];
          const float x1 = a[(e + 1) / Vec::kCount][(e + 1) % Vec::kCount];
          uint32_t ph[2], pl[2];
          fixed2(x0, x1, ph, pl);
          if (kBoth) {
            const float y0 = b[e / Vec::kCount][e % Vec::kCount];
            const float y1 = b[(e + 1) / Vec::kCount][(e + 1) % Vec::kCount];
            uint32_t qh[2], ql[2];
            fixed2(y0, y1, qh, ql);
            if (x0 > y0) {
              h += ph[0] - qh[0];
              l += static_cast<int32_t>(pl[0] - ql[0]);
            }
            if (x1 > y1) {
              h += ph[1] - qh[1];
              l += static_cast<int32_t>(pl[1] - ql[1]);
            }
          } else {                             // the magic numbers' bits come out below
            h += ph[0] + ph[1];
            l += static_cast<int32_t>(pl[0] + pl[1]);
          }
        }
        if (!kBoth) {
          h -= kValues * kBitsH;
          l -= static_cast<int32_t>(kValues * kBitsL);
        }
      } else {
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
#pragma unroll
          for (int i = 0; i < Vec::kCount; ++i)
            w.template weigh<kVec, kBoth>(a[d], b[d], at + d * kStep, i, h, l, bad);
      }
      sum += joined(h, l);
    }
    sum = warp_sum(sum);
    if (lane == 0) sums[g] = sum;
    total += sum;
  }
  __syncwarp();
  return total;
}

// Inclusive sums over the lanes.
__device__ __forceinline__ unsigned long long warp_scan(unsigned long long v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long n = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += n;
  }
  return v;
}

// The whole part of u total, not rounded: u is m 2^-e with 24 bits of m, and the product's up to
// 88 bits are formed in two halves (fp32 weights give sums of 45 bits and more, so that a
// float64 product would round).  Below 0 and NaN u counts as 0, from 1 on as just below 1.
__device__ __forceinline__ unsigned long long part_of(float u, unsigned long long total) {
  if (!(u > 0.f)) return 0;
  if (u >= 1.f) return total - 1;
  const uint32_t bits = __float_as_uint(u);
  const int exponent = static_cast<int>(bits >> 23);         // 0 .. 126; 0: subnormal
  const unsigned long long m = (bits & 0x7fffffu) | (exponent > 0 ? 0x800000u : 0u);
  const int e = 150 - max(exponent, 1);                      // 24 .. 149
  const unsigned long long lo = m * total, hi = __umul64hi(m, total);
  if (e < 64) return hi << (64 - e) | lo >> e;               // hi < 2^24
  return e < 128 ? hi >> (e - 64) : 0;
}

// The first element of [begin, end) at which `before` and the weights so far pass t
// (one warp, all lanes; the caller knows that there is one).  sums, run: sum_part's.
template <typename T, bool kVec, bool kBoth>
__device__ __noinline__ int find_in_part(const Weights<T>& w, int begin, int end, int run,
                                            const unsigned long long* sums,
                                            unsigned long long before, unsigned long long t) {
  using Vec = Loaded<T, kVec>;
  constexpr int kStep = 32 * Vec::kCount;
  const int lane = threadIdx.x & 31;
  bool bad = false;
  while (end - begin > run && before + *sums <= t) {     // the run that holds it
    before += *sums++;
    begin += run;
  }
  end = min(end, begin + run);
  for (int from = begin; from < end; from += kDepth * kStep) {
    // the step that holds it, then the vector again
    unsigned long long sums_of[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int at = from + lane * Vec::kCount + d * kStep;
      Vec a, b;
      a.load(w.p, at, end);
      if (kBoth) b.load(w.q, at, end);
      uint32_t h = 0;
      int32_t l = 0;
#pragma unroll
      for (int i = 0; i < Vec::kCount; ++i) w.template weigh<kVec, kBoth>(a, b, at, i, h, l, bad);
      sums_of[d] = joined(h, l);
    }
    int step = -1;
    unsigned long long mine = 0;
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const unsigned long long sum = warp_sum(sums_of[d]);
      if (step < 0) {
        if (before + sum > t) {
          step = d;
          mine = sums_of[d];
        } else {
          before += sum;
        }
      }
    }
    if (step < 0) continue;
    const unsigned long long upto = warp_scan(mine);
    const int owner = __ffs(__ballot_sync(0xffffffffu, before + upto > t)) - 1;
    const int at = from + lane * Vec::kCount + step * kStep;
    int found = at;
    if (lane == owner) {
      Vec a, b;
      a.load(w.p, at, end);
      if (kBoth) b.load(w.q, at, end);
      uint32_t h = 0;
      int32_t l = 0;
#pragma unroll
      for (int i = 0; i < Vec::kCount; ++i) {
        if (before + upto - mine + joined(h, l) <= t) found = at + i;   // not passed before i
        w.template weigh<kVec, kBoth>(a, b, at, i, h, l, bad);
      }
    }
    return __shfl_sync(0xffffffffu, found, owner);
  }
  return -1;
}

// How many drafts are kept (one warp, all lanes).  The drafts are asked for beside their
// number, so that two loads follow each other and not three.
template <typename T>
__device__ __forceinline__ int kept_drafts(const VerifyArgs& a, int b, int& n, int& token,
                                           bool& bad_token) {
  const int lane = threadIdx.x & 31;
  const T* p = static_cast<const T*>(a.target) + b * a.target_stride_b;
  const T* q = static_cast<const T*>(a.draft) + b * a.draft_stride_b;
  const int32_t* drafts = a.draft_tokens + static_cast<int64_t>(b) * a.max_drafts;
  const float* uniforms = a.uniforms + static_cast<int64_t>(b) * (a.max_drafts + 1);
  const int32_t* lens = a.draft_lens != nullptr ? a.draft_lens + b : nullptr;
  n = a.max_drafts;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    int x = -1;
    float u = 0.f;
    if (i < a.max_drafts) {
      x = drafts[i];
      u = uniforms[i];
    }
    if (i0 == 0 && lens != nullptr) n = max(0, min(n, *lens));
    bool keep = false;
    const bool known = x >= 0 && x < a.vocab;
    if (i < n && known) {
      // as the draw counts them: NaN and below 0 as 0, above 1 as 1
      const float px = __saturatef(value_at(p + i * a.target_stride_t + x));
      const float qx =
          a.draft != nullptr ? __saturatef(value_at(q + i * a.draft_stride_t + x)) : 1.f;
      keep = static_cast<double>(u) * qx < px;
    }
    const unsigned refused = __ballot_sync(0xffffffffu, !keep);
    if (refused != 0) {
      const int first = __ffs(refused) - 1;
      if (i0 + first >= n) return n;           // the lanes past the last draft
      token = __shfl_sync(0xffffffffu, x, first);
      bad_token = token < 0 || token >= a.vocab;
      return i0 + first;
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
  __shared__ unsigned long long run_sums[kWarps][kGroups];
  __shared__ unsigned long long cta_sums[2][kMaxCluster];   // [round][rank]
  __shared__ int s_kept, s_drafts, s_token, s_bad_token;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
  const int b = blockIdx.y;
  cluster_arrive();                            // this CTA's shared memory is there

  pdl_launch_dependents();
  pdl_wait();
  // what the end needs, on its way from the start
  const float u = a.uniforms[static_cast<int64_t>(b) * (a.max_drafts + 1) + a.max_drafts];
  const int seq_len = a.kept_lens != nullptr && rank == 0 ? a.seq_lens[b] : 0;
  if (warp == 0) {
    bool bad_token = false;
    int n, token = -1;
    const int j = kept_drafts<T>(a, b, n, token, bad_token);
    if (lane == 0) {
      s_kept = j;
      s_drafts = n;
      s_token = token;
      s_bad_token = bad_token;
    }
  }
  __syncwarp();
  cluster_wait();
  __syncthreads();
  const int j = s_kept, n = s_drafts;
  const bool refused = j < n;
  const int64_t draft_row = static_cast<int64_t>(b) * a.max_drafts;

  Weights<T> w;
  w.p = static_cast<const T*>(a.target) + b * a.target_stride_b + j * a.target_stride_t;
  w.q = refused && a.draft != nullptr
            ? static_cast<const T*>(a.draft) + b * a.draft_stride_b + j * a.draft_stride_t
            : nullptr;
  w.token = refused && a.draft == nullptr ? s_token : -1;

  // slices of whole 16-byte pieces
  constexpr int kPiece = 16 / static_cast<int>(sizeof(T));
  const int pieces = (a.vocab + kPiece - 1) / kPiece;
  const int per_warp = (pieces + ranks * kWarps - 1) / (ranks * kWarps) * kPiece;
  const int part = rank * kWarps + warp;
  const int begin = static_cast<int>(min(static_cast<long long>(a.vocab),
                                         static_cast<long long>(part) * per_warp));
  const int end = min(a.vocab, begin + per_warp);

  // runs of whole steps, at most kGroups of them
  constexpr int kStep = kDepth * 32 * Loaded<T, kVec>::kCount;
  const int run = (per_warp + kGroups * kStep - 1) / (kGroups * kStep) * kStep;

  unsigned long long total = 0, before = 0;
  bool bad = false;
  for (int round = 0; round < 2; ++round) {
    const unsigned long long mine =
        w.q != nullptr ? sum_part<T, kVec, true>(w, begin, end, run, run_sums[warp], bad)
                       : sum_part<T, kVec, false>(w, begin, end, run, run_sums[warp], bad);
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
    const unsigned long long t = part_of(u, total);
    for (int k = 0; k < warp; ++k) before += warp_sums[k];
    if (t >= before && t - before < warp_sums[warp]) {
      const int v =
          w.q != nullptr
              ? find_in_part<T, kVec, true>(w, begin, end, run, run_sums[warp], before, t)
              : find_in_part<T, kVec, false>(w, begin, end, run, run_sums[warp], before, t);
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
      if (a.kept_lens != nullptr) a.kept_lens[b] = seq_len - (n - j);
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
