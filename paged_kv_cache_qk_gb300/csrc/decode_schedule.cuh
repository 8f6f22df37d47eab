// Work schedule, row destinations and ring drain shared by the paged decode
// kernels (bf16 and 8-bit caches): which runs of key tiles a CTA walks (split
// or balanced schedule, see decode.cu), and where a row's result goes.
#pragma once

#include "device_common.cuh"
#include "kernels.h"
#include "score_rules.cuh"

namespace pkvqk {

constexpr float kLn2 = 0.693147180559945309f;

constexpr int kDestFinal = 0;   // bf16 output + lse
constexpr int kDestSplit = 1;   // partial at [row][split] (split schedule)
constexpr int kDestSlot = 2;    // partial at [slot][row in unit] (balanced schedule)

// A run of 16-key tiles of one (sequence, head group): keys [k0, k1).
struct Segment {
  int b, hg, seq_len, k0, k1, ntiles, dest, split;
  int first;                // scored: keys below it are visible to no row of the sequence
  long long slot;
};

__device__ __forceinline__ int clamped_len(const DecodeArgs& a, int b) {
  int L = a.seq_lens[b];
  if (L < 0) L = 0;
  const long long cap = static_cast<long long>(a.max_blocks_per_seq) * a.block_size;
  if (L > cap) {
    report(a.status_flags, kFlagBadBlock);
    L = static_cast<int>(cap);
  }
  return L;
}

// Pages of a sequence of L keys that the call walks: all of them, or with score rules
// those from the first key that a row sees.
struct PageSpan {
  int first_key, first_page, pages;
};

template <bool kScored>
__device__ __forceinline__ PageSpan page_span(const DecodeArgs& a, int b, int L) {
  const int P = (L + a.block_size - 1) / a.block_size;
  if constexpr (!kScored) {
    return {0, 0, P};
  } else {
    if (a.rules.window == 0 && a.rules.first_keys == nullptr) return {0, 0, P};
    const int p = L - a.q_len;                 // position of the sequence's first row
    int lo = window_start(a.rules, p);
    if (a.rules.first_keys != nullptr) {
      // the first key that a row sees; a row that sees none has no say
      const int past = prefix_end(a.rules, b, L);
      lo = L;
      for (int t = 0; t < a.q_len; ++t) {
        const int key = max(window_start(a.rules, p + t),
                            a.rules.first_keys[static_cast<long long>(b) * a.q_len + t]);
        if (key < max(p + t + 1, past)) lo = min(lo, key);
      }
    }
    lo = min(lo, L);
    const int first_page = lo < L ? lo / a.block_size : P;
    return {lo, first_page, P - first_page};
  }
}

template <bool kScored = false>
__device__ __forceinline__ long long unit_pages(const DecodeArgs& a, int u) {
  const int b = u % a.batch;
  return page_span<kScored>(a, b, clamped_len(a, b)).pages;
}

__device__ __forceinline__ void set_range(Segment& s, int k0, int k1, int tk) {
  s.k0 = k0;
  s.k1 = k1;
  s.ntiles = k1 > k0 ? (k1 - k0 + tk - 1) / tk : 0;
}

// Balanced schedule of this CTA: its page range and where its walk starts.
struct Plan {
  long long tp, lo, hi;     // total pages; this CTA's pages [lo, hi)
  long long g_eff;          // CTAs that get pages: min(grid, total pages)
  int u_start;              // first unit with pages at or after lo
  long long s_start;        // pages before unit u_start
};

// Produces the CTA's segments in order; producer and consumers each run
// their own copy and see the same sequence.
template <bool kScored = false>
struct SegmentSourceOf {
  const DecodeArgs* a;
  const Plan* plan;
  int tk;                   // keys per tile
  int balanced;
  int done;
  int u;
  long long s;              // pages before unit u

  __device__ void init(const DecodeArgs& args, const Plan* p, int tile_keys) {
    a = &args;
    plan = p;
    tk = tile_keys;
    balanced = args.num_splits == 0;
    done = 0;
    u = 0;
    s = 0;
    if (balanced) {
      u = p->u_start;
      s = p->s_start;
    }
  }

  // pages [p0, p1) of the span; a scored sequence starts at its first key's tile
  __device__ __forceinline__ void set_pages(Segment& seg, const PageSpan& span, int p0, int p1) {
    int k0 = (span.first_page + p0) * a->block_size;
    if (kScored) k0 = max(k0, span.first_key & ~(tk - 1));
    seg.first = span.first_key;
    set_range(seg, k0, min((span.first_page + p1) * a->block_size, seg.seq_len), tk);
  }

  __device__ bool next(Segment& seg) {
    if (!balanced) {
      if (done) return false;
      done = 1;
      seg.b = blockIdx.z;
      seg.hg = blockIdx.y;
      seg.split = blockIdx.x;
      seg.slot = 0;
      seg.seq_len = clamped_len(*a, seg.b);
      const PageSpan span = page_span<kScored>(*a, seg.b, seg.seq_len);
      const int P = span.pages;
      int p0 = seg.split * a->chunk_pages;
      int p1 = (seg.split == a->num_splits - 1) ? P : p0 + a->chunk_pages;
      p0 = min(p0, P);
      p1 = min(p1, P);
      set_pages(seg, span, p0, p1);
      seg.dest = a->num_splits == 1 ? kDestFinal : kDestSplit;
      return true;
    }
    const int U = a->batch * a->groups;
    while (u < U && s < plan->hi) {
      const int cur = u;
      const long long start = s;
      const int len = clamped_len(*a, cur % a->batch);
      const PageSpan span = page_span<kScored>(*a, cur % a->batch, len);
      const long long P = span.pages;
      u += 1;
      s += P;
      const long long plo = max(start, plan->lo) - start;
      const long long phi = min(s, plan->hi) - start;
      if (phi <= plo) continue;                            // empty unit or no overlap
      seg.b = cur % a->batch;
      seg.hg = cur / a->batch;
      seg.split = 0;
      seg.seq_len = len;
      set_pages(seg, span, static_cast<int>(plo), static_cast<int>(phi));
      const bool whole = plo == 0 && phi == P;
      seg.dest = whole ? kDestFinal : kDestSlot;
      seg.slot = static_cast<long long>(blockIdx.x) + cur;
      // the CTA holding the unit's first page records which CTAs cut it:
      // page x belongs to CTA floor(((x + 1) * G' - 1) / TP), G' = g_eff
      if (start >= plan->lo && threadIdx.x == 0) {
        const int c_last = static_cast<int>((s * plan->g_eff - 1) / plan->tp);
        a->unit_info[cur] = make_int2(blockIdx.x, c_last);
      }
      return true;
    }
    return false;
  }
};

using SegmentSource = SegmentSourceOf<>;

// Block-wide plan of the balanced schedule (every thread takes part).
template <bool kScored = false>
__device__ inline void make_plan(const DecodeArgs& a, Plan* plan, long long* wsum) {
  const int U = a.batch * a.groups;
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nwarps = nt >> 5;
  const int chunk = (U + nt - 1) / nt;
  const int u_lo = min(U, tid * chunk), u_hi = min(U, u_lo + chunk);
  long long mine = 0;
  for (int u = u_lo; u < u_hi; ++u) mine += unit_pages<kScored>(a, u);
  long long v = mine;                                       // inclusive warp scan
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  if (lane == 31) wsum[warp] = v;
  if (tid == 0) plan->u_start = U;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < nwarps ? wsum[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long n = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += n;
    }
    if (lane < nwarps) wsum[lane] = w;
  }
  __syncthreads();
  const long long tp = wsum[nwarps - 1];
  const long long before = (warp ? wsum[warp - 1] : 0) + v - mine;   // pages before u_lo
  // with fewer pages than CTAs only the first tp CTAs get pages, so that
  // every CTA between a unit's first and last owner holds some of it
  const long long G = min(static_cast<long long>(gridDim.x), tp > 0 ? tp : 1);
  const long long c = blockIdx.x;
  const long long lo = c < G ? c * tp / G : tp, hi = c < G ? (c + 1) * tp / G : tp;
  long long run = before;
  for (int u = u_lo; u < u_hi; ++u) {
    const long long P = unit_pages<kScored>(a, u);
    if (run + P > lo) {
      atomicMin(&plan->u_start, u);
      break;
    }
    run += P;
  }
  __syncthreads();
  run = before;
  for (int u = u_lo; u < u_hi; ++u) {
    if (u == plan->u_start) plan->s_start = run;
    run += unit_pages<kScored>(a, u);
  }
  if (tid == 0) {
    plan->tp = tp;
    plan->lo = lo;
    plan->hi = hi;
    plan->g_eff = G;
    if (plan->u_start == U) plan->s_start = tp;
  }
  __syncthreads();
}

// Units without any key: zero output, lse -inf, nothing to combine.  Unit u
// is handled by CTA u mod G (all threads of the CTA).
template <bool kScored = false>
__device__ inline void write_empty_units(const DecodeArgs& a, int hpc) {
  const int U = a.batch * a.groups;
  for (int u = blockIdx.x; u < U; u += gridDim.x) {
    if (unit_pages<kScored>(a, u) != 0) continue;
    const int b = u % a.batch, hg = u / a.batch;
    const int rows = a.rows_per_unit;
    for (int idx = threadIdx.x; idx < rows * (kHeadDim / 8); idx += blockDim.x) {
      const int r = idx / (kHeadDim / 8), c8 = idx % (kHeadDim / 8);
      // unit row r = (t * HPC + hh) * group + gi
      const int gi = r % a.group, th = r / a.group, hh = th % hpc, t = th / hpc;
      const int h = (hg * hpc + hh) * a.group + gi;
      const long long row = (static_cast<long long>(b) * a.q_len + t) * a.num_q_heads + h;
      *reinterpret_cast<uint4*>(a.out + row * kHeadDim + c8 * 8) = make_uint4(0, 0, 0, 0);
      if (c8 == 0 && a.lse_out != nullptr) a.lse_out[row] = -INFINITY;
    }
    if (threadIdx.x == 0) a.unit_info[u] = make_int2(blockIdx.x, blockIdx.x);
  }
}

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  const uint32_t off = (1024u - (smem_addr(p) & 1023u)) & 1023u;
  return p + off;
}

// After a timeout: wait (bounded) for the last copy issued into every stage
// so that no TMA write lands in shared memory after the CTA exits.
template <int STAGES>
__device__ void drain(uint64_t* full, int issued) {
  for (int s = 0; s < STAGES; ++s) {
    if (issued <= s) continue;
    const int last = s + ((issued - 1 - s) / STAGES) * STAGES;
    mbar_wait(&full[s], (last / STAGES) & 1);
  }
}

// -------------------------------------------------------- row destinations

struct RowDest {
  __nv_bfloat16* out;   // final bf16 row (or null)
  float* lse;           // final lse (or null)
  float* po;            // partial fp32 row (or null)
  float* plse;          // partial lse (or null)
};

template <int HPC>
__device__ __forceinline__ RowDest row_dest(const DecodeArgs& a, const Segment& seg, int t,
                                            int hh, int gi) {
  RowDest d{nullptr, nullptr, nullptr, nullptr};
  const int h = (seg.hg * HPC + hh) * a.group + gi;
  const long long row = (static_cast<long long>(seg.b) * a.q_len + t) * a.num_q_heads + h;
  if (seg.dest == kDestFinal) {
    d.out = a.out + row * kHeadDim;
    d.lse = a.lse_out != nullptr ? a.lse_out + row : nullptr;
  } else {
    const long long idx = seg.dest == kDestSplit
                              ? row * a.num_splits + seg.split
                              : seg.slot * a.rows_per_unit + (t * HPC + hh) * a.group + gi;
    d.po = a.ws_o + idx * kHeadDim;
    d.plse = a.ws_lse + idx;
  }
  return d;
}

// A row without a visible key has the sum l = 0; a NaN sum stays NaN.
__device__ __forceinline__ float final_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }

}  // namespace pkvqk
