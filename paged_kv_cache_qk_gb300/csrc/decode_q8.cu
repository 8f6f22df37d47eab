// Split-KV paged decode attention (and the causal multi-query verify variant)
// over an 8-bit cache: codes (e4m3 or int8) with one scale per 16 slots of a
// page and kv head.
//
// For q row r and key n:  s_rn = scale * sk * <q_r, ck_n>,  out_r = sum_n
// softmax(s_r)_n sv cv_n.  Schedules, segments and destinations are those of the
// bf16 decode kernel (decode_schedule.cuh): split or balanced.
//
// Bound: the cache's bytes, 2 (128 + 4 / 16) per key and kv head.  What the SM
// has to do per byte is twice that of a bf16 cache, so the code per key counts:
//  * both products run as m16n8k16 f16 mma with the cache as the 16-row operand
//    and the q rows as the 8 columns (n-tiles: rows 0-7, 8-15): S^T = K Q^T and
//    O^T += V^T P^T.  A GQA group or verify block of up to 8 rows costs 16 mma per
//    16 keys where the q rows as the 16-row operand would cost 32, and a lane
//    holds 4 scores instead of 8.
//  * codes become f16 in registers (exact, q8_common.cuh).  K rows are read as
//    16-byte words; the dims a word brings to a k-step are the same for every key,
//    so q is laid out to match and K needs no transpose.  V comes through
//    transposing 8x8 b16 loads, whose pairs of adjacent dims are dealt to rows g
//    and g + 8 of the operand.  Lane group g reads key row ((g >> 1) | (g & 1) <<
//    2): consecutive groups then differ in swizzle bit 2 and the 16-byte reads
//    are free of bank conflicts.
//  * sk multiplies the fp32 score; log2 sv is added to it (x = s + log2 sv), P' =
//    2^(x - m) then carries sv into O and 1 / sv takes it out of the row sum:
//    P' <= 2^14 whatever the scales.  P' is rounded to f16 (2^-11), the row sum
//    takes it unrounded in fp32.
//  * the running reference m is raised only when a score passes it by 2^4, found
//    by a warp vote, so the usual tile has no shuffles and rescales nothing.
//  * two tiles go through a warp at once, so that one's loads and conversions fill
//    the latencies of the other's products (a tile alone takes a warp ~1050 cycles,
//    a pair ~1850; 64 sequences of mixed lengths, 4 kv heads: 68.9 -> 59.5 us).
// One warp per kv head at 8 heads a CTA, else two: they take the pairs in turn, by
// their place in the ring (decode_q8_ring.cuh), and merge at the end of a segment
// through shared memory.  The producer warp issues
// one TMA box for K and one for V per 16-key tile into the ring.  Scales are read
// by the consumer warps, one tile per lane, 32 tiles ahead (by the producer warp they
// held its boxes up every 32 tiles: 206 us against 158 on 64 x 8192).
//
// Measured: 64 sequences x 8192 keys, 16 q and 8 kv heads, 157 us = 6.85 TB/s (a plain
// copy 6.77; the bf16 cache 301 us); 8 x 32768 83 us = 6.47 TB/s; 64 mixed lengths at
// 32 q and 4 kv heads 51 us = 4.7 TB/s; 32 x 5 rows 75 us = 4.2 TB/s, where a warp's
// instructions for two n-tiles bound it.
#include "decode_q8_ring.cuh"
#include "decode_schedule.cuh"
#include "q8_common.cuh"

namespace pkvqk {

namespace {

constexpr int kTK = 16;                        // keys per tile: one scale group
static_assert(kTK == kScaleGroup, "a tile has one scale per head and tensor");
constexpr int kHeadTileBytes = kTK * kHeadDim;
constexpr float kHeadroom = 4.f;               // log2 by which a score may pass m
constexpr float kBias = 10.f;                  // P' = 2^(x - m + kBias) <= 2^14

template <int HPC, int NT>
struct GeometryQ8 : RingQ8<HPC, NT> {
  using Ring = RingQ8<HPC, NT>;
  static_assert(Ring::kStageBytes == 2 * HPC * kHeadTileBytes, "a stage holds K and V of a tile");
  static constexpr int kQBytes = Ring::kQInSmem ? 8 * NT * 32 * 8 : 0;
  // one n-tile of a warp's result, per head: O, then (l, mu, top) of two rows a lane
  static constexpr int kMergeBytes = Ring::kSplit > 1 ? 32 * (32 + 6) * 4 : 0;
  static constexpr int kOffMerge = Ring::kStages * Ring::kStageBytes;
  static constexpr int kOffQ = kOffMerge + HPC * kMergeBytes;
  static constexpr int kSmemBytes = kOffQ + Ring::kConsumers * kQBytes + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
  static constexpr int kThreads = (Ring::kConsumers + 1) * 32;
};

// ----------------------------------------------------------------- producer

template <int HPC, int NT>
__device__ void produce_q8(const CUtensorMap* kmap, const CUtensorMap* vmap, const DecodeArgs& a,
                           const Plan* plan, uint8_t* stages, uint64_t* full, uint64_t* empty,
                           volatile int* abort_flag, int* issued_out) {
  using Geo = GeometryQ8<HPC, NT>;
  constexpr int STAGES = Geo::kStages;
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
    prefetch_tensormap(kmap);
    prefetch_tensormap(vmap);
  }
  const uint64_t pol = l2_evict_first_policy();
  SegmentSource src;
  src.init(a, plan, kTK);
  Segment seg;
  int it = 0;
  bool ok = true;
  while (ok && src.next(seg)) {
    const int32_t* bt = a.block_tables + static_cast<int64_t>(seg.b) * a.max_blocks_per_seq;
    const int tiles = paired(seg.ntiles);
    for (int i0 = 0; i0 < tiles && ok; i0 += 32) {
      int blk = static_cast<int>(a.num_blocks), slot0 = 0;   // outside the cache: zeros
      const int i = i0 + lane;
      if (i < seg.ntiles) {
        const int key = seg.k0 + i * kTK;
        const int page = key / a.block_size;
        slot0 = key - page * a.block_size;
        blk = __ldg(bt + page);
        if (blk < 0 || blk >= a.num_blocks) report(a.status_flags, kFlagBadBlock);
      }
      const int n = min(32, tiles - i0);
      for (int j = 0; j < n; ++j) {
        const int bj = __shfl_sync(0xffffffffu, blk, j);
        const int sj = __shfl_sync(0xffffffffu, slot0, j);
        int good = 1;
        if (lane == 0) {
          const int s = it % STAGES;
          if (it >= STAGES) good = mbar_wait(&empty[s], ((it / STAGES) - 1) & 1) ? 1 : 0;
          if (good) {
            mbar_arrive_expect_tx(&full[s], Geo::kStageBytes);
            uint8_t* dst = stages + s * Geo::kStageBytes;
            // blocks outside the cache read as zeros
            tma_load_4d(dst, kmap, &full[s], 0, sj, seg.hg * HPC, bj, pol);
            tma_load_4d(dst + HPC * kHeadTileBytes, vmap, &full[s], 0, sj, seg.hg * HPC, bj, pol);
          } else {
            *abort_flag = 1;
            report(a.status_flags, kFlagTimeout);
          }
        }
        good = __shfl_sync(0xffffffffu, good, 0);
        if (!good) {
          ok = false;
          break;
        }
        ++it;
      }
    }
  }
  if (lane == 0) *issued_out = it;
}

// ----------------------------------------------------------------- consumer

// D += A (16x16, row) * B (16x8, col), f16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t& r0, uint32_t& r1,
                                              uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

// The scales of tile i of a segment (one lane per tile); 1 outside the segment
// and for block ids outside the cache.
__device__ __forceinline__ float2 tile_scales(const DecodeArgs& a, const ScaleView& sv,
                                              const Segment& seg, int kvh, int i) {
  if (i >= seg.ntiles) return make_float2(1.f, 1.f);
  const int key = seg.k0 + i * kTK;
  const int page = key / a.block_size;
  const int blk = __ldg(a.block_tables + static_cast<int64_t>(seg.b) * a.max_blocks_per_seq + page);
  if (blk < 0 || blk >= a.num_blocks) return make_float2(1.f, 1.f);
  const int64_t o = blk * sv.block_stride +
                    ((key - page * a.block_size) / kScaleGroup) * sv.group_stride +
                    kvh * sv.head_stride;
  return make_float2(__ldg(sv.k + o), __ldg(sv.v + o));
}

template <int HPC, int NT, int kFormat>
__device__ void consume_q8(const DecodeArgs& a, const ScaleView& sv, const Plan* plan,
                           uint8_t* stages, uint64_t* full, uint64_t* empty, uint64_t* merge_full,
                           uint64_t* merge_empty, volatile int* abort_flag) {
  using Geo = GeometryQ8<HPC, NT>;
  constexpr int STAGES = Geo::kStages;
  constexpr int kSplit = Geo::kSplit;
  const int lane = threadIdx.x & 31;
  const int hh = (threadIdx.x >> 5) % HPC, part = (threadIdx.x >> 5) / HPC;
  const int g = lane >> 2, c = lane & 3;
  const int R = a.q_len * a.group;
  const int krow = (g >> 1) | ((g & 1) << 2);  // key row of lane group g
  const int vrow = (lane & 7) >> 1 | ((lane & 1) << 2);

  // shared-memory offsets of this lane's reads, within a head's tile
  uint32_t koff[2], voff[4];
#pragma unroll
  for (int j = 0; j < 2; ++j) koff[j] = swz128(krow, c + 4 * j);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    voff[i] = swz128((((lane >> 3) & 1) << 3) + vrow, 2 * i + (lane >> 4));

  SegmentSource src;
  src.init(a, plan, kTK);
  Segment seg;
  int it0 = 0;                                 // ring position of the segment's first tile
  uint32_t merges = 0;
  bool aborted = false;
  for (; !aborted && src.next(seg); it0 += paired(seg.ntiles)) {
    const int kvh = seg.hg * HPC + hh;
    float2 next = tile_scales(a, sv, seg, kvh, lane);

    // q rows as f16, dims in the order the K words bring them
    uint32_t qb[Geo::kQInSmem ? 1 : NT][8][2];
    const uint32_t q_frag = smem_addr(stages + Geo::kOffQ + (threadIdx.x >> 5) * Geo::kQBytes) + lane * 8;
    if (Geo::kQInSmem) __syncwarp();           // reads of the segment before
    float rf[NT][2];                           // score factor of rows 2c, 2c + 1
    int lim[NT][2];
#pragma unroll(Geo::kQInSmem ? 1 : NT)
    for (int nt = 0; nt < NT; ++nt) {
      const int rr = 8 * nt + g;
      const int t = rr / a.group, gi = rr - t * a.group;
      const __nv_bfloat16* qrow =
          a.q + (static_cast<int64_t>(seg.b) * a.q_len + t) * a.q_stride_t +
          static_cast<int64_t>(kvh * a.group + gi) * a.q_stride_h;
      uint4 u[2][2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
          u[j][hf] = rr < R ? __ldg(reinterpret_cast<const uint4*>(qrow + 64 * j + 16 * c + 8 * hf))
                            : make_uint4(0u, 0u, 0u, 0u);
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float f[8];
          unpack8(u[j][hf], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
        }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      float inverse;
      const float up = q_row_scale(amax, inverse);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float f[8];
          unpack8(u[j][hf], f);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int step = j * 4 + hf * 2 + w;
            const uint32_t b0 = pack_f16x2(f[4 * w] * up, f[4 * w + 1] * up);
            const uint32_t b1 = pack_f16x2(f[4 * w + 2] * up, f[4 * w + 3] * up);
            if constexpr (Geo::kQInSmem) {
              asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(q_frag + (step * NT + nt) * 256),
                           "r"(b0), "r"(b1)
                           : "memory");
            } else {
              qb[nt][step][0] = b0;
              qb[nt][step][1] = b1;
            }
          }
        }
      const float mine = inverse * a.scale_log2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float factor = __shfl_sync(0xffffffffu, mine, (2 * c + e) * 4);
        const int row = 8 * nt + 2 * c + e;
        const int end = row < R ? min(seg.seq_len - a.q_len + row / a.group + 1, seg.k1) : 0;
        if (nt == 0) {
          rf[0][e] = factor;
          lim[0][e] = end;
        } else {
          rf[NT - 1][e] = factor;
          lim[NT - 1][e] = end;
        }
      }
    }
    const int lim_all = min(seg.seq_len - a.q_len + 1, seg.k1);   // visible to every row

    float o[NT][8][4], mu[NT][2], top[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
        o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mu[nt][e] = 0.f;                       // P' = 2^(x - mu)
        top[nt][e] = -INFINITY;                // a score above it raises mu
        l[nt][e] = 0.f;
      }
    }

    float ks_l = 1.f, lv_l = 0.f, iv_l = 1.f;
    // tiles i and i + 1 of the segment at once; false: a wait gave up
    constexpr int U = 2;
    auto pair = [&](int i) {
      const int it = it0 + i;
      float ks[U], lv[U], iv[U];
      uint32_t kt[U];                          // shared-memory address of the K tile
#pragma unroll
      for (int u = 0; u < U; ++u) {
        ks[u] = __shfl_sync(0xffffffffu, ks_l, (i + u) & 31);
        lv[u] = __shfl_sync(0xffffffffu, lv_l, (i + u) & 31);
        iv[u] = __shfl_sync(0xffffffffu, iv_l, (i + u) & 31);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int s = (it + u) % STAGES;
        if (!mbar_wait(&full[s], ((it + u) / STAGES) & 1)) return false;
        kt[u] = smem_addr(stages + s * Geo::kStageBytes + hh * kHeadTileBytes);
      }
      constexpr uint32_t kToV = HPC * kHeadTileBytes;
      const int key0 = seg.k0 + i * kTK;

      // slots past the sequence's end may hold anything; P' is 0 there, but an
      // e4m3 code can be NaN, so their V rows are zeroed (this warp's own)
      if (kFormat == kFormatE4m3 && key0 + U * kTK > seg.seq_len) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r0 = min(max(0, seg.seq_len - key0 - u * kTK), kTK);
          for (int e = r0 * 8 + lane; e < kTK * 8; e += 32)
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(kt[u] + kToV + e * 16),
                         "r"(0)
                         : "memory");
        }
        __syncwarp();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the next TMA write
      }

      // S^T (16 keys x 8 rows) = K Q^T over 8 steps of 16 dims; with one n-tile the
      // two halves of the dims in chains of their own
      constexpr int kChains = NT == 1 ? 2 : 1;
      float sc[U][NT][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float chain[kChains][NT][4];
#pragma unroll
        for (int j = 0; j < kChains; ++j)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            chain[j][nt][0] = chain[j][nt][1] = chain[j][nt][2] = chain[j][nt][3] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 ka = lds128(kt[u] + koff[j]), kb = lds128(kt[u] + koff[j] + 8 * 128);
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a0, a1, a2, a3;
            codes_adjacent<kFormat>(wa[w], a0, a2);
            codes_adjacent<kFormat>(wb[w], a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t b0, b1;
              if constexpr (Geo::kQInSmem)
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                             : "=r"(b0), "=r"(b1)
                             : "r"(q_frag + ((j * 4 + w) * NT + nt) * 256));
              else {
                b0 = qb[nt][j * 4 + w][0];
                b1 = qb[nt][j * 4 + w][1];
              }
              mma_f16(chain[j % kChains][nt], a0, a1, a2, a3, b0, b1);
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[u][nt][e] = kChains == 2 ? chain[0][nt][e] + chain[kChains - 1][nt][e]
                                        : chain[0][nt][e];
      }

      // x = s + log2 sv (log2 units); elements 0, 1: key krow, 2, 3: key krow + 8
      bool above = false;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[u][nt][e] = fmaf(sc[u][nt][e], rf[nt][e & 1] * ks[u], lv[u]);
      if (key0 + U * kTK > lim_all) {          // some row does not see all these keys
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key0 + u * kTK + krow + (e >> 1) * 8 >= lim[nt][e & 1]) sc[u][nt][e] = -INFINITY;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) above |= sc[u][nt][e] > top[nt][e & 1];
      if (__any_sync(0xffffffffu, above)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(fmaxf(sc[0][nt][e], sc[0][nt][2 + e]),
                            fmaxf(sc[1][nt][e], sc[1][nt][2 + e]));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            if (m > top[nt][e]) {              // uniform over the row's lanes
              const float now = m - kBias;
              const float alpha = top[nt][e] == -INFINITY ? 0.f : exp2f(mu[nt][e] - now);
              mu[nt][e] = now;
              top[nt][e] = m + kHeadroom;
              l[nt][e] *= alpha;
#pragma unroll
              for (int mt = 0; mt < 8; ++mt) {
                o[nt][mt][e] *= alpha;
                o[nt][mt][2 + e] *= alpha;
              }
            }
          }
      }
      uint32_t pb[U][NT][2];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = ex2_sfu(sc[u][nt][e] - mu[nt][e & 1]);
          l[nt][0] = fmaf(p[0] + p[2], iv[u], l[nt][0]);
          l[nt][1] = fmaf(p[1] + p[3], iv[u], l[nt][1]);
          pb[u][nt][0] = transpose8x8(pack_f16x2(p[0], p[1]));
          pb[u][nt][1] = transpose8x8(pack_f16x2(p[2], p[3]));
        }

      // O^T (128 dims x 8 rows) += V^T P^T; dims 2g, 2g + 1 of a 16-dim block sit
      // in operand rows g, g + 8
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
          uint32_t v0, v1, v2, v3;
          ldsm_x4_trans(kt[u] + kToV + voff[i4], v0, v1, v2, v3);
          uint32_t a0, a1, a2, a3;
          codes_alternate<kFormat>(v0, a0, a1);
          codes_alternate<kFormat>(v1, a2, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(o[nt][2 * i4], a0, a1, a2, a3, pb[u][nt][0], pb[u][nt][1]);
          codes_alternate<kFormat>(v2, a0, a1);
          codes_alternate<kFormat>(v3, a2, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(o[nt][2 * i4 + 1], a0, a1, a2, a3, pb[u][nt][0], pb[u][nt][1]);
        }
      __syncwarp();
      if (lane == 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) mbar_arrive(&empty[(it + u) % STAGES]);
      }
      return true;
    };
    for (int i = 0; i < seg.ntiles; i += U) {
      if ((i & 31) == 0) {                     // the next 32 tiles' scales
        ks_l = usable_scale(next.x);
        const float vs = usable_scale(next.y);
        lv_l = log2f(vs);
        iv_l = __frcp_rn(vs);
        next = tile_scales(a, sv, seg, kvh, i + 32 + lane);
      }
      if (kSplit > 1 && pair_owner(it0 + i, kSplit) != part) continue;   // the other warp's
      if (!pair(i)) {
        *abort_flag = 1;
        report(a.status_flags, kFlagTimeout);
        aborted = true;
        break;
      }
    }
    if (kSplit > 1 && aborted) break;

    // The end of a segment runs once or a few times, so its code is kept small: loops
    // over n-tiles and rows whose turn's values are always those of index 0.  Unrolled,
    // its first run waited on instruction fetches: 7 us, 13 us with two n-tiles.
#pragma unroll 1
    for (int nt = 0; nt < NT && !aborted; ++nt) {
      // two warps of a head: the second hands its rows over, one n-tile at a time
      if constexpr (kSplit > 1) {
        float4* mo = reinterpret_cast<float4*>(stages + Geo::kOffMerge + hh * Geo::kMergeBytes);
        float* ml = reinterpret_cast<float*>(mo + 8 * 32);
        bool ok = true;
        if (part == 1) {
          if (merges > 0) ok = mbar_wait(&merge_empty[hh], (merges - 1) & 1);
          if (ok) {
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
              mo[mt * 32 + lane] = make_float4(o[0][mt][0], o[0][mt][1], o[0][mt][2], o[0][mt][3]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              ml[(3 * e) * 32 + lane] = l[0][e];
              ml[(3 * e + 1) * 32 + lane] = mu[0][e];
              ml[(3 * e + 2) * 32 + lane] = top[0][e];
            }
          }
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(&merge_full[hh]);
        } else {
          ok = mbar_wait(&merge_full[hh], merges & 1);
          if (ok) {
            float w[2][2];                     // [row][this warp, the other]
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float mu1 = ml[(3 * e + 1) * 32 + lane];
              const bool has0 = top[0][e] != -INFINITY, has1 = ml[(3 * e + 2) * 32 + lane] != -INFINITY;
              const float m = has0 ? (has1 ? fmaxf(mu[0][e], mu1) : mu[0][e]) : mu1;
              w[e][0] = has0 ? exp2f(mu[0][e] - m) : 0.f;
              w[e][1] = has1 ? exp2f(mu1 - m) : 0.f;
              l[0][e] = l[0][e] * w[e][0] + ml[(3 * e) * 32 + lane] * w[e][1];
              mu[0][e] = m;
            }
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              const float4 x = mo[mt * 32 + lane];
              o[0][mt][0] = o[0][mt][0] * w[0][0] + x.x * w[0][1];
              o[0][mt][1] = o[0][mt][1] * w[1][0] + x.y * w[1][1];
              o[0][mt][2] = o[0][mt][2] * w[0][0] + x.z * w[0][1];
              o[0][mt][3] = o[0][mt][3] * w[1][0] + x.w * w[1][1];
            }
          }
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(&merge_empty[hh]);
        }
        ++merges;
        if (!ok) {
          *abort_flag = 1;
          report(a.status_flags, kFlagTimeout);
          aborted = true;
          break;
        }
      }
      if (kSplit == 1 || part == 0) {
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
          float sum = l[0][0];
          sum += __shfl_xor_sync(0xffffffffu, sum, 4);
          sum += __shfl_xor_sync(0xffffffffu, sum, 8);
          sum += __shfl_xor_sync(0xffffffffu, sum, 16);
          const int rr = 8 * nt + 2 * c + e;
          if (rr < R) {
            const int t = rr / a.group, gi = rr - t * a.group;
            const RowDest d = row_dest<HPC>(a, seg, t, hh, gi);
            const float inv = inverse_sum(sum), lse = final_lse(mu[0][0], sum);
            if (d.out != nullptr) {
#pragma unroll
              for (int mt = 0; mt < 8; ++mt)
                *reinterpret_cast<uint32_t*>(d.out + 16 * mt + 2 * g) =
                    pack_bf16x2(o[0][mt][0] * inv, o[0][mt][2] * inv);
              if (g == 0 && d.lse != nullptr) *d.lse = lse;
            } else {
#pragma unroll
              for (int mt = 0; mt < 8; ++mt)
                *reinterpret_cast<float2*>(d.po + 16 * mt + 2 * g) =
                    make_float2(o[0][mt][0] * inv, o[0][mt][2] * inv);
              if (g == 0) *d.plse = lse;
            }
          }
          l[0][0] = l[0][1];
          mu[0][0] = mu[0][1];
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            o[0][mt][0] = o[0][mt][1];
            o[0][mt][2] = o[0][mt][3];
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {            // the second n-tile's turn
        l[0][e] = l[NT - 1][e];
        mu[0][e] = mu[NT - 1][e];
        top[0][e] = top[NT - 1][e];
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[0][mt][e] = o[NT - 1][mt][e];
    }
  }
}

// Towards L2 while the previous kernel runs, as in the bf16 kernel: the first
// ring of tiles (split schedule) or the sequence lengths (balanced).  A prefetch
// binds no value; what decides its address is read past L1.
template <int HPC, int NT>
__device__ void prefetch_before_wait_q8(const CUtensorMap* kmap, const CUtensorMap* vmap,
                                        const DecodeArgs& a) {
  const int lane = threadIdx.x & 31;
  if (a.num_splits == 0) {
    for (int i = lane * 32; i < a.batch; i += 32 * 32) prefetch_l2(a.seq_lens + i);
    return;
  }
  if (lane >= GeometryQ8<HPC, NT>::kStages) return;
  const int b = blockIdx.z, hg = blockIdx.y, j = blockIdx.x;
  const long long cap = static_cast<long long>(a.max_blocks_per_seq) * a.block_size;
  long long L = __ldcg(a.seq_lens + b);
  L = L < 0 ? 0 : (L > cap ? cap : L);
  const long long chunk = static_cast<long long>(a.chunk_pages) * a.block_size;
  const long long k0 = static_cast<long long>(j) * chunk;
  const long long k1 = (j == a.num_splits - 1) ? L : min(L, k0 + chunk);
  const long long key = k0 + static_cast<long long>(lane) * kTK;
  if (key >= k1) return;
  const long long page = key / a.block_size;
  const int blk = __ldcg(a.block_tables + static_cast<long long>(b) * a.max_blocks_per_seq + page);
  if (blk < 0 || blk >= a.num_blocks) return;
  const int slot = static_cast<int>(key - page * a.block_size);
  tma_prefetch_4d(kmap, 0, slot, hg * HPC, blk);
  tma_prefetch_4d(vmap, 0, slot, hg * HPC, blk);
}

// ------------------------------------------------------------------ kernel

template <int HPC, int NT, int kFormat>
__global__ void __launch_bounds__(GeometryQ8<HPC, NT>::kThreads, 1)
paged_decode_q8_kernel(const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const DecodeArgs a,
                       const ScaleView sv) {
  using Geo = GeometryQ8<HPC, NT>;
  constexpr int STAGES = Geo::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[STAGES];
  __shared__ uint64_t empty[STAGES];
  __shared__ int abort_flag;
  __shared__ int issued;
  __shared__ Plan plan;
  __shared__ long long wsum[32];
  __shared__ uint64_t merge_full[HPC], merge_empty[HPC];
  constexpr int kProducer = Geo::kConsumers;   // warp index of the producer
  uint8_t* stages = align1024(smem_raw);

  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], HPC);               // one warp of each head reads a stage
    }
    for (int h = 0; h < HPC; ++h) {
      mbar_init(&merge_full[h], 1);
      mbar_init(&merge_empty[h], 1);
    }
    abort_flag = 0;
    issued = 0;
    fence_barrier_init();
  }
  if (warp == kProducer) prefetch_before_wait_q8<HPC, NT>(&kmap, &vmap, a);
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();

  if (a.num_splits == 0) {
    make_plan(a, &plan, wsum);
    write_empty_units(a, HPC);
  }
  if (warp == kProducer)
    produce_q8<HPC, NT>(&kmap, &vmap, a, &plan, stages, full, empty, &abort_flag, &issued);
  else
    consume_q8<HPC, NT, kFormat>(a, sv, &plan, stages, full, empty, merge_full, merge_empty,
                                 &abort_flag);
  __syncthreads();
  if (abort_flag && threadIdx.x == kProducer * 32) drain<STAGES>(full, issued);
}

template <int HPC, int NT, int kFormat>
cudaError_t launch_one(const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeArgs& a,
                       const ScaleView& sv, int grid_ctas, cudaStream_t stream) {
  using Geo = GeometryQ8<HPC, NT>;
  auto kern = paged_decode_q8_kernel<HPC, NT, kFormat>;
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = set_smem_limit_once(kern, Geo::kSmemBytes, smem_set);
  if (e != cudaSuccess) return e;
  const dim3 grid = a.num_splits == 0 ? dim3(grid_ctas, 1, 1)
                                      : dim3(a.num_splits, a.num_kv_heads / HPC, a.batch);
  return launch_pdl(kern, grid, dim3(Geo::kThreads), Geo::kSmemBytes, stream, kmap, vmap, a, sv);
}

template <int HPC>
cudaError_t launch_hpc(const DecodePlan& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                       const DecodeArgs& a, const ScaleView& sv, int format, int grid_ctas,
                       cudaStream_t stream) {
  if (format == kFormatE4m3)
    return p.rows <= 8 ? launch_one<HPC, 1, kFormatE4m3>(kmap, vmap, a, sv, grid_ctas, stream)
                       : launch_one<HPC, 2, kFormatE4m3>(kmap, vmap, a, sv, grid_ctas, stream);
  return p.rows <= 8 ? launch_one<HPC, 1, kFormatInt8>(kmap, vmap, a, sv, grid_ctas, stream)
                     : launch_one<HPC, 2, kFormatInt8>(kmap, vmap, a, sv, grid_ctas, stream);
}

}  // namespace

DecodePlan plan_decode_q8(int num_kv_heads, int rows) {
  DecodePlan p;
  int hpc = 8;
  while (hpc > 1 && (num_kv_heads % hpc) != 0) hpc >>= 1;
  p.heads_per_cta = hpc;
  p.tensor_core = true;
  p.rows = rows;
  p.tile_keys = kTK;
  p.ctas_per_sm = hpc >= 4 ? 1 : (hpc == 2 ? 2 : 3);
  return p;
}

cudaError_t launch_paged_decode_q8(const DecodePlan& p, const CUtensorMap& kmap,
                                   const CUtensorMap& vmap, const DecodeArgs& a,
                                   const ScaleView& sv, int format, int grid_ctas,
                                   cudaStream_t stream) {
  switch (p.heads_per_cta) {
    case 8: return launch_hpc<8>(p, kmap, vmap, a, sv, format, grid_ctas, stream);
    case 4: return launch_hpc<4>(p, kmap, vmap, a, sv, format, grid_ctas, stream);
    case 2: return launch_hpc<2>(p, kmap, vmap, a, sv, format, grid_ctas, stream);
    case 1: return launch_hpc<1>(p, kmap, vmap, a, sv, format, grid_ctas, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkvqk
