// Causal multi-query attention over the paged bf16 cache under score rules
// (score_rules.cuh): the tiles, roles and softmax of prefill_kernel.cuh, whose helpers it
// uses, with three differences.
//
// Rules.  A row sees one interval of keys; a CTA walks the key tiles from its rows' first
// visible key to their last, and its splits are counted from the page of the first (a
// window's row tiles differ in their keys, not in how many).  Scores are capped and biased
// in registers before their maximum is taken (scored_half_tile), or need no maximum at all
// (bounded_half_tile); a kernel is built for each, so that a call pays for what it asks for.
//
// Persistence.  Rows that see few keys make CTAs of few key tiles, and around its tiles a CTA
// of its own spent 7.4 to 8.3 us: its places and lengths 1.2 to 1.8, Q, K and the first scores
// 1.9 to 2.5, the last product and the output 2.4, its end and the next CTA's start 1.5 to 2
// (stamps of the clock in each CTA; a key tile of both row tiles takes 1.9 to 2.4).  So one CTA
// an SM stays and takes over the pending CTAs of the grid one after another
// (clusterlaunchcontrol: the grid's order, the heaviest first, and no counter in memory
// that calls would share).  The producer reads the next place's lengths, first keys and
// block ids while the last tiles run, Q is loaded as soon as the last scores of the place
// before are computed, and one row tile's output is written while the other's tiles run:
// 4 us are left between two places' tiles.  For that the output goes from registers to
// memory, not through Q's shared memory.  A CTA a place, and this: 16 ragged prompts of
// documents 72 and 62 us, fresh 4 x 2048 under a cap 86 and 84, 19 x 512 in a window of 4096
// 353 and 352.  With every SM's places fixed beforehand in place of taken: 78, 82, 351.
// (Since then the cap costs less, and the code is smaller: 50, 69, 269.)
//
// Code.  The roles run different code at the same time, and a place's set-up and output run
// once in dozens of microseconds: what they lose to fetching instructions is no small part.
// So loops over a tile's chunks and the output's halves are not unrolled, and the first
// scores' issue, each place's reading and, without a cap or a bias, each softmax exists once.
// Documents, fresh 4 x 2048 and the window above: 61.6, 79.3 and 285 us unrolled, 53.2, 72.6
// and 280 so; warps waited 1.9 cycles an instruction for instructions before (documents),
// 0.6 since.
//
// Key tiles of 64 with two score buffers a row tile, so that the next scores are there when
// a row tile's warps are done with the last, were slower: the scores of 64 keys cost the tensor
// core as much as those of 128 (19 x 512 in a window 352 -> 391 us, fresh 4 x 2048 83 -> 96).
//
// Every barrier runs on from place to place: a role counts its uses.  Tile B's barriers
// count only the places that have a tile B.
//
// Every wait is bounded, as in prefill_kernel.cuh; after one has run out no role starts
// another place.
#pragma once

#include "prefill_kernel.cuh"
#include "score_rules.cuh"

#include <climits>

namespace pkvqk {

namespace {

// Score rules a kernel is built for: intervals of keys alone, and what scores go through.
// kRuleBounded: a cap without a bias, small enough for one reference (bounded_half_tile).
constexpr int kRuleIntervals = 1, kRuleCap = 2, kRuleBias = 4, kRuleBounded = 8;
// Capped scores without a bias lie in [-cap, cap].  Up to this cap (log2 units: 55.4 of the
// scores' own) one reference serves every row, cap / 4: weights 2^(s - cap / 4) stay between
// 2^-100 and 2^60, where fp32 and bf16 keep all their bits, and 2^20 of them with values up
// to 2^46 fit an fp32 sum; their products with values of 2^-26 and more are normal numbers.
// (In the decode kernel, which waits for HBM, the same gained nothing: 64 x 8192 300.9 ->
// 300.2 us, and its registers cost the mma tiles 5 %.)
constexpr float kBoundedCap = 80.f;

// How far (log2) scores may rise above a row's reference before it follows them.  P reaches
// 2^32 then, which bf16 holds as well as 1 and fp32 sums of 2^20 of them with values up to
// 2^74 too, and weights down to 2^-126 of the largest keep their bits.  Once a row has seen a
// tile its reference hardly ever moves: 19 x 512 tokens in a window of 4096 whose scores have a
// deviation of 3 took 287 us with 2^8, and take 244 so.
constexpr float kScoredRise = 32.f;

constexpr int kJobs = 2;                       // places whose facts are held at once

// What the roles need to know of a place in the grid.
struct Job {
  Work w;
  int key_begin;                               // keys below it are visible to no row
  int first_tile;                              // key tiles before it, over all places
  int token0;                                  // of the place's first row, in its sequence
  int prefix_end;                              // keys below it are visible whatever follows
};
constexpr int kJobTokens = 2 * kM + 1;         // tokens that a place's rows can touch

struct ScoredBars {
  uint64_t full_k[kStages], full_v[kStages], empty_k[kStages], empty_v[kStages];
  uint64_t s_full[2], p_full[2], pv_done[2], drain, xch[2][4];
  uint64_t q_full[2];                          // Q tile x in shared memory
  uint64_t q_empty[2];                         // the last scores from Q tile x computed
  uint64_t job_full[kJobs], job_empty[kJobs];
  uint64_t next_full;                          // answer about the next place landed
  alignas(16) uint4 next;
  Job job[kJobs];
  uint32_t tmem_base;
  int32_t abort;
};
constexpr int kScoredOffSlots = kDataBytes + 1024;
static_assert(sizeof(ScoredBars) <= 1024, "barrier block");
// first visible key of each token of a place, with documents
constexpr int kOffFirst = kScoredOffSlots + kSlotBytes;
constexpr int kScoredSmemBytes =
    kOffFirst + kJobs * kJobTokens * static_cast<int>(sizeof(int)) + 1024;  // + alignment slack

// ---------------------------------------------------------------- places

// Ask for a pending CTA of the grid to take over; the answer lands in bars->next.
__device__ __forceinline__ void ask_next(ScoredBars* bars) {
  tc5::fence_smem_for_async();                 // the last answer has been read
  mbar_arrive_expect_tx(&bars->next_full, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128"
      " [%0], [%1];" ::"r"(smem_addr(&bars->next)),
      "r"(smem_addr(&bars->next_full))
      : "memory");
}

// The answer: whether there was one, and its place.
__device__ __forceinline__ bool read_next(const ScoredBars* bars, int& bx, int& by) {
  uint32_t x, y, z, got;                       // the grid has one z
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%4];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %3, 1, 0, p;\n\t"
      "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, %1, %2, _}, r;\n\t}"
      : "=r"(x), "=r"(y), "=r"(z), "=r"(got)
      : "r"(smem_addr(&bars->next))
      : "memory");
  bx = static_cast<int>(x);
  by = static_cast<int>(y);
  return got != 0 && z == 0;
}

// Packed prompts of different lengths: the grid's places are those of the row tiles there
// are, every sequence's last first, in place of batch times the longest sequence's.  Place
// `x`'s sequence and row tile (one warp, all lanes); false: past the last.
constexpr int kPackedBatch = 128;              // sequences whose row tiles a warp counts at once
constexpr int kPackedMajor = 2;                // PrefillArgs::mt_major
__device__ __forceinline__ bool packed_place(const PrefillArgs& a, int x, Work& w) {
  const int lane = threadIdx.x & 31;
  const int per = a.num_kv_heads * a.num_splits;
  int rank = x / per;
  x -= rank * per;
  w.g = x / a.num_splits;
  w.j = x - w.g * a.num_splits;
  int tiles[kPackedBatch / 32];                // row tiles of sequences lane, lane + 32, ...
#pragma unroll
  for (int k = 0; k < kPackedBatch / 32; ++k) {
    const int b = k * 32 + lane;
    tiles[k] = 0;
    if (b >= a.batch) continue;
    const long long c0 = a.cu_seqlens_q[b];
    const long long c1 = min(static_cast<long long>(a.cu_seqlens_q[b + 1]),
                             static_cast<long long>(a.total_q));
    const int n = static_cast<int>(max(0ll, min(c1 - c0, static_cast<long long>(a.q_len))));
    if (n > 0) tiles[k] = (n * a.group - 1) / (2 * kM) + 1;
  }
  auto from = [&](int mt) {                    // row tiles mt and later of all sequences
    int n = 0;
#pragma unroll
    for (int k = 0; k < kPackedBatch / 32; ++k) n += max(0, tiles[k] - mt);
    return __reduce_add_sync(0xffffffffu, n);
  };
  if (rank >= from(0)) return false;
  int lo = 0, hi = a.m_tiles;                  // from(lo) > rank >= from(hi)
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (from(mid) > rank) lo = mid;
    else hi = mid;
  }
  w.mt = lo;
  rank -= from(hi);                            // among the sequences that have this row tile
  w.b = 0;
#pragma unroll
  for (int k = 0; k < kPackedBatch / 32; ++k) {
    const uint32_t have = __ballot_sync(0xffffffffu, tiles[k] > lo);
    const bool me = tiles[k] > lo && __popc(have & ((1u << lane) - 1)) == rank;
    const uint32_t at = __ballot_sync(0xffffffffu, me);
    if (at != 0) w.b = k * 32 + __ffs(at) - 1;
    rank -= __popc(have);                      // below 0 from the sequence found on
  }
  return true;
}

// The place's rows and keys (one warp, all lanes); its tokens' first keys go to first_keys.
// False: it has no rows.
__device__ __forceinline__ bool make_job(const PrefillArgs& a, int bx, int by, int* first_keys,
                                         Job& job) {
  Work& w = job.w;
  if (a.mt_major == kPackedMajor) {
    if (!packed_place(a, bx, w)) return false;
    read_place(a, w);
  } else {
    w = place_work(a, bx, by);
  }
  const int row0 = w.mt * 2 * kM;
  if (row0 >= w.rows) return false;
  const int t0 = div_group(a, row0), t1 = div_group(a, min(row0 + 2 * kM, w.rows) - 1);
  const long long cap = static_cast<long long>(a.max_blocks_per_seq) * a.block_size;
  const long long L = min(static_cast<long long>(max(w.L, 0)), cap);
  w.L = static_cast<int>(L);
  w.has_b = row0 + kM < w.rows;
  job.prefix_end = prefix_end(a.rules, w.b, w.L);
  const int p0 = w.L - w.q_len;                // position of the sequence's first new token
  // The first key that any of the rows sees.  A row's bound is the later of its window's
  // start and its first key, and the least of these bounds may lie behind both the earliest
  // window's start and the least first key.  A row that sees no key has no say.
  int first = window_start(a.rules, p0 + t0);
  if (a.rules.first_keys != nullptr) {
    first = INT_MAX;
    for (int t = t0 + static_cast<int>(threadIdx.x & 31); t <= t1; t += 32) {
      const long long row = w.q0 + t;
      const int key = row >= 0 && row < a.total_q ? a.rules.first_keys[row] : INT_MAX;
      first_keys[t - t0] = key;
      const int lo = max(window_start(a.rules, p0 + t), key);
      if (lo < max(p0 + t + 1, job.prefix_end)) first = min(first, lo);
    }
    first = __reduce_min_sync(0xffffffffu, first);
  }
  job.key_begin = min(w.L, first);
  // splits are counted from the page of the first key
  const long long base = job.key_begin / a.block_size * a.block_size;
  const long long chunk_keys = static_cast<long long>(a.chunk_pages) * a.block_size;
  const int tbs = box_shift(a.block_size);     // boxes start at multiples of their slots
  w.k0 = max(static_cast<int>(min(L, base + w.j * chunk_keys)), job.key_begin >> tbs << tbs);
  w.k1 = (w.j == a.num_splits - 1) ? w.L
                                   : static_cast<int>(min(L, base + (w.j + 1) * chunk_keys));
  job.token0 = t0;
  const int end = max(p0 + t1 + 1, job.prefix_end);
  w.key_end = max(w.k0, min(w.k1, end));
  if (w.key_end <= job.key_begin) w.key_end = w.k0;          // nothing to see
  w.ntiles = (w.key_end - w.k0 + kN - 1) / kN;
  return true;
}

// ------------------------------------------------------------- producer

__device__ void produce_places(const PrefillArgs& a, const CUtensorMap* kmap,
                               const CUtensorMap* vmap, const CUtensorMap* qmap, uint8_t* smem,
                               ScoredBars* bars, int* first_keys, int* issued_out,
                               int* q_issued_out) {
  const int lane = threadIdx.x & 31;
  const int bs = a.block_size, tbs = box_shift(bs), tb = 1 << tbs, ppt = kN >> tbs;
  const int oob = static_cast<int>(a.num_blocks);   // past the extent: TMA fills zeros
  Job cur{};
  int asked = 0;                               // answers had
  bool due = false;                            // one is on its way
  bool ok = true;
  // page id of box `lane` of a place's key tile i, when the box holds a visible key; loaded
  // ahead of its use
  auto box_visible = [&](const Work& w, int i) {
    return lane < ppt && w.k0 + i * kN + lane * tb < w.key_end;
  };
  auto page_id = [&](const Work& w, int i) {
    const int32_t* bt = a.block_tables + static_cast<long long>(w.b) * a.max_blocks_per_seq;
    return i < w.ntiles && box_visible(w, i) ? __ldg(bt + (w.k0 + i * kN + lane * tb) / bs) : oob;
  };
  int jobs = 0, it = 0, issued = 0;            // places handed out, key tiles asked for
  // the next place that has rows, the CTA's own first; false: none is left, or a wait gave
  // up.  Its first keys' slot is that of the place before the current one, whose rows have left
  // it once job_empty says so.
  bool own = true;
  auto next_place = [&](Job& job) {
    int bx = blockIdx.x, by = blockIdx.y;
    while (true) {
      if (!own) {
        if (lane == 0) ask_next(bars);
        __syncwarp();
        due = true;
        ok = mbar_wait(&bars->next_full, asked & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        due = false;
        ++asked;
        const bool got = read_next(bars, bx, by);
        __syncwarp();
        if (!got) return false;
      }
      own = false;
      if (jobs >= kJobs) {
        ok = mbar_wait(&bars->job_empty[jobs % kJobs], (jobs / kJobs - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
      }
      if (make_job(a, bx, by, first_keys + (jobs % kJobs) * kJobTokens, job)) return true;
    }
  };
  int q_issued[2] = {0, 0};
  auto wait_here = [&](uint64_t* bar, uint32_t parity) {
    bool w = true;
    if (lane == 0) w = mbar_wait(bar, parity);
    return __shfl_sync(0xffffffffu, static_cast<int>(w), 0) != 0;
  };
  auto load_q = [&](int x) {
    if (q_issued[x] > 0 && !wait_here(&bars->q_empty[x], (q_issued[x] - 1) & 1)) return false;
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars->q_full[x], kTile);
      const int tok = static_cast<int>(cur.w.q0 + div_group(a, cur.w.mt * 2 * kM + x * kM));
      for (int dh = 0; dh < 2; ++dh)
        tma_load_rows(smem + kOffQ + x * kTile + dh * kHalf, qmap, &bars->q_full[x], dh * 64,
                      cur.w.g * a.group, tok);
    }
    ++q_issued[x];
    return true;
  };
#pragma unroll 1
  while (true) {
    // The next place is asked for only here, while the row tiles still work on what the ring
    // holds: places are few, and one that is taken early waits while another SM could have
    // it (16 ragged prompts took 68 us asked for at the third key tile, 62 here).
    if (!next_place(cur)) break;
    const Work& w = cur.w;
    const int id_first = page_id(w, 0);
    const int slot = jobs % kJobs;
    cur.first_tile = it;
    __syncwarp();                              // every lane's first keys are written
    if (lane == 0) {
      bars->job[slot] = cur;
      mbar_arrive(&bars->job_full[slot]);
    }
    __syncwarp();
    ++jobs;
    if (a.q_tma && w.ntiles > 0 && !load_q(0)) {
      ok = false;
      break;
    }
    int id_next = id_first;
    for (int i = 0; i < w.ntiles && ok; ++i, ++it) {
      const int s = it & 1;
      const uint32_t rel = ((it >> 1) - 1) & 1;          // release of the tile before last
      uint8_t* kt = smem + kOffK + s * kTile;
      uint8_t* vt = smem + kOffV + s * kTile;
      int blk = id_next;
      if (box_visible(w, i) && (blk < 0 || static_cast<long long>(blk) >= a.num_blocks)) {
        report(a.status_flags, kFlagBadBlock);
        blk = oob;
      }
      id_next = page_id(w, i + 1);
      int slot0 = 0;
      if (lane < ppt) {
        const int key = w.k0 + i * kN + lane * tb;         // first key of box `lane`
        slot0 = key - (key / bs) * bs;
      }
      if (it >= 2 && !wait_here(&bars->empty_k[s], rel)) {
        ok = false;
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(&bars->full_k[s], kTile);
      __syncwarp();
      if (lane < ppt) {
        tma_load_5d_keep(kt + lane * tb * 128, kmap, &bars->full_k[s], 0, slot0, 0, w.g, blk);
        tma_load_5d_keep(kt + kHalf + lane * tb * 128, kmap, &bars->full_k[s], 0, slot0, 1, w.g,
                         blk);
      }
      if (i == 0 && a.q_tma && w.has_b && !load_q(1)) {
        issued = -(it + 1);                    // K of this tile is in flight, V is not
        ok = false;
        break;
      }
      if (it >= 2 && !wait_here(&bars->empty_v[s], rel)) {
        issued = -(it + 1);
        ok = false;
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(&bars->full_v[s], kTile);
      __syncwarp();
      if (lane < ppt)
        tma_load_5d_keep(vt + lane * tb * 256, vmap, &bars->full_v[s], 0, slot0, 0, w.g, blk);
      issued = it + 1;
    }
    if (!ok) break;
  }
  // no place any more: a job without a row tile ends the other roles
  if (ok) {
    const int slot = jobs % kJobs;
    if (jobs >= kJobs) ok = wait_here(&bars->job_empty[slot], (jobs / kJobs - 1) & 1);
    if (ok && lane == 0) {
      bars->job[slot].w.ntiles = -1;
      mbar_arrive(&bars->job_full[slot]);
    }
  }
  if (!ok && lane == 0) {
    bars->abort = 1;
    report(a.status_flags, kFlagTimeout);
    if (due) mbar_wait(&bars->next_full, asked & 1);       // it lands before the CTA leaves
  }
  __syncwarp();
  *issued_out = issued;
  q_issued_out[0] = q_issued[0];
  q_issued_out[1] = q_issued[1];
}

// ------------------------------------------------------------ MMA issue

// One lane of a converged warp.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(p));
  return p != 0;
}

// The whole warp walks the loop and one elected lane issues: operands of the matrix
// instructions are then uniform values, where a loop of one lane alone had each moved over
// before its instruction (19 x 512 in a window of 4096 279 -> 269 us, without the cap 268 ->
// 248; fresh 4 x 2048 70.5 -> 68.9).
__device__ void issue_places(const PrefillArgs& a, uint8_t* smem, ScoredBars* bars,
                             uint32_t tmem) {
  constexpr uint32_t idesc_s = tc5::idesc_bf16_f32(kM, kN, false);
  constexpr uint32_t idesc_pv = tc5::idesc_bf16_f32(kM, kHeadDim, true);
  const uint64_t d0 = desc_k_major(smem_addr(smem + kOffQ), 0);
  const uint32_t hi = static_cast<uint32_t>(d0 >> 32);
  const uint32_t q_lo = static_cast<uint32_t>(d0);
  const uint32_t k_lo = static_cast<uint32_t>(desc_k_major(smem_addr(smem + kOffK), 0));
  const int tbs = box_shift(a.block_size);
  const uint32_t v_lo = static_cast<uint32_t>(
      tc5::smem_desc_sw128(smem_addr(smem + kOffV), 128u << tbs, 1024));
  uint32_t v_step[kN / 16];
#pragma unroll
  for (int ks = 0; ks < kN / 16; ++ks) v_step[ks] = v_step_offset(ks, tbs) >> 4;
  uint32_t p_uses = 0, q_uses = 0;             // bit x: parity of tile x's next use
  const bool lead = elected();
  bool ok = true;
  for (int jobs = 0; ok; ++jobs) {
    const int slot = jobs % kJobs;
    ok = warp_wait(&bars->job_full[slot], (jobs / kJobs) & 1);
    if (!ok) break;
    const int n = bars->job[slot].w.ntiles, it0 = bars->job[slot].first_tile;
    const bool has_b = bars->job[slot].w.has_b;
    __syncwarp();
    if (lead) mbar_arrive(&bars->job_empty[slot]);
    if (n < 0) break;
    if (n == 0) continue;
    const int last = has_b ? 1 : 0;            // the row tile that reads a stage last
    // S_x = Q_x K^T of key tile i
    auto mma_s = [&](int x, int i) {
      const int s = (it0 + i) & 1;
      const uint32_t qa = q_lo + (x * kTile >> 4), kb = k_lo + (s * kTile >> 4);
      const uint32_t dst = tmem + kColS + x * kN;
#pragma unroll
      for (int kk = 0; kk < kHeadDim / 16; ++kk) {
        const uint32_t step = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
        tc5::mma_f16_lh(dst, qa + step, hi, kb + step, hi, idesc_s, kk > 0 ? 1u : 0u);
      }
      tc5::commit(&bars->s_full[x]);
      if (x == last) tc5::commit(&bars->empty_k[s]);
      if (i == n - 1) tc5::commit(&bars->q_empty[x]);
    };
    // O_x += P_x V of key tile i
    auto mma_pv = [&](int x, int i) {
      const int s = (it0 + i) & 1;
      const uint32_t vb = v_lo + (s * kTile >> 4);
      const uint32_t dst = tmem + kColO + x * kN, p0 = tmem + kColS + x * kN;
#pragma unroll
      for (int ks = 0; ks < kN / 16; ++ks)
        tc5::mma_f16_ts_lh(dst, p0 + (ks >> 2) * (kN / 2) + (ks & 3) * 8, vb + v_step[ks], hi,
                           idesc_pv, (i > 0 || ks > 0) ? 1u : 0u);
      if (i == n - 1) tc5::commit(&bars->pv_done[x]);
      if (x == last) tc5::commit(&bars->empty_v[s]);
    };
    auto wait_use = [&](uint64_t* bar, uint32_t& uses, int x) {
      const uint32_t parity = uses >> x & 1;
      uses ^= 1u << x;
      return warp_wait(bar + x, parity);
    };
    // turn i of row tile x: its product with key tile i, then the scores of key tile i + 1;
    // turn -1: the first scores
#pragma unroll 1
    for (int i = -1; i < n && ok; ++i) {
      const int it = it0 + i;
      if (i >= 0) ok = warp_wait(&bars->full_v[it & 1], (it >> 1) & 1);
      if (ok && i + 1 < n) ok = warp_wait(&bars->full_k[(it + 1) & 1], ((it + 1) >> 1) & 1);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (x > last || !ok) break;
        ok = i < 0 ? wait_use(bars->q_full, q_uses, x) : wait_use(bars->p_full, p_uses, x);
        if (!ok) break;
        tc5::fence_after_sync();
        if (lead) {
          if (i >= 0) mma_pv(x, i);
          if (i + 1 < n) mma_s(x, i + 1);
        }
        __syncwarp();
      }
    }
  }
  if (!ok && lead) {
    bars->abort = 1;
    report(a.status_flags, kFlagTimeout);
    tc5::commit(&bars->drain);                 // everything issued so far ...
    mbar_wait(&bars->drain, 0);                // ... has finished
  }
}

// --------------------------------------------------------------- softmax

// add + cap * tanh(k v) of 32 raw scores, k = scale / softcap, in packed pairs.  The polynomial
// has the cap in its coefficients and, for kSmallestK <= k <= kLargestK, k too: v R(v^2) is
// then five instructions a pair; another k is multiplied first.  (Caps are 2^-20 .. 2^20 of
// the scores' own: the last coefficient, 0.044 cap k^7, does not overflow, and at the smallest
// of both is 2^-136, a subnormal of 13 bits.  Its term is at most 2^-10 of the value, which
// then loses 2^-24.)
constexpr float kSmallestK = 0x1p-16f, kLargestK = 0x1p14f;

__device__ __forceinline__ void cap_chunk(float (&v)[32], float k, float cap, float add) {
  // the largest |v| decides what is computed; a NaN that is masked later does not count
  float b4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 32; e += 2)
    b4[(e >> 1) & 3] = max3(b4[(e >> 1) & 3], fabsf(v[e]), fabsf(v[e + 1]));
  const float big = max3(b4[0], b4[1], fmaxf(b4[2], b4[3])) * k;
  const bool folded = k >= kSmallestK && k <= kLargestK;
  const float inner = folded ? k : 1.f;
  uint64_t c[4];
  float f = cap * inner;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = pack2(f * tanh_q(i), f * tanh_q(i));
    f *= inner * inner;
  }
  const uint64_t add2_ = pack2(add, add);
  auto near = [&](uint64_t x) {
    const uint64_t u = mul2(x, x);
    return fma2(x, fma2(fma2(fma2(c[3], u, c[2]), u, c[1]), u, c[0]), add2_);
  };
  if (folded && !__any_sync(0xffffffffu, big * big > kTanhSquare)) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) unpack2(near(pack2(v[e], v[e + 1])), v[e], v[e + 1]);
  } else {
    const float outer = folded ? 1.f : k;      // exact where k is folded: the same bits
    const uint64_t outer2 = pack2(outer, outer);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float x0 = v[e] * k, x1 = v[e + 1] * k;
      unpack2(near(mul2(pack2(v[e], v[e + 1]), outer2)), v[e], v[e + 1]);
      if (!(x0 * x0 <= kTanhSquare)) v[e] = fmaf(cap, tanh_far(x0), add);
      if (!(x1 * x1 <= kTanhSquare)) v[e + 1] = fmaf(cap, tanh_far(x1), add);
    }
  }
}

// Scores of the keys outside [lo, hi) to -inf.  Most masked tiles are cut at one end: the
// other's comparisons are skipped where none of the warp's rows needs them.
__device__ __forceinline__ void hide_keys(float (&v)[32], int lo, int hi) {
  if (__any_sync(0xffffffffu, hi < 32)) {
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = e < hi ? v[e] : -INFINITY;
  }
  if (__any_sync(0xffffffffu, lo > 0)) {
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = e >= lo ? v[e] : -INFINITY;
  }
}

// P of a half tile of which none of the warp's rows sees a key.
__device__ __forceinline__ void zero_half_tile(uint32_t pcol) {
  uint32_t z[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) z[j] = 0u;
  tc5::tmem_st16(pcol, z);
  tc5::tmem_st16(pcol + 16, z);
}

// half_tile under a cap without a bias, against the one reference that serves every row
// (kBoundedCap): no maximum is taken, O is never rescaled, and the row's halves need not meet
// before the end (fresh 4 x 2048 139 -> 107 us, 19 x 512 in a window of 4096 431 -> 360).
template <bool kMasked>
__device__ __forceinline__ float bounded_half_tile(uint32_t scol, uint32_t pcol, int kbase,
                                                   int nlo, int nvis, float k, float cap,
                                                   float ref) {
  uint64_t acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = pack2(0.f, 0.f);
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    float v[32];
    tc5::tmem_ld32(scol + c * 32, v);
    tc5::wait_ld();
    cap_chunk(v, k, cap, -ref);
    if (kMasked) hide_keys(v, nlo - kbase - c * 32, nvis - kbase - c * 32);
    uint32_t pk[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const float p0 = ex2_approx(v[2 * q]), p1 = ex2_approx(v[2 * q + 1]);
      acc[q & 3] = add2(acc[q & 3], pack2(p0, p1));
      pk[q] = pack_bf16x2(p0, p1);
    }
    tc5::tmem_st16(pcol + c * 16, pk);
  }
  float t0, t1;
  unpack2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), t0, t1);
  return t0 + t1;
}

// half_tile over a bf16 cache under score rules: scores go through the cap and the
// bias (log2 units) before their maximum is taken.  Keys kbase + e with nlo <= kbase + e <
// nvis count (kMasked); `at` is the tile's first key less the row's position.  An
// unmasked tile has no key past any of the warp's positions, where the bias
// -slope (p - n) = slope e + slope (base - p) is one packed FMA a pair of keys, its constant
// part joined with the reference; a masked one may (a prefix), and takes |p - n|.
template <int kRules, bool kMasked, typename Publish>
__device__ __forceinline__ float scored_half_tile(uint32_t scol, uint32_t pcol, int kbase, int nlo,
                                                  int nvis, float sl2, const ScoreRules& rules,
                                                  float slope, int at, float& m_ref,
                                                  Publish&& publish) {
  float psum = 0.f;
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    float v[32];
    tc5::tmem_ld32(scol + c * 32, v);
    tc5::wait_ld();
    const int k0 = kbase + c * 32;
    if (kRules & kRuleCap) {
      cap_chunk(v, sl2 * rules.inv_cap, rules.cap, 0.f);
    } else if (kRules & kRuleBias) {
      const uint64_t scale2 = pack2(sl2, sl2);
#pragma unroll
      for (int e = 0; e < 32; e += 2)
        unpack2(mul2(pack2(v[e], v[e + 1]), scale2), v[e], v[e + 1]);
    }
    float shift = 0.f;                         // what the chunk's scores still lack
    if (kRules & kRuleBias) {
      const float d0 = static_cast<float>(at + k0);        // exact: |d| < 2^24 or far away
      if (kMasked) {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = fmaf(-slope, fabsf(d0 + static_cast<float>(e)), v[e]);
      } else {
        const uint64_t slope2 = pack2(slope, slope);
#pragma unroll
        for (int e = 0; e < 32; e += 2)
          unpack2(fma2(slope2, pack2(static_cast<float>(e), static_cast<float>(e + 1)),
                       pack2(v[e], v[e + 1])),
                  v[e], v[e + 1]);
        shift = slope * d0;
      }
    }
    if (kMasked) hide_keys(v, nlo - k0, nvis - k0);
    float m4[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) m4[j] = -INFINITY;
#pragma unroll
    for (int e = 0; e < 32; e += 2) m4[(e >> 1) & 3] = max3(m4[(e >> 1) & 3], v[e], v[e + 1]);
    float mt = max3(m4[0], m4[1], fmaxf(m4[2], m4[3]));
    if (kRules == kRuleIntervals) mt *= sl2;
    else mt += shift;
    const bool grow = mt > m_ref + kScoredRise;
    if (__any_sync(0xffffffffu, grow)) {
      const float m_new = grow ? ceilf(mt) : m_ref;
      const float f = grow ? pow2_int(m_ref - m_new) : 1.f;
      if (c == 1) scale_p<0, 16>(pcol, f);
      psum *= f;
      m_ref = m_new;
    }
    if (c == 1) publish(m_ref);
    const float u = shift - ((m_ref == -INFINITY) ? 0.f : m_ref);
    const uint64_t scale2 = pack2(sl2, sl2), shift2 = pack2(u, u);
    uint64_t acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = pack2(0.f, 0.f);
    uint32_t pk[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const uint64_t z = pack2(v[2 * q], v[2 * q + 1]);
      float x0, x1;
      unpack2(kRules == kRuleIntervals ? fma2(z, scale2, shift2) : add2(z, shift2), x0, x1);
      const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
      acc[q & 3] = add2(acc[q & 3], pack2(p0, p1));
      pk[q] = pack_bf16x2(p0, p1);
    }
    tc5::tmem_st16(pcol + c * 16, pk);
    float t0, t1;
    unpack2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), t0, t1);
    psum += t0 + t1;
  }
  return psum;
}

// ----------------------------------------------------------------- rows

// 32 bytes to a 32-byte aligned address.
__device__ __forceinline__ void store32(void* to, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void store_words(void* to, const uint32_t (&v)[8]) {
  if ((reinterpret_cast<uintptr_t>(to) & 31u) == 0) {
    store32(to, v);
  } else {
    reinterpret_cast<uint4*>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// 64 bytes of each lane's row (none where `to` is null).  A lane's own bytes in its own row
// leave the SM a sector at a time; two lanes exchange 32 bytes and write their rows one after
// the other, 64 bytes together (16 ragged prompts of documents 53.3 -> 51.3 us, fresh 4 x 2048
// 72.9 -> 71.2; four lanes and 128 bytes, with three times the exchanges: 52.0, 72.0).
__device__ __forceinline__ void store_rows64(uint32_t (&v)[16], uint8_t* to) {
  const bool odd = (threadIdx.x & 1) != 0;
  uint32_t w[2][8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? v[k] : v[8 + k], 1);
    w[0][k] = odd ? got : v[k];                // of the even lane's row
    w[1][k] = odd ? v[8 + k] : got;            // of the odd lane's
  }
  const unsigned long long mine = reinterpret_cast<unsigned long long>(to);
  const unsigned long long other = __shfl_xor_sync(0xffffffffu, mine, 1);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint8_t* row = reinterpret_cast<uint8_t*>((p != 0) == odd ? mine : other);
    if (row != nullptr) store_words(row + (odd ? 32 : 0), w[p]);
  }
}

// This thread's half of an output row of tile x: O / l for dims 64h .. 64h + 63 (bf16, or
// the fp32 partial of the split), and the log-sum-exp (half 0).  Every lane of the warp
// takes part in the loads from tensor memory.
__device__ __forceinline__ void write_scored_rows(const PrefillArgs& a, const Work& w,
                                                  uint32_t o_cols, int rg, int half, float m_ref,
                                                  float l) {
  const int t0 = div_group(a, rg);
  const bool valid = rg < w.rows && w.q0 + t0 >= 0 && w.q0 + t0 < a.total_q;
  const int t = valid ? t0 : 0;
  const int h = w.g * a.group + (valid ? rg - t * a.group : 0);
  const long long row = (w.q0 + t) * a.num_q_heads + h;
  // a sum of 0: no visible key; a NaN sum stays NaN
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const float lse = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * kLn2;
  const bool have_o = w.ntiles > 0;            // uniform over the CTA
  const int d0 = half * (kHeadDim / 2);
  const bool split = a.num_splits > 1;
  const long long prow = row * a.num_splits + w.j;
#pragma unroll 1
  for (int c = 0; c < kHeadDim / 64; ++c) {
    float o[32];
    if (have_o) {
      tc5::tmem_ld32(o_cols + c * 32, o);
      tc5::wait_ld();
    }
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = have_o ? o[e] * inv : 0.f;
    if (split) {
      uint8_t* to = reinterpret_cast<uint8_t*>(a.ws_o + prow * kHeadDim + d0 + c * 32);
#pragma unroll
      for (int e = 0; e < 32; e += 16) {
        uint32_t v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(o[e + k]);
        store_rows64(v, valid ? to + e * 4 : nullptr);
      }
    } else {
      uint32_t v[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = pack_bf16x2(o[2 * k], o[2 * k + 1]);
      store_rows64(v, valid ? reinterpret_cast<uint8_t*>(a.out + row * kHeadDim + d0 + c * 32)
                            : nullptr);
    }
  }
  if (valid && half == 0) {
    if (split) a.ws_lse[prow] = lse;
    else if (a.lse_out != nullptr) a.lse_out[row] = lse;
  }
}

// Q rows of tile x by its warps, where q's layout allows no box: thread i of the 256 takes
// 64 dims (half i / 128) of row i % 128.
__device__ __forceinline__ void load_q_tile(const PrefillArgs& a, const Work& w, uint8_t* smem,
                                            int x) {
  const int i = threadIdx.x & 255, r = i & (kM - 1), dh = i >> 7;
  const int rg = w.mt * 2 * kM + x * kM + r;
  const int t0 = div_group(a, rg);
  const bool valid = rg < w.rows && w.q0 + t0 >= 0 && w.q0 + t0 < a.total_q;
  const int t = valid ? t0 : 0;
  const uint4* src = reinterpret_cast<const uint4*>(
      a.q + (valid ? w.q0 + t : 0) * a.q_stride_t +
      static_cast<long long>(w.g * a.group + (valid ? rg - t * a.group : 0)) * a.q_stride_h);
  uint8_t* to = smem + kOffQ + x * kTile + dh * kHalf;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(to + swz128(r, c)) =
        valid ? __ldg(src + dh * 8 + c) : make_uint4(0u, 0u, 0u, 0u);
  tc5::fence_smem_for_async();
}

// What a thread of the softmax keeps from place to place.
struct Uses {
  uint32_t s = 0, pv = 0, swaps = 0;           // of s_full, pv_done and the pair's barrier
};

template <int kRules>
__device__ __forceinline__ bool softmax_place(const PrefillArgs& a, const Job& job, uint8_t* smem,
                                              ScoredBars* bars, const int* first_keys,
                                              float* slots, uint32_t lanes, int x, int half,
                                              Uses& uses) {
  const Work& w = job.w;
  const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const int r = wq * 32 + lane;                // row of tile x = tensor-memory lane
  const int rg = w.mt * 2 * kM + x * kM + r;
  const uint32_t s_cols = lanes + kColS + x * kN + half * (kN / 2);
  const uint32_t o_cols = lanes + kColO + x * kN + half * (kHeadDim / 2);
  uint64_t* xbar = &bars->xch[x][wq];
  const int n = w.ntiles, k0 = w.k0;
  if (!a.q_tma && n > 0) {
    load_q_tile(a, w, smem, x);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->q_full[x]);
  }
  // keys [lo, lim) are visible to this row, which stands at `pos`
  int lo = 0, lim = k0, pos = 0;
  float slope = 0.f;
  {
    const int t = div_group(a, rg);
    if (rg < w.rows && w.q0 + t >= 0 && w.q0 + t < a.total_q) {
      pos = w.L - w.q_len + t;
      lo = window_start(a.rules, pos);
      if (a.rules.first_keys != nullptr) lo = max(lo, first_keys[t - job.token0]);
      lim = max(k0, min(w.k1, max(pos + 1, job.prefix_end)));
      if ((kRules & kRuleBias) && a.rules.slopes != nullptr)
        slope = a.rules.slopes[w.g * a.group + rg - t * a.group] * 1.4426950408889634f;
    }
  }
  // of the warp's rows: whole tiles lie in [lo_max, lim_min), none of their keys past a
  // position where distances count; nothing is visible outside [lo_least, lim_most)
  int lim_min = __reduce_min_sync(0xffffffffu, lim);
  const int lo_max = __reduce_max_sync(0xffffffffu, lo);
  const int lo_least = __reduce_min_sync(0xffffffffu, lim > k0 ? lo : INT_MAX);
  const int lim_most = __reduce_max_sync(0xffffffffu, lim);
  if (kRules & kRuleBias)
    lim_min = min(lim_min, __reduce_min_sync(0xffffffffu, lim > k0 ? pos + 1 : k0));
  const int tail_tile = (x == 0 && k0 + n * kN > w.key_end) ? n - 1 : -1;
  const int head_tile = (x == 0 && k0 < job.key_begin) ? 0 : -1;

  const float sl2 = a.scale_log2;
  // reference max (log2 units), integer once set
  float m_ref = kRules & kRuleBounded ? 0.25f * a.rules.cap : -INFINITY;
  float l = 0.f;                               // this half's sum of P
  bool ok = true;
  for (int i = 0; i < n && ok; ++i) {
    // S_x(i) landed, and with it PV_x(i - 1): O_x is complete up to tile i - 1
    if (!warp_wait(&bars->s_full[x], uses.s++ & 1)) return false;
    tc5::fence_after_sync();
    const int kb = k0 + i * kN;
    const int nvis = min(kN, max(0, lim - kb));
    const bool whole = lim_min >= kb + kN && lo_max <= kb;
    const int h0 = kb + half * (kN / 2);
    const bool hidden = lim_most <= h0 || lo_least >= h0 + kN / 2;
    const float m_start = m_ref;
    auto publish = [&](float m) { swap_publish(m, slots, xbar, uses.swaps, half, r); };
    float psum = 0.f;
    if (hidden) {
      zero_half_tile(s_cols);
      if (!(kRules & kRuleBounded)) publish(m_ref);
    } else if constexpr ((kRules & kRuleBounded) != 0) {
      const float k = sl2 * a.rules.inv_cap;
      psum = whole ? bounded_half_tile<false>(s_cols, s_cols, half * (kN / 2), 0, nvis, k,
                                              a.rules.cap, m_ref)
                   : bounded_half_tile<true>(s_cols, s_cols, half * (kN / 2), lo - kb, nvis, k,
                                             a.rules.cap, m_ref);
    } else {
      psum = kRules != kRuleIntervals && whole ? scored_half_tile<kRules, false>(s_cols, s_cols, half * (kN / 2), 0, nvis, sl2,
                                                     a.rules, slope, kb - pos, m_ref, publish)
                   : scored_half_tile<kRules, true>(s_cols, s_cols, half * (kN / 2), lo - kb, nvis,
                                                    sl2, a.rules, slope, kb - pos, m_ref, publish);
    }
    if constexpr ((kRules & kRuleBounded) != 0) {
      l += psum;
    } else {
      // one reference per row: the higher of the two halves'
      const float m_other = swap_read(slots, xbar, uses.swaps, half, r, ok);
      if (!ok) return false;
      if (__all_sync(0xffffffffu, m_ref == m_start && m_other == m_start)) {
        l += psum;                             // neither half moved (the usual tile)
      } else {
        const float m_row = fmaxf(m_ref, m_other);
        if (__any_sync(0xffffffffu, m_ref < m_row)) {
          const float f = m_ref < m_row ? pow2_int(m_ref - m_row) : 1.f;
          scale_p<0, 32>(s_cols, f);
          psum *= f;
        }
        m_ref = m_row;
        const bool rose = m_row > m_start;     // -inf -> finite counts
        const float alpha = rose ? pow2_int(m_start - m_row) : 1.f;
        if (i > 0 && __any_sync(0xffffffffu, rose)) {
#pragma unroll 1
          for (int c = 0; c < kHeadDim / 64; ++c) {
            float o[32];
            tc5::tmem_ld32(o_cols + c * 32, o);
            tc5::wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= alpha;
            tc5::tmem_st32(o_cols + c * 32, o);
          }
        }
        l = l * alpha + psum;
      }
    }
    // Slots past the last visible key, and before the first, may hold anything; P is 0
    // there, but 0 x NaN is NaN, so their V rows are zeroed (by tile A, each half its
    // dims, before either PV reads them).
    if (i == tail_tile || i == head_tile) {
      const int it = job.first_tile + i, s = it & 1;
      if (!warp_wait(&bars->full_v[s], (it >> 1) & 1)) return false;
      if (kb + r >= w.key_end || kb + r < job.key_begin) {
        uint8_t* vrow = smem + kOffV + s * kTile + v_row_offset(r, half, box_shift(a.block_size));
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(vrow + c * 16) = z;
      }
      tc5::fence_smem_for_async();
    }
    tc5::wait_st();
    tc5::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->p_full[x]);
  }
  // the row's sum of P: both halves'
  l += pair_swap(l, slots, xbar, uses.swaps, half, r, ok);
  // O_x is complete once the last PV has finished
  if (ok && n > 0) ok = warp_wait(&bars->pv_done[x], uses.pv++ & 1);
  if (!ok) return false;
  tc5::fence_after_sync();
  write_scored_rows(a, w, o_cols, rg, half, m_ref, l);
  tc5::fence_before_sync();                    // O_x read before the next place's P_x is
  return true;
}

template <int kRules>
__device__ void softmax_places(const PrefillArgs& a, uint8_t* smem, ScoredBars* bars,
                               float* xslots, uint32_t tmem, int x, int half) {
  const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(wq * 32) << 16);
  float* slots = xslots + x * 4 * kM;          // [parity][half][row] of tile x
  Uses uses;
  bool ok = true;
  for (int jobs = 0;; ++jobs) {
    const int slot = jobs % kJobs;
    ok = warp_wait(&bars->job_full[slot], (jobs / kJobs) & 1);
    if (!ok) break;
    const Job& job = bars->job[slot];
    const bool over = job.w.ntiles < 0;
    if (!over && (x == 0 || job.w.has_b))
      ok = softmax_place<kRules>(a, job, smem, bars,
                                 reinterpret_cast<const int*>(smem + kOffFirst) + slot * kJobTokens,
                                 slots, lanes, x, half, uses);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->job_empty[slot]);
    if (over || !ok) break;
  }
  if (!ok) {
    bars->abort = 1;
    report(a.status_flags, kFlagTimeout);
  }
}

// ------------------------------------------------------------------ kernel

template <int kRules>
__global__ void __maxnreg__(96)
scored_prefill_kernel(const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ PrefillArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  ScoredBars* bars = reinterpret_cast<ScoredBars*>(smem + kDataBytes);
  __shared__ int issued, q_issued[2];
  const int warp = threadIdx.x >> 5;

  if (threadIdx.x == kProducerWarp * 32) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
    prefetch_tensormap(&qmap);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full_k[s], 1);
      mbar_init(&bars->full_v[s], 1);
      mbar_init(&bars->empty_k[s], 1);
      mbar_init(&bars->empty_v[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->s_full[x], 1);
      mbar_init(&bars->p_full[x], kSoftmaxWarps / 2);
      for (int q = 0; q < 4; ++q) mbar_init(&bars->xch[x][q], 2);
      mbar_init(&bars->pv_done[x], 1);
      mbar_init(&bars->q_full[x], a.q_tma ? 1 : kSoftmaxWarps / 2);
      mbar_init(&bars->q_empty[x], 1);
    }
    for (int s = 0; s < kJobs; ++s) {
      mbar_init(&bars->job_full[s], 1);
      mbar_init(&bars->job_empty[s], kSoftmaxWarps + 1);
    }
    mbar_init(&bars->next_full, 1);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    issued = q_issued[0] = q_issued[1] = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tc5::tmem_alloc(&bars->tmem_base, kTmemCols);
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  // launched as a programmatic dependent: q, the appended K/V, the tables and the lengths
  // may come from the previous kernel in the stream
  pdl_wait();
  pdl_launch_dependents();

  if (warp < kSoftmaxWarps) {
    // warp = 8 x + 4 half + lane quadrant
    softmax_places<kRules>(a, smem, bars, reinterpret_cast<float*>(smem + kScoredOffSlots), tmem,
                           warp >> 3, (warp >> 2) & 1);
  } else if (warp == kProducerWarp) {
    int n = 0, q[2];
    produce_places(a, &kmap, &vmap, &qmap, smem, bars, reinterpret_cast<int*>(smem + kOffFirst),
                   &n, q);
    if ((threadIdx.x & 31) == 0) {
      issued = n;
      q_issued[0] = q[0];
      q_issued[1] = q[1];
    }
    __syncwarp();
  } else {
    issue_places(a, smem, bars, tmem);
    __syncwarp();
  }
  tc5::fence_before_sync();
  __syncthreads();
  // after a timeout: wait (bounded) for the copies in flight
  if (bars->abort && threadIdx.x == kProducerWarp * 32) {
    const bool v_missing = issued < 0;
    const int n = v_missing ? -issued : issued;
    for (int i = n - 2 < 0 ? 0 : n - 2; i < n; ++i) {
      mbar_wait(&bars->full_k[i & 1], (i >> 1) & 1);
      if (!(v_missing && i == n - 1)) mbar_wait(&bars->full_v[i & 1], (i >> 1) & 1);
    }
    for (int x = 0; x < 2; ++x)
      if (a.q_tma && q_issued[x] > 0) mbar_wait(&bars->q_full[x], (q_issued[x] - 1) & 1);
  }
  if (warp == kMmaWarp) {
    tc5::fence_after_sync();
    tc5::tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

}  // namespace pkvqk
