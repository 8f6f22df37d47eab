// The ring of key tiles of the 8-bit decode kernel: its stages, and which of a
// head's consumer warps takes which tiles.  Plain C++, for the kernel and for the
// host test of its rule.
//
// A consumer waits for a stage's tile by the parity of the stage's round.  That tells
// the current round from the one before and no more, so a warp must take part in every
// round of a stage that it reads: had it skipped one, its wait could be answered by the
// round it skipped, and it would read a tile that has not landed.  Pairs of tiles are
// therefore dealt by their place in the ring, not in their segment, and the stages are a
// whole number of turns: each stage belongs to one warp of a head for good.
#pragma once

#if defined(__CUDACC__)
#define PKVQK_HD __host__ __device__
#else
#define PKVQK_HD
#endif

namespace pkvqk {

// HPC kv heads a CTA, NT n-tiles of 8 q rows
template <int HPC, int NT>
struct RingQ8 {
  static constexpr int kSplit = HPC == 8 ? 1 : 2;     // consumer warps per head
  static constexpr int kConsumers = HPC * kSplit;
  // With 9 to 16 rows and nine warps a CTA (168 registers) the q fragments, 32
  // registers, are read from shared memory, [k-step][n-tile][lane] of each warp:
  // pairs of tiles then spill ~30 registers at their edges and still beat single
  // tiles (32 x 5 rows of 4 a kv head, 7 splits: 84.5 -> 75.5 us).
  static constexpr bool kQInSmem = NT == 2 && kConsumers == 8;
  static constexpr int kBudgetKb = HPC >= 4 ? 192 : (HPC == 2 ? 96 : 64);
  static constexpr int kStageBytes = 2 * HPC * 16 * 128;      // K and V of 16 keys
  static constexpr int kRaw = kBudgetKb * 1024 / kStageBytes;
  static constexpr int kMostStages = kQInSmem ? 10 : 12;
  static constexpr int kTurn = 2 * kSplit;            // tiles in a pair for each warp
  static constexpr int kStages = (kRaw > kMostStages ? kMostStages : kRaw) / kTurn * kTurn;
  static_assert(kStages >= 2 * kTurn || (kSplit == 1 && kStages >= 2), "ring");
};

// A segment's tiles in whole pairs (the consumers take two at once): an odd one is
// followed by one of zeros, whose keys nobody sees.
PKVQK_HD constexpr int paired(int ntiles) { return (ntiles + 1) & ~1; }

// Which of a head's `split` warps takes the pair of tiles at ring position `at` (even).
PKVQK_HD constexpr int pair_owner(int at, int split) { return at / 2 % split; }

}  // namespace pkvqk

#undef PKVQK_HD
