// Host walk of the 8-bit decode kernel's ring of key tiles, by the kernel's own stage
// counts and dealing rule (csrc/decode_q8_ring.cuh).
//
// 1. For segments of every tile count modulo 4, alone and after one another: each
//    tile's round of its stage is waited for by exactly one warp of a head, and no warp
//    skips a round of a stage that it waits on, so a wait by parity means its own round.
// 2. The same protocol run step by step, with copies that land late and in any order:
//    no warp reads a stage before its tile has landed, and nobody waits for good.
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "../../paged_kv_cache_qk_gb300/csrc/decode_q8_ring.cuh"

namespace {

int failures = 0;

void fail(const char* what, int hpc, int nt, int tile) {
  if (failures++ < 8) std::printf("%s: %d heads a CTA, %d n-tiles, tile %d\n", what, hpc, nt, tile);
}

// Ring positions of the pairs that warp `part` of a head takes, as the consumer loop
// deals them.
std::vector<int> pairs_of(const std::vector<int>& segments, int split, int part) {
  std::vector<int> at;
  int it0 = 0;
  for (int ntiles : segments) {
    for (int i = 0; i < ntiles; i += 2)
      if (split == 1 || pkvqk::pair_owner(it0 + i, split) == part) at.push_back(it0 + i);
    it0 += pkvqk::paired(ntiles);
  }
  return at;
}

template <int HPC, int NT>
void walk(const std::vector<int>& segments) {
  using R = pkvqk::RingQ8<HPC, NT>;
  int total = 0;
  for (int n : segments) total += pkvqk::paired(n);
  std::vector<int> seen(total, 0);
  for (int part = 0; part < R::kSplit; ++part) {
    std::vector<int> last(R::kStages, -1);          // round of the warp's last wait, per stage
    for (int at : pairs_of(segments, R::kSplit, part))
      for (int t = at; t < at + 2; ++t) {
        ++seen[t];
        const int s = t % R::kStages, round = t / R::kStages;
        if (round != last[s] + 1) fail("a round skipped", HPC, NT, t);
        last[s] = round;
      }
  }
  for (int t = 0; t < total; ++t)
    if (seen[t] != 1) fail("a tile not read once", HPC, NT, t);
}

// Barriers count completed phases; a wait for parity p passes unless the current phase
// has it.
bool passes(int phases, int p) { return (phases & 1) != p; }

template <int HPC, int NT>
void run(const std::vector<int>& segments, std::mt19937& rng) {
  using R = pkvqk::RingQ8<HPC, NT>;
  constexpr int S = R::kStages;
  int total = 0;
  for (int n : segments) total += pkvqk::paired(n);
  std::vector<int> full(S, 0), empty(S, 0), holds(S, -1);   // holds: the landed tile, -1 none
  std::vector<int> lands(total, -1);                        // step at which a tile lands
  std::vector<std::vector<int>> todo;
  for (int part = 0; part < R::kSplit; ++part)
    todo.push_back(pairs_of(segments, R::kSplit, part));
  std::vector<size_t> next(R::kSplit, 0);
  std::vector<int> busy(R::kSplit, 0);                      // steps left of the pair being read
  int sent = 0, idle = 0;
  const int late = static_cast<int>(rng() % 4);
  for (int step = 0;; ++step) {
    bool moved = false, done = sent == total;
    for (int t = 0; t < sent; ++t)
      if (lands[t] == step) {
        holds[t % S] = t;
        ++full[t % S];
        moved = true;
      }
    while (sent < total) {
      const int s = sent % S;
      if (sent >= S && !passes(empty[s], ((sent / S) - 1) & 1)) break;
      holds[s] = -1;
      lands[sent] = step + 1 + static_cast<int>(rng() % 3) + (rng() % 8 < 2 ? late * 12 : 0);
      ++sent;
      moved = true;
    }
    for (int part = 0; part < R::kSplit; ++part) {
      if (next[part] == todo[part].size()) continue;
      done = false;
      const int at = todo[part][next[part]];
      if (busy[part] == 0) {
        bool ready = true;
        for (int t = at; t < at + 2; ++t) ready = ready && passes(full[t % S], (t / S) & 1);
        if (!ready) continue;
        busy[part] = 3;
      }
      for (int t = at; t < at + 2; ++t)                     // read at every step of the pair
        if (holds[t % S] != t) {
          fail("read before it landed", HPC, NT, t);
          return;
        }
      moved = true;
      if (--busy[part] == 0) {
        for (int t = at; t < at + 2; ++t) ++empty[t % S];
        ++next[part];
      }
    }
    for (int t = 0; t < sent; ++t) done = done && lands[t] <= step;
    if (done) return;
    idle = moved ? 0 : idle + 1;
    if (idle > 200) return fail("nobody moves", HPC, NT, sent);
  }
}

template <int HPC, int NT>
void check() {
  for (int a = 0; a <= 41; ++a) {
    walk<HPC, NT>({a});
    for (int b = 0; b <= 17; ++b)
      for (int c : {0, 1, 2, 6, 30}) walk<HPC, NT>({a, b, c, 23});
  }
  std::mt19937 rng(HPC * 16 + NT);
  for (int i = 0; i < 3000; ++i) {
    std::vector<int> segments;
    for (int n = 1 + static_cast<int>(rng() % 4); n > 0; --n)
      segments.push_back(static_cast<int>(rng() % (n == 1 ? 60 : 14)));
    run<HPC, NT>(segments, rng);
  }
}

}  // namespace

int main() {
  check<8, 1>(); check<8, 2>();
  check<4, 1>(); check<4, 2>();
  check<2, 1>(); check<2, 2>();
  check<1, 1>(); check<1, 2>();
  std::printf("%d failures\n", failures);
  return failures != 0;
}
