// Host walk of the multi-query attention kernel's launch order (csrc/prefill_order.cuh):
// every CTA's place lies inside the call and every place is taken once, in grids of all
// sizes that the entry points allow: 65535 sequences, 2^31 - 1 CTAs a sequence.
// Built with wrapping integers, as the GPU's are.
#include <cstdio>
#include <random>
#include <vector>

#include "../../paged_kv_cache_qk_gb300/csrc/prefill_order.cuh"

namespace {

int failures = 0;

pkvqk::PrefillPlace place(bool wanted, long long gx, int batch, int m_tiles, int hkv, int splits,
                          int x, int y) {
  const bool major = pkvqk::row_tile_major(wanted, gx, batch);
  const auto p = pkvqk::place_cta(major, x, y, static_cast<int>(gx), batch, m_tiles, hkv, splits);
  if (p.b < 0 || p.b >= batch || p.g < 0 || p.g >= hkv || p.j < 0 || p.j >= splits || p.mt < 0 ||
      p.mt >= m_tiles) {
    if (failures++ < 8)
      std::printf("batch %d, %d row tiles, %d heads, %d splits: CTA (%d, %d) has %d %d %d %d\n",
                  batch, m_tiles, hkv, splits, x, y, p.b, p.g, p.j, p.mt);
  }
  return p;
}

void whole_grid(bool wanted, int batch, int m_tiles, int hkv, int splits) {
  const int gx = m_tiles * hkv * splits;
  std::vector<int> seen(static_cast<size_t>(gx) * batch, 0);
  for (int y = 0; y < batch; ++y)
    for (int x = 0; x < gx; ++x) {
      const auto p = place(wanted, gx, batch, m_tiles, hkv, splits, x, y);
      ++seen[((static_cast<size_t>(p.b) * hkv + p.g) * splits + p.j) * m_tiles + p.mt];
    }
  for (int n : seen)
    if (n != 1) ++failures;
}

}  // namespace

int main() {
  for (bool wanted : {false, true})
    for (int batch : {1, 2, 7})
      for (int m_tiles : {1, 3, 8})
        for (int hkv : {1, 4})
          for (int splits : {1, 5}) whole_grid(wanted, batch, m_tiles, hkv, splits);
  std::mt19937 rng(7);
  for (int i = 0; i < 200000; ++i) {
    const int m_tiles = 1 << (rng() % 9), hkv = 1 + rng() % 256, splits = 1 + rng() % 256;
    const long long gx = 1ll * m_tiles * hkv * splits;
    const int batch = 1 + rng() % 65535;
    for (int y : {0, batch / 2, batch - 1, static_cast<int>(rng() % batch)})
      for (long long x : {0ll, gx - 1, static_cast<long long>(rng() % gx)})
        place(rng() % 2 != 0, gx, batch, m_tiles, hkv, splits, static_cast<int>(x), y);
  }
  std::printf("%d failures\n", failures);
  return failures != 0;
}
