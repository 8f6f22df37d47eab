// Host walk of the multi-query attention kernel's launch order under the launch's rule
// (csrc/prefill_order.h): every CTA's place, by the arithmetic of place_work in
// csrc/prefill_kernel.cuh, lies inside the call and every place is taken once, in grids
// of all sizes that the entry points allow: 65535 sequences, 2^31 - 1 CTAs a sequence.
// Built with wrapping integers, as the GPU's are.
#include <cstdio>
#include <random>
#include <vector>

#include "../../paged_kv_cache_qk_gb300/csrc/prefill_order.h"

namespace {

int failures = 0;

struct Place {
  int b, g, j, mt;
};

Place place(bool wanted, long long gx, int batch, int m_tiles, int hkv, int splits, int cta_x,
            int cta_y) {
  Place p;
  int x = cta_x;
  if (pkvqk::row_tile_major(wanted, gx, batch)) {
    const int per_mt = batch * hkv * splits;
    x = cta_y * static_cast<int>(gx) + cta_x;
    p.mt = m_tiles - 1 - x / per_mt;
    x %= per_mt;
    p.b = x / (hkv * splits);
    x %= hkv * splits;
    p.g = x / splits;
    p.j = x % splits;
  } else {
    p.mt = m_tiles - 1 - x % m_tiles;
    x /= m_tiles;
    p.g = x % hkv;
    p.j = x / hkv;
    p.b = cta_y;
  }
  if (p.b < 0 || p.b >= batch || p.g < 0 || p.g >= hkv || p.j < 0 || p.j >= splits || p.mt < 0 ||
      p.mt >= m_tiles) {
    if (failures++ < 8)
      std::printf("batch %d, %d row tiles, %d heads, %d splits: CTA (%d, %d) has %d %d %d %d\n",
                  batch, m_tiles, hkv, splits, cta_x, cta_y, p.b, p.g, p.j, p.mt);
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
