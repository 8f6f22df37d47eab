// Order in which the multi-query attention kernel's CTAs take their work: which
// (sequence, kv head, split, pair of row tiles) the CTA at (x, y) of a grid of
// gx = m_tiles * num_kv_heads * num_splits by `batch` CTAs has.  Plain C++, for the
// kernel and for the host test of its arithmetic.
#pragma once

#include <climits>

#if defined(__CUDACC__)
#define PKVQK_HD __host__ __device__ __forceinline__
#else
#define PKVQK_HD inline
#endif

namespace pkvqk {

struct PrefillPlace {
  int b, g, j, mt;
};

// Whether the grid may run over every sequence's last row tiles first: where that is
// wanted and a CTA's number in the whole grid fits 32 bits.
PKVQK_HD bool row_tile_major(bool wanted, long long gx, int batch) {
  return wanted && gx * batch <= INT_MAX;
}

PKVQK_HD PrefillPlace place_cta(bool mt_major, int x, int y, int gx, int batch, int m_tiles,
                                int num_kv_heads, int num_splits) {
  PrefillPlace p;
  if (mt_major) {
    // the launch order runs over all sequences' last row tiles first: for
    // fresh prompts a row tile's keys grow with its index, so this hands the
    // longest work out first
    const int per_mt = batch * num_kv_heads * num_splits;
    x += y * gx;
    p.mt = m_tiles - 1 - x / per_mt;
    x %= per_mt;
    p.b = x / (num_kv_heads * num_splits);
    x %= num_kv_heads * num_splits;
    p.g = x / num_splits;
    p.j = x % num_splits;
  } else {
    // within a (sequence, kv head) the last row tile (the most keys) first
    p.mt = m_tiles - 1 - x % m_tiles;
    x /= m_tiles;
    p.g = x % num_kv_heads;
    p.j = x / num_kv_heads;
    p.b = y;
  }
  return p;
}

}  // namespace pkvqk

#undef PKVQK_HD
