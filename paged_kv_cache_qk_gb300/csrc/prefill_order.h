// Rule of the multi-query attention kernel's launch order, for the launch and for the
// host test of the kernel's arithmetic under it.
#pragma once

#include <climits>

namespace pkvqk {

// Whether the grid of gx = m_tiles * num_kv_heads * num_splits by `batch` CTAs may run
// over every sequence's last row tiles first: where that is wanted and a CTA's number in
// the whole grid, which the kernel then works out, fits 32 bits.
inline bool row_tile_major(bool wanted, long long gx, int batch) {
  return wanted && gx * batch <= INT_MAX;
}

}  // namespace pkvqk
