// What the scored attention kernels do to a score, and which keys a row sees.
//
// A score s = scale <q, K_n> of the row at position p becomes, in this order,
//     s = c tanh(s / c)          (a cap c > 0)
//     s = s - slope_h |p - n|    (a bias by distance)
// and counts where lo <= n < hi, with
//     lo = max(0, p - window + 1, first_key of the row),
//     hi = max(p + 1, min(prefix_len of the sequence, seq_len)):
// every combination of a causal mask, a window, first keys and a prefix leaves a row one
// interval of keys.  (Documents are first keys under the causal mask; a row's interval has no
// end of its document, so a prefix is the first document's and ends inside it.)  Scores are
// kept in units of log2(e), so that the softmax's 2^x takes them as they are.
//
// tanh without cancellation: up to |x| = 0.5 x Q(x^2), Q of degree 3 fitted to tanh(x) / x at
// Chebyshev nodes (largest relative error 5.5e-7, 5.9e-7 evaluated in fp32), which takes no
// special-function unit; beyond, 1 - 2 / (1 + e^2x), whose absolute error of ~1.2e-7 is
// 2.6e-7 of the value at most there.  A score's own size decides which it gets, so that no
// row's bits depend on another's; a warp computes the second form only where one of its
// scores needs it (exponentials and reciprocals are what the softmax itself is short of).
#pragma once

#include "device_common.cuh"
#include "kernels.h"

namespace pkvqk {

constexpr float kTanhSquare = 0.25f;           // x^2 up to which the polynomial serves
__device__ __forceinline__ constexpr float tanh_q(int i) {
  return i == 0 ? 0.99999946f : i == 1 ? -0.33326375f : i == 2 ? 0.13190912f : -0.04441858f;
}

// 1 - 2 / (1 + e^(2 x)), e^(2 x) = 2^(2 log2(e) x)
__device__ __forceinline__ float tanh_far(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * 2.885390081777927f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return fmaf(-2.f, r, 1.f);
}

// What raw scores are multiplied by: to log2 units, or to units of the cap.
__device__ __forceinline__ float score_factor(const ScoreRules& r, float scale_log2) {
  return r.cap > 0.f ? scale_log2 * r.inv_cap : scale_log2;
}

// N scores (pairs of them) of every lane of a warp, in units of the cap, to capped ones.
template <int N>
__device__ __forceinline__ void cap_scores(const ScoreRules& r, float (&x)[N]) {
  // the largest |score| decides what is computed; a NaN that is hidden later does not count
  float big = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) big = fmaxf(big, fabsf(x[i]));
  const bool far = __any_sync(0xffffffffu, big * big > kTanhSquare);
  const uint64_t cap2 = pack2(r.cap, r.cap);
  auto near = [&](uint64_t z) {
    const uint64_t u = mul2(z, z);
    uint64_t q = pack2(tanh_q(3), tanh_q(3));
#pragma unroll
    for (int k = 2; k >= 0; --k) q = fma2(q, u, pack2(tanh_q(k), tanh_q(k)));
    return mul2(mul2(z, cap2), q);
  };
  if (!far) {
#pragma unroll
    for (int i = 0; i < N; i += 2) unpack2(near(pack2(x[i], x[i + 1])), x[i], x[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float x0 = x[i], x1 = x[i + 1];
      unpack2(near(pack2(x0, x1)), x[i], x[i + 1]);
      if (!(x0 * x0 <= kTanhSquare)) x[i] = r.cap * tanh_far(x0);
      if (!(x1 * x1 <= kTanhSquare)) x[i + 1] = r.cap * tanh_far(x1);
    }
  }
}

// The keys [lo, hi) that the row at position p sees; row: its place among the call's
// token rows, L: its sequence's keys.
struct Interval {
  int lo, hi;
};
__device__ __forceinline__ int window_start(const ScoreRules& r, int p) {
  return r.window > 0 && p >= r.window ? p - r.window + 1 : 0;
}
__device__ __forceinline__ int prefix_end(const ScoreRules& r, int b, int L) {
  return r.prefix_lens != nullptr ? min(r.prefix_lens[b], L) : 0;
}
__device__ __forceinline__ Interval visible_keys(const ScoreRules& r, int b, long long row, int p,
                                                 int L) {
  if (r.window == 0 && r.first_keys == nullptr && r.prefix_lens == nullptr) return {0, p + 1};
  Interval v;
  v.lo = window_start(r, p);
  if (r.first_keys != nullptr) v.lo = max(v.lo, r.first_keys[row]);
  v.hi = max(p + 1, prefix_end(r, b, L));
  return v;
}

}  // namespace pkvqk
