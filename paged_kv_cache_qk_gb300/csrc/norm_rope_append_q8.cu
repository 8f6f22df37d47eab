// Fused per-head RMSNorm + neox RoPE on q and k, with k and v quantised into an
// 8-bit paged cache.
//
// Cache: value = code * scale, a code being e4m3 or int8 and one fp32
// power-of-two scale per group of 16 consecutive slots of a page, kv head and
// tensor (K or V).  With a power of two, y / s is exact (one rounding, to the
// code), a code whose group's scale grows by 2^j is rescaled by an exact
// 2^-j (one more rounding of that code), and code * scale is exact in bf16.
// For e4m3 the choice of the power costs no relative precision above its
// subnormals; for int8 it costs at most one bit of the eight.
//
// A group's scale is 2^e, e the smallest integer with max|y| <= M 2^e (M = 448
// or 127) over the group's tokens of this call, read off the bits of max|y|;
// where the call does not write the group's slot 0 the group holds earlier
// tokens: the scale never shrinks, and when it grows the codes of the slots
// that the call does not write are rescaled.
//
// Work split: the maximum ties the tokens of one group together, so a CTA takes
// a window of 16 consecutive tokens (one per half-warp, lane l holding elements
// 4l.. and 64+4l.. as in the bf16 append) and, of the q and kv heads, a
// contiguous share.  Tokens of one group are adjacent in token order (a run);
// the window in which a run starts owns all of it, so every group is written by
// one CTA, without atomics.  Its runs are taken in chunks of whole runs, at most
// 16 tokens each: one chunk where groups and windows are aligned or shifted against
// each other alike (it then reaches into the next window), two at most where runs
// of different sequences meet.  A token's rotary angles are read (table) or
// computed once per CTA and chunk and serve all its heads; the next head's values
// load while a head is being quantised.
//
// Bound, many tokens: instructions and the latencies between them, not HBM (4 x 2048
// tokens, 16 q and 8 kv heads: 37.7 us where the bytes need 17.4; 205 instructions a
// warp and head vector against the bf16 append's 150, issue slots 62 % busy).  Few
// tokens: the chain slots -> angles, values, scales -> maxima -> codes (64 tokens 4.1
// us, the bf16 append 2.5).  A K value nearer the middle of two codes than the fp32
// norm's and rotation's 2^-20 could get either code; settling those in pairs of floats
// costs calls of few tokens 0.1 us (64) to 0.9 (32 x 5), and is done there; many tokens
// 5 us of 38, for the registers it takes, and is not.
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "kernels.h"
#include "rope_math.cuh"
#include "rope_rotate.cuh"

namespace pkvqk {

namespace {

constexpr int kWindow = 16;                    // tokens per CTA, one per half-warp
constexpr int kThreads = kWindow * 16;
// Many tokens: four CTAs share an SM at 64 registers, with a few spills; few: two,
// without (16 q and 8 kv heads, 1024 tokens: 9.4 us with two, 10.7 with four; 1600:
// 11.5, 11.9; 2048: 14.7, 14.0; 8192: 49.6, 37.4; three CTAs an SM 41.2).  A window's
// head vectors are cut so that at most two waves of CTAs come (512 tokens 7.5 us, three
// waves 9.8; 2048: 14.0, 17.0; 4096: 20.3, 22.7), or three where two would leave a CTA
// more than a quarter of them (8192: 37.4 us, two waves 39.2).
constexpr int kManyTokens = 2048;
constexpr int kManyCtas = 4, kFewCtas = 2;
static_assert(kWindow == kScaleGroup, "a run spans at most two windows");

template <int kFormat>
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int k = static_cast<int>(u >> 23) - 127;
  const uint32_t mant = u & 0x7fffffu;
  // 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6
  const int e = kFormat == kFormatE4m3 ? k - 8 + (mant > 0x600000u ? 1 : 0)
                                       : k - 6 + (mant > 0x7e0000u ? 1 : 0);
  return max(kScaleMinExp, min(kScaleMaxExp, amax > 0.f ? e : kScaleMinExp));
}

// Four values to four codes: nearest, ties to even; beyond the largest code
// (infinities, or a scale at its limit) the largest.
template <int kFormat>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if (kFormat == kFormatE4m3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
  auto code = [](float x) {
    return static_cast<uint32_t>(max(-127, min(127, __float2int_rn(x)))) & 0xffu;
  };
  return code(a) | (code(b) << 8) | (code(c) << 16) | (code(d) << 24);
}

template <int kFormat>
__device__ __forceinline__ void decode4(uint32_t w, float (&f)[4]) {
  if (kFormat == kFormatE4m3) {
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<uint16_t>(w)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<uint16_t>(w >> 16)));
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
  }
}

// max(a, |b|, |c|) for a >= 0, NaN if any is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The largest |y| of eight values; where that is not finite, NaN in y becomes 0
// (which is how it is stored), infinities do not count, the result is of the finite
// ones, and `bad` is set if the values are a token's (the zeros of a half-warp without
// one become NaN where eps is 0).
__device__ __forceinline__ float max_finite(float (&y)[8], bool token, bool& bad) {
  float m = max_abs3(max_abs3(0.f, y[0], y[1]), y[2], y[3]);
  m = max_abs3(max_abs3(m, y[4], y[5]), y[6], y[7]);
  if (!(m <= 3.402823466e38f)) {
    bad = bad || token;
    m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = y[e] == y[e] ? y[e] : 0.f;
      const float v = fabsf(y[e]);
      m = fmaxf(m, v <= 3.402823466e38f ? v : 0.f);
    }
  }
  return m;
}

// Over the half-warp.  Shuffles: one reduction instruction per half, with two masks
// in a warp, runs them one after the other (4 x 2048 tokens 42.5 us against 38.4).
__device__ __forceinline__ float half_warp_max(float m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// Where a token's codes and its group's scale live: offsets for head 0.
struct Place {
  int64_t code, scale;
};

__device__ __forceinline__ Place place(const AppendQ8Args& a, int64_t slot) {
  // 32-bit where that holds it: a 64-bit division is ~100 instructions
  const int64_t blk = slot <= 0xffffffffll
                          ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(a.base.block_size)
                          : slot / a.base.block_size;
  const int in = static_cast<int>(slot - blk * a.base.block_size);
  Place p;
  p.code = blk * a.base.block_stride + in * a.base.slot_stride;
  p.scale = blk * a.scales.block_stride + (in / kScaleGroup) * a.scales.group_stride;
  return p;
}

// A group whose scale grew: its other slots' codes follow it.
struct Grown {
  uint8_t* codes;                              // the group's slot 0
  uint32_t written;                            // slots that the call writes: left alone
  float ratio;                                 // old scale / new scale
};
constexpr int kMostGrown = kWindow;            // per head: one a run

struct Smem {
  // cos hi, cos lo, sin hi, sin lo of the half-warps' tokens, 64 frequencies each
  alignas(16) float trig[4][kWindow][kHeadDim / 2];
  alignas(16) float knots[kSinCosKnots][4];
  alignas(16) float amax[2][kWindow];          // [parity][half-warp]
  alignas(16) Grown grown[3][kMostGrown];
  int num_grown[3];
  alignas(16) int64_t slot[2 * kWindow + 1];   // of tokens window - 1 .. window + 31, -1: none
  int64_t pos[2 * kWindow + 1];                // theirs; 0 where there is no token
};

// The half-warp's angles of position pos into its part of shared memory: from the
// table, or computed (four frequencies a lane).
__device__ __forceinline__ void put_angles(const NormRopeAppendArgs& n, Smem& sm, int64_t pos,
                                           bool computed, int hw, int l) {
  __syncwarp();                                // reads of the token before
  if (!computed) {
    // float4 f of the row: component f % 4 of lane f / 4
    const float4* row = n.rope_table + pos * (kHeadDim / 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int f = i * 16 + l;
      *reinterpret_cast<float4*>(&sm.trig[f & 3][hw][(f >> 2) * 4]) = __ldg(row + f);
    }
  } else {
#pragma unroll 1
    for (int f = l; f < kHeadDim / 2; f += 16) {
      FF x, sn, cs;
      const int quadrant = reduce_angle(static_cast<double>(pos), n.inv_freq[f], &x);
      sincos_ff(x, quadrant, sm.knots, &sn, &cs);
      sm.trig[0][hw][f] = cs.hi;
      sm.trig[1][hw][f] = cs.lo;
      sm.trig[2][hw][f] = sn.hi;
      sm.trig[3][hw][f] = sn.lo;
    }
  }
  __syncwarp();
}

// Read where they are used (and not kept over the heads: the registers let four
// CTAs share an SM).
__device__ __forceinline__ float4 lds_f4(const float* p) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(smem_addr(p)));
  return v;
}
__device__ __forceinline__ Trig angles(const Smem& sm, int hw, int l) {
  Trig t;
  t.ch = lds_f4(&sm.trig[0][hw][4 * l]);
  t.cl = lds_f4(&sm.trig[1][hw][4 * l]);
  t.sh = lds_f4(&sm.trig[2][hw][4 * l]);
  t.sl = lds_f4(&sm.trig[3][hw][4 * l]);
  return t;
}

__device__ __forceinline__ void gains(const __nv_bfloat16* g, int l, float (&g0)[4],
                                      float (&g1)[4]) {
  unpack4(__ldg(reinterpret_cast<const uint2*>(g + 4 * l)), g0);
  unpack4(__ldg(reinterpret_cast<const uint2*>(g + 64 + 4 * l)), g1);
}

// The codes of grown groups, half-warp hw slot hw of each (8 bytes a lane, four
// groups in flight).
template <int kFormat>
__device__ __forceinline__ void rescale(const Grown* list, int count, int64_t slot_stride, int hw,
                                        int l) {
#pragma unroll 1
  for (int g = 0; g < count; g += 4) {
    uint2 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (g + i < count && !((list[g + i].written >> hw) & 1u))
        w[i] = *reinterpret_cast<const uint2*>(list[g + i].codes + hw * slot_stride + 8 * l);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (g + i >= count || ((list[g + i].written >> hw) & 1u)) continue;
      const float r = list[g + i].ratio;
      float x[4], y[4];
      decode4<kFormat>(w[i].x, x);
      decode4<kFormat>(w[i].y, y);
      *reinterpret_cast<uint2*>(list[g + i].codes + hw * slot_stride + 8 * l) =
          make_uint2(encode4<kFormat>(x[0] * r, x[1] * r, x[2] * r, x[3] * r),
                     encode4<kFormat>(y[0] * r, y[1] * r, y[2] * r, y[3] * r));
    }
  }
}

// The scale of a group from its run's maximum m; *prev: the stored one as it counts.
template <int kFormat>
__device__ __forceinline__ float group_scale(float m, float stored, uint32_t written,
                                             float* prev) {
  const float lo = __int_as_float((127 + kScaleMinExp) << 23);
  const float hi = __int_as_float((127 + kScaleMaxExp) << 23);
  const float want = __int_as_float((127 + scale_exponent<kFormat>(m)) << 23);
  *prev = stored >= lo && stored <= hi ? stored : lo;
  return (written & 1u) ? want : fmaxf(want, *prev);
}

// Is one of z = y / scale so near the middle of two codes that the fp32 norm and
// rotation may have taken it across?  They are within 13 half-ulps of y (the sum of
// squares 12 roundings deep, halved by the square root: 6; the mean 1, the square root
// 4, the difference and the product 2).  e4m3: the 20 bits below a code's mantissa
// against their middle (subnormal codes, 2^-14 of the group's maximum, are left as
// they are).
template <int kFormat>
__device__ __forceinline__ bool near_middle(const float (&z)[8]) {
  if (kFormat == kFormatE4m3) {
    uint32_t d = ~0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) d = min(d, (__float_as_uint(z[e]) - (0x80000u - 14u)) & 0xfffffu);
    return d <= 28u;
  }
  constexpr float kRound = 12582912.f;         // 1.5 * 2^23: its unit is 1
  const uint64_t up = pack2(kRound, kRound);
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const uint64_t v = pack2(z[e], z[e + 1]);
    float d0, d1;
    unpack2(sub2(v, sub2(add2(v, up), up)), d0, d1);
    m = fmaxf(m, fmaf(fabsf(z[e]), 14.f * 0x1p-24f, fabsf(d0)));
    m = fmaxf(m, fmaf(fabsf(z[e + 1]), 14.f * 0x1p-24f, fabsf(d1)));
  }
  return m >= 0.5f;
}

// The lane's eight values as codes (dims 4l.. at `code`, 64 + 4l.. 64 bytes on).
template <int kFormat>
__device__ __forceinline__ void write_codes(const float (&z)[8], uint8_t* code) {
  *reinterpret_cast<uint32_t*>(code) = encode4<kFormat>(z[0], z[1], z[2], z[3]);
  *reinterpret_cast<uint32_t*>(code + 64) = encode4<kFormat>(z[4], z[5], z[6], z[7]);
}

// hi + lo to float by truncation, the lowest bit set where something was cut off: a
// rounding to 8 bits that follows is that of the sum.
__device__ __forceinline__ float to_odd(float hi, float lo) {
  uint32_t u = __float_as_uint(hi);
  if (lo == 0.f || hi == 0.f) return hi;
  if ((lo < 0.f) != (hi < 0.f)) --u;           // towards zero
  return __uint_as_float(u | 1u);
}

// The codes of one K head vector by a half-warp from the norm and rotation in pairs of
// floats (2^-40), for the ~0.5 % of vectors with a value that fp32 leaves in doubt.
// inv: 1 / scale.
template <int kFormat>
__device__ __noinline__ void settle_codes(const NormRopeAppendArgs& n, const Smem& sm,
                                          const __nv_bfloat16* src, float inv, uint8_t* code) {
  const int l = threadIdx.x & 15, hw = threadIdx.x >> 4;
  const uint32_t half = 0xffffu << (threadIdx.x & 16);
  float x0[4], x1[4], g0[4], g1[4], z[8];
  unpack4(__ldg(reinterpret_cast<const uint2*>(src)), x0);
  unpack4(__ldg(reinterpret_cast<const uint2*>(src + 64)), x1);
  unpack4(__ldg(reinterpret_cast<const uint2*>(n.gamma_k + 4 * l)), g0);
  unpack4(__ldg(reinterpret_cast<const uint2*>(n.gamma_k + 64 + 4 * l)), g1);
  FF ss = {0.f, 0.f};                          // squares of bf16 values are exact
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = j < 4 ? x0[j & 3] : x1[j & 3];
    const FF t = two_sum(ss.hi, PKVQK_MUL(x, x));
    ss = {t.hi, PKVQK_ADD(ss.lo, t.lo)};
  }
#pragma unroll 1
  for (int o = 8; o > 0; o >>= 1)
    ss = ff_add(ss, {__shfl_xor_sync(half, ss.hi, o), __shfl_xor_sync(half, ss.lo, o)});
  const FF m = ff_add({ss.hi * (1.f / kHeadDim), ss.lo * (1.f / kHeadDim)}, {n.eps, 0.f});
  // one Newton step in pairs from the fp32 root
  const float r0 = rsqrtf(m.hi);
  const FF t = ff_mul(m, ff_mul({r0, 0.f}, {r0, 0.f}));
  const FF r = {r0, 0.5f * r0 * PKVQK_SUB(PKVQK_SUB(1.f, t.hi), t.lo)};
  bool finite = true;
#pragma unroll 1
  for (int half_of = 0; half_of < 2; ++half_of) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const FF c = {sm.trig[0][hw][4 * l + j], sm.trig[1][hw][4 * l + j]};
      const float sign = half_of ? 1.f : -1.f;
      const FF w = {sign * sm.trig[2][hw][4 * l + j], sign * sm.trig[3][hw][4 * l + j]};
      const float a = x0[j] * g0[j], b = x1[j] * g1[j];   // exact
      // first half a c - b s, second b c + a s
      const FF y = ff_mul(r, ff_add(ff_mul({half_of ? b : a, 0.f}, c), ff_mul({half_of ? a : b, 0.f}, w)));
      const float v = to_odd(y.hi * inv, y.lo * inv);
      finite = finite && fabsf(y.hi * inv) <= 3.402823466e38f;
      z[j] = half_of ? z[j] : v;
      z[4 + j] = v;
    }
  }
  if (finite) write_codes<kFormat>(z, code);   // else those of fp32 stay
}

// K (kIsK) or V of kv heads [h0, h1): the runs that start in the window.
template <int kFormat, bool kIsK, bool kFew>
__device__ __forceinline__ void append_heads(const AppendQ8Args& a, Smem& sm, bool computed,
                                             int h0, int h1) {
  const NormRopeAppendArgs& n = a.base;
  const int tid = threadIdx.x, lane = tid & 31, l = tid & 15, hw = tid >> 4;
  const int t0 = blockIdx.x * kWindow;
  // of the tokens window .. window + 31, B: those that start a run; E: those, and those
  // without a slot, so that a position of E, or 32, ends the run before it
  const int64_t my = sm.slot[lane + 1], before = sm.slot[lane];
  const uint32_t B = __ballot_sync(
      0xffffffffu, my >= 0 && (before < 0 || before / kScaleGroup != my / kScaleGroup));
  const uint32_t E = B | __ballot_sync(0xffffffffu, my < 0);
  auto next_end = [&](uint32_t from) {         // the first of E among the bits `from`
    const uint32_t e = E & from;
    return e != 0u ? __ffs(e) - 1 : 2 * kWindow;
  };

  // head k of all chunks: maxima in buffer k % 2; grown groups in list k % 3,
  // rescaled at the next head's barrier and emptied at the one after
  int k = 0, list = 0;
  bool bad = false;
  uint32_t todo = B & 0xffffu;                 // runs that start in the window
#pragma unroll 1
  while (todo != 0u) {                         // uniform over the CTA
    // chunk [b, end): whole runs that start in the window, at most 16 tokens;
    // half-warp hw has token b + hw
    const int b = __ffs(todo) - 1, most = min(b + kWindow, next_end(0xffffu << kWindow));
    const uint32_t ends = E & ((2u << most) - 1u) & ~((2u << b) - 1u);   // b + 1 .. most
    // none: more tokens than slots, some given twice
    const int end = ends != 0u ? 31 - __clz(ends) : most;
    todo &= ~0u << end;
    const int j = b + hw;
    const bool active = j < end && (((~E | B) >> j) & 1u);
    const int rs = active ? 31 - __clz(B & ((2u << j) - 1u)) : j;
    const int re = active ? min(next_end(~0u << j << 1), end) : j;
    const bool first = active && j == rs;
    uint32_t written = 0u;                     // slots of the group that the run writes
    if (rs + l < re) written = 1u << (sm.slot[rs + l + 1] & (kScaleGroup - 1));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) written |= __shfl_xor_sync(0xffffffffu, written, o);
    const int peer = rs + l < re ? rs + l - b : -1;   // half-warp whose maximum this lane takes
    const int64_t tok = active ? t0 + j : 0;
    // of head h: this lane's values, code chunk and scale
    const int64_t stride_h = kIsK ? n.k_stride_h : n.v_stride_h;
    const __nv_bfloat16* src =
        (kIsK ? n.k + tok * n.k_stride_t : n.v + tok * n.v_stride_t) + h0 * stride_h + 4 * l;
    uint8_t* code;
    float* scale;
    {
      const Place at = place(a, active ? sm.slot[j + 1] : 0);
      code = (kIsK ? a.k_codes : a.v_codes) + at.code + h0 * n.head_stride + 4 * l;
      scale = (kIsK ? a.scales.k : a.scales.v) + at.scale + h0 * a.scales.head_stride;
    }
    const int offset = active ? static_cast<int>(sm.slot[j + 1] & (kScaleGroup - 1)) : 0;
    uint2 x0w = make_uint2(0u, 0u), x1w = x0w;
    float next_scale = 0.f;
    if (active) {
      x0w = __ldg(reinterpret_cast<const uint2*>(src));
      x1w = __ldg(reinterpret_cast<const uint2*>(src + 64));
      if (!(written & 1u)) next_scale = *scale;
    }
    if (kIsK) put_angles(n, sm, active ? sm.pos[j + 1] : 0, computed, hw, l);
#pragma unroll 1
    for (int h = h0; h < h1; ++h, ++k) {
      float x0[4], x1[4], y[8];
      unpack4(x0w, x0);
      unpack4(x1w, x1);
      const float stored = next_scale;
      src += stride_h;
      if (active && h + 1 < h1) {              // the next head's
        x0w = __ldg(reinterpret_cast<const uint2*>(src));
        x1w = __ldg(reinterpret_cast<const uint2*>(src + 64));
        if (!(written & 1u)) next_scale = scale[a.scales.head_stride];
      }
      if (kIsK) {
        float o0[4], o1[4], g0[4], g1[4];
        gains(n.gamma_k, l, g0, g1);
        norm_rotate(x0, x1, g0, g1, n.eps, angles(sm, hw, l), o0, o1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] = o0[e];
          y[4 + e] = o1[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] = x0[e];
          y[4 + e] = x1[e];
        }
      }
      float m = max_finite(y, active, bad);
      m = half_warp_max(m);
      if (l == 0) sm.amax[k & 1][hw] = m;
      __syncthreads();
      rescale<kFormat>(sm.grown[list], sm.num_grown[list], n.slot_stride, hw, l);
      list = list == 2 ? 0 : list + 1;
      if (tid == 0) sm.num_grown[list == 2 ? 0 : list + 1] = 0;
      m = peer >= 0 ? sm.amax[k & 1][peer] : 0.f;
      m = half_warp_max(m);
      if (active) {
        float prev;
        const float now = group_scale<kFormat>(m, stored, written, &prev);
        const float inv = __frcp_rn(now);      // exact for a power of two
        const uint64_t inv2 = pack2(inv, inv);
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) unpack2(mul2(pack2(y[e], y[e + 1]), inv2), z[e], z[e + 1]);
        write_codes<kFormat>(z, code);
        // V is not rounded before
        if (kIsK && kFew && __any_sync(0xffffu << (threadIdx.x & 16), near_middle<kFormat>(z)))
          settle_codes<kFormat>(n, sm, src - stride_h, inv, code);
        if (first && l == 0) {
          *scale = now;
          if (!(written & 1u) && now > prev)
            sm.grown[list][atomicAdd(&sm.num_grown[list], 1)] = {
                code - offset * n.slot_stride, written, prev * inv};
        }
      }
      code += n.head_stride;
      scale += a.scales.head_stride;
    }
  }
  __syncthreads();
  rescale<kFormat>(sm.grown[list], sm.num_grown[list], n.slot_stride, hw, l);
  __syncthreads();
  if (tid < 3) sm.num_grown[tid] = 0;          // for the next tensor (it has a barrier before use)
  if (bad) report(n.status_flags, kFlagBadValue);
}

template <int kFormat, int kMinCtas>
__global__ void __launch_bounds__(kThreads, kMinCtas)
norm_rope_append_q8_kernel(const __grid_constant__ AppendQ8Args a) {
  __shared__ Smem sm;
  const NormRopeAppendArgs& n = a.base;
  const int tid = threadIdx.x, l = tid & 15, hw = tid >> 4;
  const int t0 = blockIdx.x * kWindow;         // first token of the window
  // head vectors of this part: K of the kv heads, V of them, q heads
  const int hkv = n.num_kv_heads, items = n.num_q_heads + 2 * hkv;
  const int i0 = static_cast<int>(static_cast<int64_t>(blockIdx.y) * items / a.parts);
  const int i1 = static_cast<int>(static_cast<int64_t>(blockIdx.y + 1) * items / a.parts);

  pdl_launch_dependents();
  pdl_wait();

  // slots of the window and the next one; are their positions in the table?
  bool outside = false;
  if (tid < 2 * kWindow + 1) {
    const int64_t t = static_cast<int64_t>(t0) - 1 + tid;
    const bool live = t >= 0 && t < n.num_tokens;
    int64_t slot = live ? n.slot_mapping[t] : -1;
    if (slot >= n.num_blocks * n.block_size) {
      report(n.status_flags, kFlagBadSlot);
      slot = -1;
    }
    sm.slot[tid] = slot < 0 ? -1 : slot;
    if (tid < 3) sm.num_grown[tid] = 0;
    const int64_t pos = live ? n.positions[t] : 0;
    sm.pos[tid] = pos;
    outside = tid > 0 && !(pos >= 0 && pos < n.table_positions);
  }
  const bool computed = __syncthreads_or(outside) != 0;
  if (computed) {
    for (int e = tid; e < kSinCosKnots * 4; e += kThreads)
      (&sm.knots[0][0])[e] = (&n.sincos_tab[0][0])[e];
    __syncthreads();
  }
  constexpr bool kFew = kMinCtas == kFewCtas;
  if (i0 < hkv) append_heads<kFormat, true, kFew>(a, sm, computed, i0, min(i1, hkv));
  if (i0 < 2 * hkv && i1 > hkv)
    append_heads<kFormat, false, kFew>(a, sm, computed, max(i0 - hkv, 0), min(i1 - hkv, hkv));

  // ---- q heads of this part
  const int q0 = max(i0 - 2 * hkv, 0), q1 = i1 - 2 * hkv;
  if (q0 >= q1) return;
  const bool live = t0 + hw < n.num_tokens;
  const int64_t tok = live ? t0 + hw : 0;
  put_angles(n, sm, sm.pos[hw + 1], computed, hw, l);
  float g0[4], g1[4];
  gains(n.gamma_q, l, g0, g1);
  const __nv_bfloat16* src = n.q + tok * n.q_stride_t;
  __nv_bfloat16* dst = a.q_out + tok * a.q_out_stride_t;
  constexpr int kAhead = 4;                    // vectors whose loads go first
#pragma unroll 1
  for (int h = q0; h < q1; h += kAhead) {
    uint2 in[kAhead][2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      in[i][0] = in[i][1] = make_uint2(0u, 0u);
      if (live && h + i < q1) {
        const __nv_bfloat16* x = src + (h + i) * n.q_stride_h;
        in[i][0] = *reinterpret_cast<const uint2*>(x + 4 * l);
        in[i][1] = *reinterpret_cast<const uint2*>(x + 64 + 4 * l);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (h + i >= q1) break;
      float x0[4], x1[4], o0[4], o1[4];
      unpack4(in[i][0], x0);
      unpack4(in[i][1], x1);
      norm_rotate(x0, x1, g0, g1, n.eps, angles(sm, hw, l), o0, o1);
      if (live) {
        __nv_bfloat16* d = dst + (h + i) * a.q_out_stride_h;
        *reinterpret_cast<uint2*>(d + 4 * l) =
            make_uint2(pack_bf16x2(o0[0], o0[1]), pack_bf16x2(o0[2], o0[3]));
        *reinterpret_cast<uint2*>(d + 64 + 4 * l) =
            make_uint2(pack_bf16x2(o1[0], o1[1]), pack_bf16x2(o1[2], o1[3]));
      }
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope_append_q8(const AppendQ8Args& args, int sm_count,
                                       cudaStream_t stream) {
  if (args.base.num_tokens == 0) return cudaSuccess;
  AppendQ8Args a = args;
  const int windows = (a.base.num_tokens + kWindow - 1) / kWindow;
  const int items = a.base.num_q_heads + 2 * a.base.num_kv_heads;
  // parts of a window, at least one head vector each
  const bool many = a.base.num_tokens >= kManyTokens;
  const int wave = sm_count * (many ? kManyCtas : kFewCtas);
  int want = 2 * wave / windows;
  if (want < 4) want = (3 * wave + windows - 1) / windows;
  a.parts = want > items ? items : want;
  const dim3 grid(windows, a.parts);
  if (a.format == kFormatE4m3)
    return launch_pdl(many ? norm_rope_append_q8_kernel<kFormatE4m3, kManyCtas>
                           : norm_rope_append_q8_kernel<kFormatE4m3, kFewCtas>,
                      grid, dim3(kThreads), 0, stream, a);
  return launch_pdl(many ? norm_rope_append_q8_kernel<kFormatInt8, kManyCtas>
                         : norm_rope_append_q8_kernel<kFormatInt8, kFewCtas>,
                    grid, dim3(kThreads), 0, stream, a);
}

}  // namespace pkvqk
