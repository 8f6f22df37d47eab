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
// the window in which a run starts owns all of it, so it may reach up to 15
// tokens into the next window (second pass) and every group is written by one
// CTA, without atomics.  A token's rotary angles are read (table) or computed
// once per CTA and serve all its heads.
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "kernels.h"
#include "rope_math.cuh"
#include "rope_rotate.cuh"

namespace pkvqk {

namespace {

constexpr int kWindow = 16;                    // tokens per CTA, one per half-warp
constexpr int kThreads = kWindow * 16;
static_assert(kWindow == kScaleGroup, "a run spans at most two windows");

// A run as one of its tokens sees it: window-relative tokens [s, e) of one
// group, the slots they write, s < 0 where the token is not this CTA's.
struct Run {
  int s, e;
  uint32_t slots;
  __device__ bool active() const { return s >= 0; }
  __device__ bool fresh() const { return (slots & 1u) != 0; }
};

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

// Finite part of |y|, and whether anything was not finite.
__device__ __forceinline__ float finite_abs(float y, bool& bad) {
  const float a = fabsf(y);
  const bool fin = a <= 3.402823466e38f;       // false for NaN too
  bad |= !fin;
  return fin ? a : 0.f;
}

__device__ __forceinline__ uint32_t half_mask() {
  return 0xffffu << (threadIdx.x & 16);
}

// Where a token's codes and its group's scale live.
struct Place {
  int64_t code, scale;                         // element offsets for head 0
  int64_t group_code;                          // code offset of the group's slot 0
};

__device__ __forceinline__ Place place(const AppendQ8Args& a, int64_t slot) {
  const int64_t blk = slot / a.base.block_size;
  const int in = static_cast<int>(slot - blk * a.base.block_size);
  Place p;
  p.group_code = blk * a.base.block_stride +
                 static_cast<int64_t>(in & ~(kScaleGroup - 1)) * a.base.slot_stride;
  p.code = p.group_code + static_cast<int64_t>(in & (kScaleGroup - 1)) * a.base.slot_stride;
  p.scale = blk * a.scales.block_stride + (in / kScaleGroup) * a.scales.group_stride;
  return p;
}

// The rest of a group follows its scale from `old` to `now`: the slots that the
// run does not write, by the half-warp of the run's first token (8 bytes a
// lane, eight slots in flight).
template <int kFormat>
__device__ __forceinline__ void rescale_group(uint8_t* codes, int64_t slot_stride, uint32_t written,
                                              float ratio, int l) {
#pragma unroll 1
  for (int b = 0; b < kScaleGroup; b += 8) {
    uint2 w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!((written >> (b + j)) & 1u))
        w[j] = *reinterpret_cast<const uint2*>(codes + (b + j) * slot_stride + 8 * l);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if ((written >> (b + j)) & 1u) continue;
      float f[4], g[4];
      decode4<kFormat>(w[j].x, f);
      decode4<kFormat>(w[j].y, g);
      *reinterpret_cast<uint2*>(codes + (b + j) * slot_stride + 8 * l) =
          make_uint2(encode4<kFormat>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio),
                     encode4<kFormat>(g[0] * ratio, g[1] * ratio, g[2] * ratio, g[3] * ratio));
    }
  }
}

struct Smem {
  // cos hi, cos lo, sin hi, sin lo; read as float4
  alignas(16) float trig[4][2 * kWindow][kHeadDim / 2];
  alignas(16) float knots[kSinCosKnots][4];
  alignas(16) float amax[2][2][2 * kWindow];   // [parity][K, V][token]
  alignas(16) int64_t slot[2 * kWindow + 1];   // of tokens window - 1 .. window + 31, -1: none
};

template <int kFormat>
__global__ void __launch_bounds__(kThreads)
norm_rope_append_q8_kernel(const __grid_constant__ AppendQ8Args a) {
  __shared__ __align__(16) Smem sm;
  const NormRopeAppendArgs& n = a.base;
  const int tid = threadIdx.x, lane = tid & 31, l = tid & 15, hw = tid >> 4;
  const int t0 = blockIdx.x * kWindow;         // first token of the window
  const int items = n.num_q_heads + n.num_kv_heads;   // kv heads first, then q heads
  const int i0 = static_cast<int>(static_cast<int64_t>(blockIdx.y) * items / a.parts);
  const int i1 = static_cast<int>(static_cast<int64_t>(blockIdx.y + 1) * items / a.parts);

  pdl_launch_dependents();
  pdl_wait();

  if (tid < 2 * kWindow + 1) {
    const int64_t t = static_cast<int64_t>(t0) - 1 + tid;
    int64_t slot = t >= 0 && t < n.num_tokens ? n.slot_mapping[t] : -1;
    if (slot >= n.num_blocks * n.block_size) {
      report(n.status_flags, kFlagBadSlot);
      slot = -1;
    }
    sm.slot[tid] = slot < 0 ? -1 : slot;
  }
  __syncthreads();
  // starts and validity of tokens window .. window + 31
  const int64_t my = sm.slot[lane + 1], before = sm.slot[lane];
  const bool valid = my >= 0;
  const uint32_t V = __ballot_sync(0xffffffffu, valid);
  const uint32_t B = __ballot_sync(
      0xffffffffu, valid && (before < 0 || before / kScaleGroup != my / kScaleGroup));
  auto run_of = [&](int j) {
    Run r{-1, -1, 0u};
    const uint32_t upto = B & ((2u << j) - 1u);
    if (((V >> j) & 1u) && upto != 0u) {
      const int s = 31 - __clz(upto);
      if (s < kWindow) {
        const uint32_t after = (B | ~V) & ~((2u << s) - 1u);
        r.s = s;
        r.e = after != 0u ? __ffs(after) - 1 : 2 * kWindow;
      }
    }
    return r;
  };
  auto slots_of = [&](Run& r) {                // the half-warp together
    uint32_t m = 0u;
    for (int j = r.s + l; r.active() && j < r.e; j += 16)
      m |= 1u << (sm.slot[j + 1] & (kScaleGroup - 1));
    r.slots = __reduce_or_sync(half_mask(), m);
  };
  Run run[2] = {run_of(hw), run_of(kWindow + hw)};
  slots_of(run[0]);
  slots_of(run[1]);
  const bool second = run_of(kWindow).active();        // uniform over the CTA

  // angles: from the table where every token of the window (and of runs that
  // reach past it) is in it, else computed, four lanes' frequencies a thread
  const int tok[2] = {t0 + hw, t0 + kWindow + hw};
  int64_t pos[2];
  bool outside = false;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    pos[p] = (p == 0 || run[p].active()) && tok[p] < n.num_tokens ? n.positions[tok[p]] : 0;
    outside |= (p == 0 || run[p].active()) && !(pos[p] >= 0 && pos[p] < n.table_positions);
  }
  const bool computed = __syncthreads_or(outside) != 0;
  if (computed) {
    for (int e = tid; e < kSinCosKnots * 4; e += kThreads)
      (&sm.knots[0][0])[e] = (&n.sincos_tab[0][0])[e];
    __syncthreads();
#pragma unroll 1
    for (int p = 0; p < (second ? 2 : 1); ++p)
#pragma unroll 1
      for (int f = l; f < kHeadDim / 2; f += 16) {
        FF x, sn, cs;
        const int quadrant = reduce_angle(static_cast<double>(pos[p]), n.inv_freq[f], &x);
        sincos_ff(x, quadrant, sm.knots, &sn, &cs);
        const int j = p * kWindow + hw;
        sm.trig[0][j][f] = cs.hi;
        sm.trig[1][j][f] = cs.lo;
        sm.trig[2][j][f] = sn.hi;
        sm.trig[3][j][f] = sn.lo;
      }
    __syncwarp();                              // a half-warp reads its own tokens only
  }
  auto trig_of = [&](int p) {
    Trig t;
    if (computed) {
      const int j = p * kWindow + hw;
      t.ch = *reinterpret_cast<const float4*>(&sm.trig[0][j][4 * l]);
      t.cl = *reinterpret_cast<const float4*>(&sm.trig[1][j][4 * l]);
      t.sh = *reinterpret_cast<const float4*>(&sm.trig[2][j][4 * l]);
      t.sl = *reinterpret_cast<const float4*>(&sm.trig[3][j][4 * l]);
    } else {
      const float4* row = n.rope_table + (pos[p] * (kHeadDim / 8) + l) * 4;
      t.ch = __ldg(row);
      t.cl = __ldg(row + 1);
      t.sh = __ldg(row + 2);
      t.sl = __ldg(row + 3);
    }
    return t;
  };
  const Trig tr = trig_of(0);
  auto gains = [&](const __nv_bfloat16* g, float (&g0)[4], float (&g1)[4]) {
    unpack4(__ldg(reinterpret_cast<const uint2*>(g + 4 * l)), g0);
    unpack4(__ldg(reinterpret_cast<const uint2*>(g + 64 + 4 * l)), g1);
  };

  // ---- kv heads of this part
  const int kv1 = min(i1, n.num_kv_heads);
  if (i0 < kv1) {
    float g0[4], g1[4];
    gains(n.gamma_k, g0, g1);
    Place at[2];
#pragma unroll
    for (int p = 0; p < 2; ++p)
      at[p] = place(a, run[p].active() ? sm.slot[p * kWindow + hw + 1] : 0);
    int parity = 0;
    bool bad = false;
#pragma unroll 1
    for (int h = i0; h < kv1; ++h, parity ^= 1) {
      float y[2][2][8];                        // [pass][K, V]
      float old[2][2];                         // scales before this call
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if (p == 1 && !second) break;
        uint2 k0, k1, v0, v1;
        k0 = k1 = v0 = v1 = make_uint2(0u, 0u);
        old[p][0] = old[p][1] = 0.f;
        if (run[p].active()) {
          const __nv_bfloat16* ks = n.k + tok[p] * n.k_stride_t + h * n.k_stride_h;
          const __nv_bfloat16* vs = n.v + tok[p] * n.v_stride_t + h * n.v_stride_h;
          k0 = __ldg(reinterpret_cast<const uint2*>(ks + 4 * l));
          k1 = __ldg(reinterpret_cast<const uint2*>(ks + 64 + 4 * l));
          v0 = __ldg(reinterpret_cast<const uint2*>(vs + 4 * l));
          v1 = __ldg(reinterpret_cast<const uint2*>(vs + 64 + 4 * l));
          if (!run[p].fresh()) {
            const int64_t so = at[p].scale + h * a.scales.head_stride;
            old[p][0] = a.scales.k[so];
            old[p][1] = a.scales.v[so];
          }
        }
        float x0[4], x1[4], o0[4], o1[4];
        unpack4(k0, x0);
        unpack4(k1, x1);
        norm_rotate(x0, x1, g0, g1, n.eps, p == 0 ? tr : trig_of(1), o0, o1);
        float w0[4], w1[4];
        unpack4(v0, w0);
        unpack4(v1, w1);
        float mk = 0.f, mv = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[p][0][j] = o0[j];
          y[p][0][4 + j] = o1[j];
          y[p][1][j] = w0[j];
          y[p][1][4 + j] = w1[j];
        }
        bool nonfinite = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          mk = fmaxf(mk, finite_abs(y[p][0][j], nonfinite));
          mv = fmaxf(mv, finite_abs(y[p][1][j], nonfinite));
        }
        if (nonfinite) {                       // NaN is stored as 0
          bad |= run[p].active();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            y[p][0][j] = y[p][0][j] == y[p][0][j] ? y[p][0][j] : 0.f;
            y[p][1][j] = y[p][1][j] == y[p][1][j] ? y[p][1][j] : 0.f;
          }
        }
        const uint32_t uk = __reduce_max_sync(half_mask(), __float_as_uint(mk));
        const uint32_t uv = __reduce_max_sync(half_mask(), __float_as_uint(mv));
        if (l == 0) {
          sm.amax[parity][0][p * kWindow + hw] = __uint_as_float(uk);
          sm.amax[parity][1][p * kWindow + hw] = __uint_as_float(uv);
        }
      }
      __syncthreads();
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if (p == 1 && !second) break;
        const Run& r = run[p];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float m = 0.f;
          for (int j = r.s + l; r.active() && j < r.e; j += 16) m = fmaxf(m, sm.amax[parity][x][j]);
          m = __uint_as_float(__reduce_max_sync(half_mask(), __float_as_uint(m)));
          if (!r.active()) continue;
          const float lo = __int_as_float((127 + kScaleMinExp) << 23);
          const float hi = __int_as_float((127 + kScaleMaxExp) << 23);
          const float want = __int_as_float((127 + scale_exponent<kFormat>(m)) << 23);
          const float prev = old[p][x] >= lo && old[p][x] <= hi ? old[p][x] : lo;
          const float now = r.fresh() ? want : fmaxf(want, prev);
          const float inv = __frcp_rn(now);    // exact: a power of two
          const float* yy = y[p][x];
          uint8_t* codes = (x == 0 ? a.k_codes : a.v_codes) + h * n.head_stride;
          *reinterpret_cast<uint32_t*>(codes + at[p].code + 4 * l) =
              encode4<kFormat>(yy[0] * inv, yy[1] * inv, yy[2] * inv, yy[3] * inv);
          *reinterpret_cast<uint32_t*>(codes + at[p].code + 64 + 4 * l) =
              encode4<kFormat>(yy[4] * inv, yy[5] * inv, yy[6] * inv, yy[7] * inv);
          if (p == 0 && r.s == hw) {           // the run's first token
            if (l == 0) (x == 0 ? a.scales.k : a.scales.v)[at[p].scale + h * a.scales.head_stride] = now;
            if (!r.fresh() && now > prev)
              rescale_group<kFormat>(codes + at[p].group_code, n.slot_stride, r.slots, prev * inv,
                                     l);
          }
        }
      }
    }
    if (bad) report(n.status_flags, kFlagBadValue);
  }

  // ---- q heads of this part
  const int q0 = max(i0 - n.num_kv_heads, 0), q1 = i1 - n.num_kv_heads;
  if (q0 >= q1) return;
  float g0[4], g1[4];
  gains(n.gamma_q, g0, g1);
  const bool live = tok[0] < n.num_tokens;
  const __nv_bfloat16* src = n.q + (live ? tok[0] : 0) * n.q_stride_t;
  __nv_bfloat16* dst = a.q_out + (live ? tok[0] : 0) * a.q_out_stride_t;
  constexpr int kAhead = 4;                    // vectors whose loads go first
#pragma unroll 1
  for (int h = q0; h < q1; h += kAhead) {
    uint2 in[kAhead][2];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      in[j][0] = in[j][1] = make_uint2(0u, 0u);
      if (live && h + j < q1) {
        const __nv_bfloat16* s = src + (h + j) * n.q_stride_h;
        in[j][0] = *reinterpret_cast<const uint2*>(s + 4 * l);
        in[j][1] = *reinterpret_cast<const uint2*>(s + 64 + 4 * l);
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (h + j >= q1) break;
      float x0[4], x1[4], o0[4], o1[4];
      unpack4(in[j][0], x0);
      unpack4(in[j][1], x1);
      norm_rotate(x0, x1, g0, g1, n.eps, tr, o0, o1);
      if (live) {
        __nv_bfloat16* d = dst + (h + j) * a.q_out_stride_h;
        *reinterpret_cast<uint2*>(d + 4 * l) =
            make_uint2(pack_bf16x2(o0[0], o0[1]), pack_bf16x2(o0[2], o0[3]));
        *reinterpret_cast<uint2*>(d + 64 + 4 * l) =
            make_uint2(pack_bf16x2(o1[0], o1[1]), pack_bf16x2(o1[2], o1[3]));
      }
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope_append_q8(const AppendQ8Args& args, cudaStream_t stream) {
  if (args.base.num_tokens == 0) return cudaSuccess;
  AppendQ8Args a = args;
  const int windows = (a.base.num_tokens + kWindow - 1) / kWindow;
  const int items = a.base.num_q_heads + a.base.num_kv_heads;
  // enough parts for six CTAs on each of 152 SMs, at most one head each
  const int want = (6 * 152 + windows - 1) / windows;
  a.parts = want < 1 ? 1 : (want > items ? items : want);
  const dim3 grid(windows, a.parts);
  return launch_pdl(a.format == kFormatE4m3 ? norm_rope_append_q8_kernel<kFormatE4m3>
                                            : norm_rope_append_q8_kernel<kFormatInt8>,
                    grid, dim3(kThreads), 0, stream, a);
}

}  // namespace pkvqk
