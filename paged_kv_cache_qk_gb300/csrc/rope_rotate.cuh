// Norm and rotation of one head vector held by a half-warp, shared by the
// bf16 and the 8-bit append kernels: lane l holds elements [4l, 4l + 4) and
// their rotate-half partners [64 + 4l, 64 + 4l + 4).
#pragma once

#include "device_common.cuh"

namespace pkvqk {

// sin/cos of this lane's four frequencies 4l .. 4l+3, float-float pairs.
struct Trig {
  float4 ch, cl, sh, sl;
};

__device__ __forceinline__ void unpack4(const uint2& u, float* f) {
  f[0] = bf16lo(u.x); f[1] = bf16hi(u.x);
  f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
}

__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// r * (a c - b s) for c = ch + cl, s = sh + sl, two elements at once (packed
// f32x2, each lane rounded as the scalar instruction rounds it): the products
// a*ch and b*sh error-free (p1 = a ch rounded, its error -(p1 - a ch) from
// one fma against -ch; q2 = b sh rounded, the error of -b sh as q2 - b sh),
// the low parts and the error terms added last.  nch, nsh, nsl are -ch, -sh,
// -sl (exact), so no negation is spent per element.
__device__ __forceinline__ uint64_t rotate2(uint64_t a, uint64_t b, uint64_t ch, uint64_t nch,
                                            uint64_t cl, uint64_t sh, uint64_t nsh, uint64_t nsl,
                                            uint64_t r) {
  const uint64_t p1 = mul2(a, ch);
  const uint64_t m1 = fma2(a, nch, p1);
  const uint64_t q2 = mul2(b, sh);
  const uint64_t e2 = fma2(b, nsh, q2);
  const uint64_t tail = add2(fma2(a, cl, mul2(b, nsl)), sub2(e2, m1));
  return mul2(r, add2(sub2(p1, q2), tail));
}

// One head vector: RMS norm with gains g, then the rotation, in fp32 (not yet
// rounded to a storage type).  Both half-warps of a warp call it together.
__device__ __forceinline__ void norm_rotate(const float (&x0)[4], const float (&x1)[4],
                                            const float (&g0)[4], const float (&g1)[4], float eps,
                                            const Trig& tr, float (&o0)[4], float (&o1)[4]) {
  // x*gamma is exact in fp32; x^2 is exact, the sum rounds
  float ss = 0.f, a0[4], a1[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    ss = fmaf(x0[j], x0[j], ss);
    ss = fmaf(x1[j], x1[j], ss);
    a0[j] = x0[j] * g0[j];
    a1[j] = x1[j] * g1[j];
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float r = rsqrtf(fmaf(ss, 1.0f / kHeadDim, eps));

  // rotate-half, pair (i, i + D/2) in this lane:
  //   out_i = a_i c - a_{i+D/2} s,   out_{i+D/2} = a_{i+D/2} c + a_i s
  const float ch[4] = {tr.ch.x, tr.ch.y, tr.ch.z, tr.ch.w};
  const float cl[4] = {tr.cl.x, tr.cl.y, tr.cl.z, tr.cl.w};
  const float sh[4] = {tr.sh.x, tr.sh.y, tr.sh.z, tr.sh.w};
  const float sl[4] = {tr.sl.x, tr.sl.y, tr.sl.z, tr.sl.w};
  const uint64_t r2 = pack2(r, r);
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const uint64_t y0 = pack2(a0[j], a0[j + 1]), y1 = pack2(a1[j], a1[j + 1]);
    const uint64_t c = pack2(ch[j], ch[j + 1]), nc = pack2(-ch[j], -ch[j + 1]);
    const uint64_t c_lo = pack2(cl[j], cl[j + 1]);
    const uint64_t s = pack2(sh[j], sh[j + 1]), ns = pack2(-sh[j], -sh[j + 1]);
    const uint64_t s_lo = pack2(sl[j], sl[j + 1]), ns_lo = pack2(-sl[j], -sl[j + 1]);
    // out_i = r (a_i c - a_{i+64} s);  out_{i+64} = r (a_{i+64} c - (-a_i) s)
    unpack2(rotate2(y0, y1, c, nc, c_lo, s, ns, ns_lo, r2), o0[j], o0[j + 1]);
    unpack2(rotate2(y1, y0, c, nc, c_lo, ns, s, s_lo, r2), o1[j], o1[j + 1]);
  }
}

}  // namespace pkvqk
