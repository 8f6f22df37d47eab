// 8-bit codes (e4m3 or int8) as f16 operands of the matrix instructions, and
// the scales that go with them: shared by the attention kernels over an 8-bit
// cache.  Every code is exact in f16 (e4m3 has 4 significant bits and the range
// 2^-9 .. 448, int8 7 bits), so the products q . code carry no rounding of the
// cache; the scales stay in fp32 outside the products.
#pragma once

#include <cuda_fp16.h>

#include "device_common.cuh"
#include "kernels.h"

namespace pkvqk {

// Two f16 values from two e4m3 codes, the low byte's in the low half.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
  return r;
}

// int8 by the f16 value 1024 + u of the bit pattern 0x6400 | u, u = code + 128,
// and an exact subtraction of 1152; sel picks the two bytes (with 0x64 from the
// constant's byte 4 above each).
__device__ __forceinline__ uint32_t int8x2_to_f16x2(uint32_t flipped, uint32_t sel) {
  const uint32_t u = __byte_perm(flipped, 0x64646464u, sel);
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 2^x on the SFU (relative error ~2^-22; -inf -> +0): what it gives is rounded to
// f16 or summed.
__device__ __forceinline__ float ex2_sfu(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Bytes (0, 1) -> lo, bytes (2, 3) -> hi.
template <int kFormat>
__device__ __forceinline__ void codes_adjacent(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (kFormat == kFormatE4m3) {
    lo = e4m3x2_to_f16x2(static_cast<uint16_t>(w));
    hi = e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
  } else {
    const uint32_t f = w ^ 0x80808080u;
    lo = int8x2_to_f16x2(f, 0x4140u);
    hi = int8x2_to_f16x2(f, 0x4342u);
  }
}

// Bytes (0, 2) -> even, bytes (1, 3) -> odd.
template <int kFormat>
__device__ __forceinline__ void codes_alternate(uint32_t w, uint32_t& even, uint32_t& odd) {
  if (kFormat == kFormatE4m3) {
    const uint32_t s = __byte_perm(w, 0u, 0x3120u);
    even = e4m3x2_to_f16x2(static_cast<uint16_t>(s));
    odd = e4m3x2_to_f16x2(static_cast<uint16_t>(s >> 16));
  } else {
    const uint32_t f = w ^ 0x80808080u;
    even = int8x2_to_f16x2(f, 0x4240u);
    odd = int8x2_to_f16x2(f, 0x4341u);
  }
}

// A stored scale as the kernels use it: [2^-64, 2^63]; zero, negative and NaN
// count as 2^-64.
__device__ __forceinline__ float usable_scale(float s) {
  const float lo = __int_as_float((127 + kScaleMinExp) << 23);
  const float hi = __int_as_float((127 + kScaleMaxExp) << 23);
  return fminf(fmaxf(s, lo), hi);
}

// bf16 rows become f16 operands after a multiplication by 2^k that brings the
// row's largest magnitude to [2^14, 2^15): exact for every value within 2^-28
// of it.  2^k from that magnitude (0, infinite or NaN: 1), and 2^-k.  k <= 72 keeps
// 2^-k times any softmax scale above 2^-13 and any K scale from becoming 0; in rows
// below 2^-57 what is under 2^-97 is dropped, 2^-18 of a score at the largest K.
__device__ __forceinline__ float q_row_scale(float amax, float& inverse) {
  const int e = static_cast<int>(__float_as_uint(amax) >> 23);   // biased
  int k = (amax > 0.f && e < 255) ? 14 + 127 - e : 0;
  k = k > 72 ? 72 : k;
  inverse = __int_as_float((127 - k) << 23);
  return __int_as_float((127 + k) << 23);
}

}  // namespace pkvqk
