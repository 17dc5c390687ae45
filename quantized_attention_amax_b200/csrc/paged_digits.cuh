// paged_digits.cuh -- 16-bit and fp32 values as sums of three 8-bit digits, so that the tensor cores can
// multiply them with 8-bit cache codes as they are (tcgen05 kind::i8 or kind::f8f6f4, no conversion of
// the codes).  Three MMA columns then stand for one row, and the products add up in 32 bits:
//   int8 caches:  v = d2 2^16 + d1 2^8 + d0, signed digits, for a query row scaled by a power of two so that
//                 |v| < 2^22: bf16 values down to 2^-14 of the row's largest are exact, smaller ones are
//                 off by at most 2^-22 of it.  Probabilities, held against a unit below twice the largest of their
//                 key tile, are 24-bit integers, unsigned digits.
//   E4M3 caches:  v = t1 + t2 / 16 + t3 / 256, each digit the E4M3 rounding of 16 times what the digits
//                 before leave: |v| < 256, relative error 2^-12, and 2^-18 absolute (2^-25 of the row's, or the key
//                 tile's, largest).
//                 A bf16 value within 2^-14 of the row's largest is exact after two.
#pragma once

#include <cuda_runtime.h>
#include <math.h>

#include "attn_common.cuh"

namespace faq {
namespace paged {

__device__ __forceinline__ uint32_t e4m3_of(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(x));
  return (uint32_t)r & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const uint32_t h2 = attn::e4m3x2_to_h2((uint16_t)code);
  return __low2float(*reinterpret_cast<const __half2*>(&h2));
}

// Digits of a query value x whose row is scaled by 2^e = sc (int8: |x sc| < 2^22, E4M3: < 256); d[0]
// carries the most.
template <bool FP8>
__device__ __forceinline__ void q_digits(float x, float sc, uint32_t (&d)[3]) {
  if (FP8) {
    float v = x * sc;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      d[k] = e4m3_of(v);
      v = (v - e4m3_value(d[k])) * 16.0f;
    }
  } else {
    const int v = __float2int_rn(x * sc);
    const int d0 = (int)(int8_t)(v & 0xFF);
    const int v1 = (v - d0) >> 8;
    const int d1 = (int)(int8_t)(v1 & 0xFF);
    d[0] = (uint32_t)((v1 - d1) >> 8) & 0xFFu;
    d[1] = (uint32_t)d1 & 0xFFu;
    d[2] = (uint32_t)d0 & 0xFFu;
  }
}

// Digits of a probability w in [0, 1]: int8 round(w 2^24) (at most 2^24 - 1), E4M3 of 256 w.
template <bool FP8>
__device__ __forceinline__ void p_digits(float w, uint32_t (&d)[3]) {
  if (FP8) {
    float v = w * 256.0f;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      d[k] = e4m3_of(v);
      if (k < 2) v = (v - e4m3_value(d[k])) * 16.0f;
    }
  } else {
    const uint32_t v = min(__float2uint_rn(w * 16777216.0f), 16777215u);
    d[0] = v >> 16;
    d[1] = (v >> 8) & 0xFFu;
    d[2] = v & 0xFFu;
  }
}

// The sum that three accumulators (d[0]'s, d[1]'s, d[2]'s) stand for.  int8: up to 2^22 in magnitude each,
// so the lower two join exactly in 32 bits.
template <bool FP8>
__device__ __forceinline__ float join_digits(uint32_t a0, uint32_t a1, uint32_t a2) {
  if (FP8)
    return fmaf(__uint_as_float(a2), 1.0f / 256.0f, fmaf(__uint_as_float(a1), 1.0f / 16.0f, __uint_as_float(a0)));
  return fmaf((float)(int)a0, 65536.0f, (float)((int)a1 * 256 + (int)a2));
}

// What one unit of join_digits is worth: of a query row scaled by sc, 1 / sc; of a probability, this.
template <bool FP8>
constexpr float kPUnit = FP8 ? 1.0f / 256.0f : 1.0f / 16777216.0f;

// The power of two that scales a query row of largest magnitude m for its digits, and its inverse (zero
// rows: 1; a row with an infinity or NaN: NaN, so that its scores are).
template <bool FP8>
__device__ __forceinline__ float digit_scale(float m, float& inv) {
  constexpr int TOP = FP8 ? 7 : 21;  // m comes to lie in [2^TOP, 2^(TOP + 1))
  const int E = (int)((__float_as_uint(m) >> 23) & 0xFFu);
  if (!(m < INFINITY)) {
    inv = __uint_as_float(0x7FC00000u);
    return 0.0f;
  }
  if (m == 0.0f) {
    inv = 1.0f;
    return 1.0f;
  }
  const int e = max(E, TOP + 2);
  inv = __uint_as_float((uint32_t)(e - TOP) << 23);           // 2^(e - 127 - TOP)
  return __uint_as_float((uint32_t)(254 - (e - TOP)) << 23);  // 2^(TOP + 127 - e)
}

}  // namespace paged
}  // namespace faq
