// codes.cuh -- the element and scale decisions of the quantised row formats,
// shared by the contiguous writers (quant.cuh) and the paged ones (rows.cuh).
#pragma once
#include <cstdint>

#include "params.h"
#include "ptx.cuh"

namespace mla {

// two fp32 -> two e4m3 bytes, `lo` in the low byte
MLA_DEV uint16_t e4m3x2_rn_sat(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
MLA_DEV uint32_t e4m3x4_rn_sat(float a, float b, float c, float d) {
  return (uint32_t)e4m3x2_rn_sat(a, b) | ((uint32_t)e4m3x2_rn_sat(c, d) << 16);
}

// scale of a block whose largest magnitude is amax: fp32(amax / 448), 1 for
// zeros; the quotient by the corrected reciprocal of e4m3_codes16, equal to the
// division for every fp32 significand
MLA_DEV float e4m3_scale(float amax) {
  if (amax >= 0x1p-60f && amax < 0x1p127f) {
    constexpr float r = 1.f / 448.f;
    const float q = __fmul_rn(amax, r);
    return __fmaf_rn(__fmaf_rn(q, -448.f, amax), r, q);
  }
  return amax == 0.f ? 1.f : __fdiv_rn(amax, 448.f);
}

// Sixteen values over their block's scale, as e4m3 codes (value i in byte i).
//
// A quotient x / scale is formed as q = x * r, r = 1 / scale rounded to nearest,
// corrected by its remainder: q + (x - q * scale) * r, each step one fused
// operation (after P. Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990). Two roundings put q up to 1.5 units
// off, where the correction may miss the rounded quotient by one fp32 step: only
// if x / scale lies within 2^-45.9 of itself of the middle between two fp32
// numbers. A code can change there only beside one of the five-bit numbers at
// which e4m3's rounding turns, and few pairs fit both: all of them give the
// division's code (the host tests derive and run through them). For scale >=
// 2^-60 only an |x| below 2^-102 could underflow a remainder, and its quotient is
// below 2^-42, zero in e4m3; smaller scales, and an infinite one, are divided by.
// On packed pairs that is 1.5 operations a value and one for the sign of a zero,
// where a division takes some ten.
MLA_DEV void e4m3_codes16(const float* x, float scale, uint32_t* w) {
  if (scale >= 0x1p-60f && scale < 0x1p127f) {
    const float inv = __frcp_rn(scale);
    const uint64_t r = f2_pack(inv, inv), m = f2_pack(-scale, -scale);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float y[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float lo = x[4 * k + 2 * j], hi = x[4 * k + 2 * j + 1];
        const uint64_t v = f2_pack(lo, hi), q = f2_mul(v, r);
        const float2 c = f2_unpack(f2_fma(f2_fma(q, m, v), r, q));
        y[2 * j] = __uint_as_float(__float_as_uint(c.x) | (__float_as_uint(lo) & 0x80000000u));
        y[2 * j + 1] = __uint_as_float(__float_as_uint(c.y) | (__float_as_uint(hi) & 0x80000000u));
      }
      w[k] = e4m3x4_rn_sat(y[0], y[1], y[2], y[3]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = e4m3x4_rn_sat(__fdiv_rn(x[4 * k], scale), __fdiv_rn(x[4 * k + 1], scale), __fdiv_rn(x[4 * k + 2], scale),
                           __fdiv_rn(x[4 * k + 3], scale));
  }
}
MLA_DEV float amax16(const float* x) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int k = 1; k < 15; k += 2) m = max3(m, fabsf(x[k]), fabsf(x[k + 1]));
  return fmaxf(m, fabsf(x[15]));
}

// UE8M0 exponent of a block: the smallest integer k >= -127 with
// 448 * 2^k >= amax, found from amax's fp32 fields: amax = f * 2^e, f in
// [1, 2), gives k = e - 8 when f <= 1.75 (448 = 1.75 * 2^8) and e - 7 above.
MLA_DEV int ue8m0_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e_field = (int)(bits >> 23);  // amax >= 0; 0 for zero and fp32 subnormals
  int k = -127;                           // zero and subnormal blocks: 448 * 2^-127 covers them
  if (e_field > 0) {
    k = (e_field - 127) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    k = k < -127 ? -127 : k;
  }
  return k;
}
// 2^-k for k in [-127, 120]: a normal fp32 value, so x * 2^-k is exact
MLA_DEV float exp2_neg(int k) { return __uint_as_float((uint32_t)(127 - k) << 23); }

// value of a non-negative e4m3 code (0x00 .. 0x7E) as fp32, from its fields
MLA_DEV float e4m3_pos_value(uint32_t c) {
  const uint32_t e = c >> 3, m = c & 7u;
  return e == 0 ? (float)m * 0x1p-9f : __uint_as_float(((e + 120u) << 23) | (m << 20));
}

// The sixteen values of one block of a 288-byte row -> its e4m3 scale code and
// the e2m1 codes (value i in nibble i of lo, value 8 + i in nibble i of hi).
// The scale v is the smallest non-negative e4m3 value with 6 v >= amax (448
// when none is large enough); the code is the nearest e2m1 magnitude of
// |x| / v, ties to the even code, with the sign of x. The decision is taken
// against the midpoints of the e2m1 magnitudes times v (at most 7 significant
// bits: exact in fp32), so no division rounds.
MLA_DEV uint32_t fp4_block(const float* x, uint32_t& lo, uint32_t& hi) {
  // midpoints between consecutive e2m1 magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6
  const float mids[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.0f};
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(x[k]));
  // a first guess from the rounded quotient, then corrected by exact tests
  // (6 v is exact: at most 6 significant bits)
  uint32_t c = e4m3x2_rn_sat(amax / 6.0f, 0.f) & 0x7Fu;
  if (c > 0x7Eu) c = 0x7Eu;
  for (int it = 0; it < 4 && c < 0x7Eu && 6.0f * e4m3_pos_value(c) < amax; ++it) ++c;
  for (int it = 0; it < 4 && c > 0u && 6.0f * e4m3_pos_value(c - 1u) >= amax; ++it) --c;
  const float v = e4m3_pos_value(c);
  float t[7];
#pragma unroll
  for (int j = 0; j < 7; ++j) t[j] = mids[j] * v;
  lo = 0;
  hi = 0;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float a = fabsf(x[k]);
    uint32_t mag = 0;
#pragma unroll
    for (int j = 0; j < 7; ++j) mag += (a > t[j] || (a == t[j] && (j & 1))) ? 1u : 0u;
    if (v == 0.f) mag = 0;
    const uint32_t code = mag | ((__float_as_uint(x[k]) >> 31) << 3);
    if (k < 8) lo |= code << (4 * k);
    else hi |= code << (4 * (k - 8));
  }
  return c;
}

}  // namespace mla
