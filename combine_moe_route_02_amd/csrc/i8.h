// Symmetric 8-bit integer codes of a row, shared by the quantisation kernels and the few-rows products:
// scale = amax / 127 and code = RNE(v * (127 / amax)) in [-127, 127], one FP32 rounding per step.
#pragma once
#include "common.h"

namespace moe {

struct RowScale { float inv, scale; };
MOE_DEV RowScale row_scale(uint32_t magnitude) {
  if (magnitude >= 0x7f800000u) return {0.f, __uint_as_float(0x7fc00000u)};
  if (magnitude == 0) return {0.f, 1.0f};
  const float amax = __uint_as_float(magnitude);
  // below 127 / FLT_MAX the multiplier overflows: such a row is a row of zeros
  const float inv = 127.0f / amax;
  return inv <= 3.402823466e38f ? RowScale{inv, amax / 127.0f} : RowScale{0.f, 1.0f};
}

// Codes of four values. Each product is rounded to FP32 and then to the nearest integer, halves to even, by
// adding 1.5 * 2^23: the sum's last bits are the integer in two's complement, so three byte permutes
// pack four codes (rounding, converting, clamping and shifting each value takes three times the
// instructions). |v| <= amax keeps the rounded product within 127. The two steps must not be fused: a
// product that FP32 rounds onto a half belongs to the even code. inv == 0: codes 0, whatever the values
// are.
MOE_DEV uint32_t codes4(float a, float b, float c, float d, float inv) {
#pragma clang fp contract(off)
  constexpr float kShift = 12582912.0f;
  const float p = a * inv, q = b * inv, r = c * inv, s = d * inv;
  const uint32_t i = __float_as_uint(p + kShift), j = __float_as_uint(q + kShift);
  const uint32_t k = __float_as_uint(r + kShift), l = __float_as_uint(s + kShift);
  const uint32_t lo = __builtin_amdgcn_perm(j, i, 0x0c0c0400), hi = __builtin_amdgcn_perm(l, k, 0x04000c0c);
  return inv == 0.f ? 0u : lo | hi;
}
MOE_DEV uint2 codes8(const u32x4& v, float inv) {
  return make_uint2(codes4(bf2f(v.x & 0xffff), bf2f(v.x >> 16), bf2f(v.y & 0xffff), bf2f(v.y >> 16), inv),
                    codes4(bf2f(v.z & 0xffff), bf2f(v.z >> 16), bf2f(v.w & 0xffff), bf2f(v.w >> 16), inv));
}

// Rows of yd between the experts and combine: 16 bits of sign, 7 exponent bits (bias 63) and 8 mantissa bits. With
// BF16 there, its rounding and the output's are two of the same size in a row (sqrt(2) of one); with one bit more
// the first is half (sqrt(1.25) = 1.12 of one). That holds where the gates spread the values; times a gate of 1 (k = 1)
// or another power of two, codes with the last bit set are ties of the output's rounding, off by half a step whichever
// way they go: sqrt(1.75) = 1.32 of one, where BF16 rows would have been exact. Magnitudes from 2^-62, gradually less
// to 2^-70, to just under 2^65; what is larger, or not finite, is code 0x7fff and comes out as NaN. The encoder takes
// values times 2^-64, so that the exponent's top bit is clear and the code is FP32's upper half without it; halves round
// away from zero. The unit multiplies the integer sum: ahead of it, the product of two small scales would become
// subnormal and lose bits that a long sum brings back into the format's range.
constexpr float kYdUnit = 0x1p-64f;
MOE_DEV uint32_t pack_yd(float lo, float hi) {
  const uint32_t a = __float_as_uint(lo), b = __float_as_uint(hi);
  const uint32_t u = min(a << 1, 0x7ffeffffu) + 0x8000u, v = min(b << 1, 0x7ffeffffu) + 0x8000u;
  return __builtin_amdgcn_perm(v | (b & 0x80000000u), u | (a & 0x80000000u), 0x07060302);
}
MOE_DEV float unpack_yd(uint32_t high) {  // the code in the upper half
  const uint32_t m = high & 0x7fff0000u;
  const float v = __uint_as_float((high & 0x80000000u) | (m >> 1)) * 0x1p64f;
  return m == 0x7fff0000u ? __uint_as_float(0x7fc00000u) : v;
}

}  // namespace moe
