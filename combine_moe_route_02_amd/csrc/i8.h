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

// inv == 0: codes 0, whatever the values are
MOE_DEV uint32_t codes4(float a, float b, float c, float d, float inv) {
  if (inv == 0.f) return 0;
  const int i = (int)rintf(a * inv), j = (int)rintf(b * inv), k = (int)rintf(c * inv), l = (int)rintf(d * inv);
  auto cl = [](int v) { return (uint32_t)(max(-127, min(127, v)) & 0xff); };
  return cl(i) | (cl(j) << 8) | (cl(k) << 16) | (cl(l) << 24);
}
MOE_DEV uint2 codes8(const u32x4& v, float inv) {
  return make_uint2(codes4(bf2f(v.x & 0xffff), bf2f(v.x >> 16), bf2f(v.y & 0xffff), bf2f(v.y >> 16), inv),
                    codes4(bf2f(v.z & 0xffff), bf2f(v.z >> 16), bf2f(v.w & 0xffff), bf2f(v.w >> 16), inv));
}

}  // namespace moe
