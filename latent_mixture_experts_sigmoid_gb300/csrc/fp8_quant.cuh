// The e4m3 quantisation rule, shared by the kernels that apply it: per block,
//   a = max(max |x|, 2^-100),  scale = a / 448,  code = e4m3(x * (448 / a)),
// in fp32 and each operation rounded once.
#pragma once

#include <stdint.h>

namespace lmoe {

constexpr float kE4m3Max = 448.0f;
constexpr float kTinyAmax = 7.888609052210118e-31f;   // 2^-100: keeps 448 / a finite

// two fp32 -> two e4m3 (round to nearest even, saturating; NaN stays NaN)
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  return pack_e4m3x2(a, b) | (pack_e4m3x2(c, d) << 16);
}

// Bits of |x|: their order is the values', NaN above infinity, so that a maximum
// over them keeps a NaN.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

struct BlockScale {
  float scale, inv;
};
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {
  const float a = __uint_as_float(max(amax_bits, __float_as_uint(kTinyAmax)));
  return {__fdiv_rn(a, kE4m3Max), __fdiv_rn(kE4m3Max, a)};
}

}  // namespace lmoe
