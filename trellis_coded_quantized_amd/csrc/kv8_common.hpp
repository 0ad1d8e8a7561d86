// kv8_common.hpp -- the 8-bit cache's numbers: e4m3 codes under the
// power-of-two scale of their block, a byte b that stands for 2^(b - 127).
#pragma once

#include "kv_common.hpp"

namespace trellis {

// The smallest b of 1..254 with 448 * 2^(b - 127) >= x, x a finite magnitude
// given by its bits: 448 is 1.75 * 2^8, so a significand above 1.75 needs one
// more (subnormal x: 1).
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits) {
  const int b = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(b, 1);
}

// 2^(127 - b), what a magnitude is multiplied with to become a code.  2^-127
// stands for 2^-127 and 2^-128, where no code but 0 comes out.
__device__ __forceinline__ float inverse_scale(uint32_t b) {
  return __builtin_bit_cast(float, b >= 254 ? 0x00400000u : (254u - b) << 23);
}

// four codes, rounded to the nearest (ties to even); |x| <= 448 or NaN
__device__ __forceinline__ uint32_t codes4(float x, float y, float z, float w) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x, y, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(z, w, lo, true);
}

// Codes of one scale rounded to those of another, b >= old.
__device__ __forceinline__ uint32_t rescaled4(uint32_t codes, uint32_t old, uint32_t b) {
  const float by = __builtin_bit_cast(float, (uint32_t)max(127 - (int)(b - old), 0) << 23);
  const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes, by, false);
  const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes, by, true);
  return codes4(lo[0], lo[1], hi[0], hi[1]);
}

__device__ __forceinline__ u32x4v rescaled(u32x4v g, uint32_t old, uint32_t b) {
  return u32x4v{rescaled4(g[0], old, b), rescaled4(g[1], old, b), rescaled4(g[2], old, b), rescaled4(g[3], old, b)};
}

}  // namespace trellis
