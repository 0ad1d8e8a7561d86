// norm_rope.hpp -- device parts that both appends use: the angles of a token,
// and eight dimensions of a head normed and rotated.
#pragma once

#include "kv_common.hpp"

namespace trellis {

// cos and sin of position * inv_freq.  The angle is f64: a far position times
// a frequency needs more than f32's 24 bits for a fraction of a turn.
__device__ __forceinline__ void turn(int32_t position, float inv_freq, float& c, float& s) {
  double turns = (double)position * (double)inv_freq * 0.15915494309189533577;    // 1 / (2 pi)
  turns -= rint(turns);
  sincospif(2.0f * (float)turns, &s, &c);
}

// y = x / sqrt(mean x^2 + eps) * w over a head, then, over the first `rotary`
// dimensions, (a, b) -> (a cos t - b sin t, b cos t + a sin t): pairs
// (i, i + rotary / 2), or (2 i, 2 i + 1) when PAIRS.  The D / 8 lanes of a head
// call it together, each with its eight dimensions from d0 on: src and weight
// point at them, raw is what src holds, cs and sn point at the token's angles.
template <typename T, int D, bool PAIRS>
__device__ __forceinline__ void norm_rotate(u32x4v raw, const uint16_t* src, const uint16_t* weight, int d0, int rotary,
                                            float eps, const float* cs, const float* sn, float (&y)[8]) {
  constexpr int LANES = D / 8;
  const int half = rotary / 2;
  const u32x4v wr = *reinterpret_cast<const u32x4v*>(weight);
  float sum = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    y[e] = T::to_f32((uint16_t)(raw[e >> 1] >> (16 * (e & 1))));
    sum += y[e] * y[e];
  }
#pragma unroll
  for (int d = LANES / 2; d; d >>= 1) sum += __shfl_xor(sum, d);
  const float inv = 1.0f / sqrtf(sum * (1.0f / D) + eps);
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = y[e] * inv * T::to_f32((uint16_t)(wr[e >> 1] >> (16 * (e & 1))));
  if (PAIRS) {
    if (d0 < rotary) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float c = cs[(d0 + e) >> 1], s = sn[(d0 + e) >> 1];
        const float lo = y[e] * c - y[e + 1] * s, hi = y[e + 1] * c + y[e] * s;
        y[e] = lo;
        y[e + 1] = hi;
      }
    }
  } else {
    // the partner of dimension d is d +- rotary / 2, a whole number of lanes
    // away: its input and weight are read again (they are in the L1) rather
    // than sent through LDS
    if (d0 < rotary) {
      const int away = d0 < half ? half : -half, i = d0 < half ? d0 : d0 - half;
      const u32x4v pr = *reinterpret_cast<const u32x4v*>(src + away);
      const u32x4v pw = *reinterpret_cast<const u32x4v*>(weight + away);
      const float sign = d0 < half ? -1.0f : 1.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float other = T::to_f32((uint16_t)(pr[e >> 1] >> (16 * (e & 1)))) * inv *
                            T::to_f32((uint16_t)(pw[e >> 1] >> (16 * (e & 1))));
        y[e] = y[e] * cs[i + e] + sign * (other * sn[i + e]);
      }
    }
  }
}

}  // namespace trellis
