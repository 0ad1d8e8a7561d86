// qk_norm_rope.hip -- RMS norm of every query and key head, rotation by
// position, and the append of keys and values to the paged cache, one pass.
#include "internal.hpp"
#include "kv_common.hpp"

namespace trellis {
namespace {

constexpr int kThreads = 256;

// y = x / sqrt(mean x^2 + eps) * w over a head, then, over the first `rotary`
// dimensions, (a, b) -> (a cos t - b sin t, b cos t + a sin t) with
// t = position * inv_freq[i]: pairs (i, i + rotary / 2), or (2 i, 2 i + 1) when
// interleaved.  Everything is f32 and rounded once; the angle is f64, since a
// far position times a frequency needs more than f32's 24 bits for a
// fraction of a turn.
//
// One workgroup per token: the angles are computed once for all heads (into
// LDS); D / 8 lanes own a head, eight dimensions each.
template <typename T, int D, bool PAIRS>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(QkNormRopeArgs a) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  __shared__ float s_cos[D / 2], s_sin[D / 2];
  const int64_t tok = blockIdx.x;
  const int tid = threadIdx.x, grp = tid / LANES, l = tid % LANES;
  const int half = a.rotary / 2;
  const int pos = a.positions[tok];
  const int slot = a.slots[tok];
  for (int i = tid; i < half; i += kThreads) {
    double turns = (double)pos * (double)a.inv_freq[i] * 0.15915494309189533577;    // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(2.0f * (float)turns, &s, &c);
    s_cos[i] = c;
    s_sin[i] = s;
  }
  __syncthreads();
  const int P = 1 << a.page_log2, off = slot & (P - 1);
  const uint32_t page = (uint32_t)(slot >> a.page_log2);
  const bool cached = slot >= 0 && page < a.pages;
  const int heads = a.heads_q + 2 * a.heads_kv;
  for (int h = grp; h < heads; h += GROUPS) {
    const bool is_q = h < a.heads_q, is_v = h >= a.heads_q + a.heads_kv;
    const int hh = is_q ? h : is_v ? h - a.heads_q - a.heads_kv : h - a.heads_q;
    const uint16_t* src = is_q ? a.q + tok * a.q_stride : is_v ? a.v + tok * a.v_stride : a.k + tok * a.k_stride;
    const u32x4v raw = *reinterpret_cast<const u32x4v*>(src + hh * D + l * 8);
    const int64_t head_base = ((int64_t)page * a.heads_kv + hh) * ((int64_t)D << a.page_log2);
    if (is_v) {
      if (cached) {
        uint16_t* dst = a.v_cache + head_base + (int64_t)(off >> 3) * D * 8 + l * 64 + (off & 7);
#pragma unroll
        for (int e = 0; e < 8; ++e) dst[e * 8] = (uint16_t)(raw[e >> 1] >> (16 * (e & 1)));
      }
      continue;
    }
    const u32x4v wr = *reinterpret_cast<const u32x4v*>((is_q ? a.q_weight : a.k_weight) + l * 8);
    float x[8], sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = T::to_f32((uint16_t)(raw[e >> 1] >> (16 * (e & 1))));
      sum += x[e] * x[e];
    }
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) sum += __shfl_xor(sum, d);
    const float inv = 1.0f / sqrtf(sum * (1.0f / D) + a.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * T::to_f32((uint16_t)(wr[e >> 1] >> (16 * (e & 1))));
    const int d0 = l * 8;
    if (PAIRS) {
      if (d0 < a.rotary) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float c = s_cos[(d0 + e) >> 1], s = s_sin[(d0 + e) >> 1];
          const float lo = x[e] * c - x[e + 1] * s, hi = x[e + 1] * c + x[e] * s;
          x[e] = lo;
          x[e + 1] = hi;
        }
      }
    } else {
      // the partner of dimension d is d +- rotary / 2: a whole number of lanes away
      const int away = half >> 3;
      const bool low = d0 < half, in = d0 < a.rotary;
      const int from = (int)__lane_id() + (in ? (low ? away : -away) : 0);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = __shfl(x[e], from);
        if (in) {
          const int i = (low ? d0 : d0 - half) + e;
          x[e] = low ? x[e] * s_cos[i] - y * s_sin[i] : x[e] * s_cos[i] + y * s_sin[i];
        }
      }
    }
    u32x4v res;
#pragma unroll
    for (int w = 0; w < 4; ++w) res[w] = T::pack(x[2 * w], x[2 * w + 1]);
    if (is_q)
      *reinterpret_cast<u32x4v*>(a.out + (tok * a.heads_q + hh) * D + d0) = res;
    else if (cached)
      *reinterpret_cast<u32x4v*>(a.k_cache + head_base + ((int64_t)l * P + off) * 8) = res;
  }
}

template <typename T, int D>
hipError_t launch_pairs(const QkNormRopeArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)a.tokens);
  if (a.interleaved)
    qk_norm_rope_kernel<T, D, true><<<grid, kThreads, 0, stream>>>(a);
  else
    qk_norm_rope_kernel<T, D, false><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_dim(const QkNormRopeArgs& a, hipStream_t stream) {
  switch (a.head_dim) {
    case 64: return launch_pairs<T, 64>(a, stream);
    case 128: return launch_pairs<T, 128>(a, stream);
    default: return launch_pairs<T, 256>(a, stream);
  }
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkNormRopeArgs& a, hipStream_t stream) {
  return a.fp16 ? launch_dim<F16>(a, stream) : launch_dim<Bf16>(a, stream);
}

}  // namespace trellis
