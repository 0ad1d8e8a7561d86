// qk_norm_rope_kv8.hip -- RMS norm of every query and key head, rotation by
// position, and the append of keys and values to the cache held in 8 bits.
#include "internal.hpp"
#include "kv8_common.hpp"
#include "norm_rope.hpp"

namespace trellis {
namespace {

constexpr int kThreads = 256;
constexpr int TB = 8;             // tokens of a workgroup that has queries

// The largest number of the 16-bit type with 4 significant bits: a larger one
// could not come back from e4m3 and a scale.
template <typename T>
__device__ __forceinline__ float type_top() {
  return __builtin_bit_cast(float, sizeof(T) && T::kExp == 0x7F80u ? 0x7F700000u : 0x47700000u);   // 1.875 2^127, 61440
}

// Infinities become NaN, magnitudes end at the type's top; returns the largest
// finite one.
template <typename T>
__device__ __forceinline__ float tame(float (&y)[8]) {
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float m = fabsf(y[e]);
    const bool finite = m < INFINITY;
    const float c = fminf(m, type_top<T>());
    y[e] = finite ? copysignf(c, y[e]) : NAN;
    top = fmaxf(top, finite ? c : 0.0f);
  }
  return top;
}

// Queries.  As in the 16-bit append: a workgroup takes TB tokens and a share of
// the heads, D / 8 lanes a head.
template <typename T, int D, bool PAIRS>
__device__ void queries(const QkNormRope8Args& a, int64_t first, int share, int shares, float (*s_cos)[D / 2],
                        float (*s_sin)[D / 2]) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  const int tokens = (int)min((int64_t)TB, a.tokens - first), half = a.rotary / 2;
  const int tid = threadIdx.x, grp = tid / LANES, d0 = tid % LANES * 8;
  const int h0 = (int)((int64_t)a.heads_q * share / shares), h1 = (int)((int64_t)a.heads_q * (share + 1) / shares);
  for (int x = tid; x < tokens * half; x += kThreads) {
    const int t = x / half, i = x - t * half;
    turn(a.positions[first + t], a.inv_freq[i], s_cos[t][i], s_sin[t][i]);
  }
  __syncthreads();
  for (int x = grp; x < (h1 - h0) * TB; x += GROUPS) {
    const int h = h0 + x / TB, t = x % TB;
    if (t >= tokens) continue;
    float y[8];
    norm_rotate<T, D, PAIRS>(a.q + (first + t) * a.q_stride + h * D + d0, a.q_weight + d0, d0, a.rotary, a.eps, s_cos[t],
                             s_sin[t], y);
    u32x4v res;
#pragma unroll
    for (int w = 0; w < 4; ++w) res[w] = T::pack(y[2 * w], y[2 * w + 1]);
    *reinterpret_cast<u32x4v*>(a.out + ((first + t) * a.heads_q + h) * D + d0) = res;
  }
}

// Keys and values.  A block of 16 slots has one owner, so that its scale and
// its rows change together: the workgroup that has the first of the block's
// tokens in its window of the list (a run; at most 16 tokens).  Heads of a run
// are taken UNITS / n at a time, one (head, token) to D / 8 lanes: values in
// registers, the block's largest magnitude through LDS, codes through LDS into
// the cache's order, so that a full block leaves as whole granules.
template <typename T, int D, bool PAIRS>
__device__ void keys_values(const QkNormRope8Args& a, int64_t first, int window, int share, int shares,
                            float (*s_cos)[D / 2], float (*s_sin)[D / 2]) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES, PER = 2, UNITS = GROUPS * PER;
  __shared__ __align__(16) uint8_t s_code[2][UNITS * D];     // keys [head][D/16][token][16], values [head][token][D]
  __shared__ uint32_t s_top[2][UNITS], s_old[2][UNITS], s_new[2][UNITS];
  __shared__ int s_off[16];
  const int tid = threadIdx.x, lane = tid & 63, grp = tid / LANES, l = tid % LANES, d0 = l * 8;
  const int half = a.rotary / 2, P = 1 << a.page_log2;
  const int v0 = (int)((int64_t)a.heads_kv * share / shares), v1 = (int)((int64_t)a.heads_kv * (share + 1) / shares);

  // lane j of every wave looks at token first - 1 + j: which begin a run, which go on with one
  const int64_t tok = first - 1 + lane;
  const int slot = tok >= 0 && tok < a.tokens ? a.slots[tok] : -1;
  const bool cached = slot >= 0 && (uint32_t)(slot >> a.page_log2) < a.pages;
  const int block = cached ? slot >> 4 : -1;
  const int before = __shfl_up(block, 1);
  const uint64_t goes_on = __ballot(cached && lane > 0 && block == before);
  uint64_t begins = __ballot(cached && lane > 0 && lane <= window && block != before);

  for (bool again = false; begins; begins &= begins - 1, again = true) {
    const int j = __builtin_ctzll(begins);
    const int n = min(16, 1 + __builtin_ctzll(~(goes_on >> (j + 1))));
    const int64_t t0 = first - 1 + j;
    const int slot0 = __builtin_amdgcn_readlane(slot, j);
    const int64_t page = slot0 >> a.page_log2;
    const int in_page = (slot0 & (P - 1)) >> 4;              // the block
    uint32_t mine = lane >= j && lane < j + n ? 1u << (slot & 15) : 0u;
#pragma unroll
    for (int d = 32; d; d >>= 1) mine |= __shfl_xor(mine, d);
    const bool anew = mine & 1u;
    if (again) __syncthreads();                              // the run before is done with LDS
    if (tid >= j && tid < j + n) s_off[tid - j] = slot & 15;
    for (int x = tid; x < n * half; x += kThreads) {
      const int t = x / half, i = x - t * half;
      turn(a.positions[t0 + t], a.inv_freq[i], s_cos[t][i], s_sin[t][i]);
    }
    const int batch = min(UNITS / n, v1 - v0);
    for (int hb = v0; hb < v1; hb += batch) {
      const int heads = min(batch, v1 - hb), units = heads * n;
      // scales of this batch's blocks: keys at even threads, values at odd ones
      uint8_t* const scale = (tid & 1 ? a.v_scale : a.k_scale) +
                             (((page * a.heads_kv + hb + (tid >> 1)) << a.page_log2) >> 4) + in_page;
      if (hb != v0) __syncthreads();
      if (tid < 2 * heads) {
        s_top[tid & 1][tid >> 1] = 0;
        s_old[tid & 1][tid >> 1] = anew ? 0u : *scale;
      }
      __syncthreads();
      float yk[PER][8], yv[PER][8];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int u = grp + i * GROUPS;
        if (u >= units) continue;
        const int h = u / n, r = u - h * n;
        const uint16_t* vs = a.v + (t0 + r) * a.v_stride + (hb + h) * D + d0;
        const u32x4v raw = *reinterpret_cast<const u32x4v*>(vs);
        norm_rotate<T, D, PAIRS>(a.k + (t0 + r) * a.k_stride + (hb + h) * D + d0, a.k_weight + d0, d0, a.rotary, a.eps,
                                 s_cos[r], s_sin[r], yk[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) yv[i][e] = T::to_f32((uint16_t)(raw[e >> 1] >> (16 * (e & 1))));
        float kt = tame<T>(yk[i]), vt = tame<T>(yv[i]);
#pragma unroll
        for (int d = LANES / 2; d; d >>= 1) {
          kt = fmaxf(kt, __shfl_xor(kt, d));
          vt = fmaxf(vt, __shfl_xor(vt, d));
        }
        if (l == 0) {                                        // magnitudes order as their bits
          atomicMax(&s_top[0][h], __builtin_bit_cast(uint32_t, kt));
          atomicMax(&s_top[1][h], __builtin_bit_cast(uint32_t, vt));
        }
      }
      __syncthreads();
      if (tid < 2 * heads) {
        const uint32_t old = s_old[tid & 1][tid >> 1], now = max(old, scale_byte(s_top[tid & 1][tid >> 1]));
        s_new[tid & 1][tid >> 1] = now;
        if (anew || now != old) *scale = (uint8_t)now;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int u = grp + i * GROUPS;
        if (u >= units) continue;
        const int h = u / n, r = u - h * n;
        const float ki = inverse_scale(s_new[0][h]), vi = inverse_scale(s_new[1][h]);
        *reinterpret_cast<u32x2v*>(&s_code[0][((h * (D / 16) + (l >> 1)) * n + r) * 16 + (l & 1) * 8]) =
            u32x2v{codes4(yk[i][0] * ki, yk[i][1] * ki, yk[i][2] * ki, yk[i][3] * ki),
                   codes4(yk[i][4] * ki, yk[i][5] * ki, yk[i][6] * ki, yk[i][7] * ki)};
        *reinterpret_cast<u32x2v*>(&s_code[1][u * D + d0]) =
            u32x2v{codes4(yv[i][0] * vi, yv[i][1] * vi, yv[i][2] * vi, yv[i][3] * vi),
                   codes4(yv[i][4] * vi, yv[i][5] * vi, yv[i][6] * vi, yv[i][7] * vi)};
      }
      __syncthreads();
      uint8_t* const kd = a.k8 + ((page * a.heads_kv + hb) * D << a.page_log2) + in_page * 256;
      uint8_t* const vd = a.v8 + ((page * a.heads_kv + hb) * D << a.page_log2) + in_page * D * 16;
      const int64_t head = (int64_t)D << a.page_log2;
      // keys: new tokens, then the block's others where its scale grew
      for (int x = tid; x < units * (D / 16); x += kThreads) {
        const int r = x % n, g = x / n % (D / 16), h = x / (n * (D / 16));
        *reinterpret_cast<u32x4v*>(kd + h * head + g * P * 16 + s_off[r] * 16) =
            *reinterpret_cast<const u32x4v*>(&s_code[0][x * 16]);
      }
      if (!anew) {
        for (int x = tid; x < heads * D; x += kThreads) {
          const int r = x & 15, g = (x >> 4) % (D / 16), h = x / D;
          if (s_new[0][h] == s_old[0][h] || (mine >> r) & 1) continue;
          u32x4v* at = reinterpret_cast<u32x4v*>(kd + h * head + g * P * 16 + r * 16);
          *at = rescaled(*at, s_old[0][h], s_new[0][h]);
        }
      }
      // values: a granule is the block's 16 tokens of one dimension
      for (int x = tid; x < heads * D; x += kThreads) {
        const int d = x % D, h = x / D;
        uint8_t* at = vd + h * head + d * 16;
        const uint8_t* code = &s_code[1][h * n * D + d];
        const bool grew = !anew && s_new[1][h] != s_old[1][h];
        if (n < 16 && !grew) {
          for (int r = 0; r < n; ++r) at[s_off[r]] = code[r * D];
          continue;
        }
        u32x4v g = {};
        if (grew) g = rescaled(*reinterpret_cast<const u32x4v*>(at), s_old[1][h], s_new[1][h]);
        for (int r = 0; r < n; ++r) {
          const int off = s_off[r], by = (off & 3) * 8;
          const uint32_t c = (uint32_t)code[r * D] << by, out = ~(0xFFu << by);
#pragma unroll
          for (int w = 0; w < 4; ++w) g[w] = off >> 2 == w ? (g[w] & out) | c : g[w];
        }
        *reinterpret_cast<u32x4v*>(at) = g;
      }
    }
  }
}

template <typename T, int D, bool PAIRS>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kv8_kernel(QkNormRope8Args a, int window, int kv_blocks,
                                                                    int kv_shares, int q_shares) {
  __shared__ __align__(16) float s_cos[16][D / 2], s_sin[16][D / 2];
  const int b = blockIdx.x;
  if (b < kv_blocks)
    keys_values<T, D, PAIRS>(a, (int64_t)(b / kv_shares) * window, window, b % kv_shares, kv_shares, s_cos, s_sin);
  else
    queries<T, D, PAIRS>(a, (int64_t)((b - kv_blocks) / q_shares) * TB, (b - kv_blocks) % q_shares, q_shares, s_cos,
                         s_sin);
}

template <typename T, int D>
hipError_t launch_pairs(const QkNormRope8Args& a, hipStream_t stream) {
  const int cus = device_cus();
  auto shared = [&](int64_t blocks, int64_t most) {          // until a compute unit has four workgroups
    const int64_t s = 4 * (int64_t)cus / blocks;
    return (int)(s > most ? most : s < 1 ? 1 : s);
  };
  const int64_t q_groups = (a.tokens + TB - 1) / TB;
  const int rounds = a.heads_q * TB * (D / 8) / kThreads;    // of a workgroup with all query heads
  const int q_shares = shared(q_groups, rounds < 1 ? 1 : rounds > 64 ? 64 : rounds);
  const int window = a.tokens > 4096 ? 16 : 1;
  const int64_t windows = (a.tokens + window - 1) / window;
  const int kv_shares = shared(window == 1 ? (windows + 15) / 16 : windows, a.heads_kv);
  const int64_t blocks = windows * kv_shares + q_groups * q_shares;
  if (blocks >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
  auto kernel = a.interleaved ? qk_norm_rope_kv8_kernel<T, D, true> : qk_norm_rope_kv8_kernel<T, D, false>;
  kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(a, window, (int)(windows * kv_shares), kv_shares, q_shares);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_dim(const QkNormRope8Args& a, hipStream_t stream) {
  switch (a.head_dim) {
    case 64: return launch_pairs<T, 64>(a, stream);
    case 128: return launch_pairs<T, 128>(a, stream);
    default: return launch_pairs<T, 256>(a, stream);
  }
}

}  // namespace

hipError_t launch_qk_norm_rope_kv8(const QkNormRope8Args& a, hipStream_t stream) {
  return a.fp16 ? launch_dim<F16>(a, stream) : launch_dim<Bf16>(a, stream);
}

}  // namespace trellis
