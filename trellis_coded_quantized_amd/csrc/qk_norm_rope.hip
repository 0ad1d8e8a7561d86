// qk_norm_rope.hip -- RMS norm of every query and key head, rotation by
// position, and the append of keys and values to the paged cache, one pass.
#include "internal.hpp"
#include "norm_rope.hpp"

namespace trellis {
namespace {

constexpr int kThreads = 256;
constexpr int TB = 8;          // tokens of a workgroup
constexpr uint32_t kXcds = 8;

// Norm and rotation (norm_rope.hpp) are f32 and rounded once.
//
// Bound by memory: every value is read once and written once.  A workgroup
// takes TB tokens and a share of the heads; the angles of its tokens are
// computed once for all its heads (into LDS).  D / 8 lanes own a query or key
// head, eight dimensions each; keys leave as 16-byte granules.  A value
// granule is eight tokens of one dimension, so values go through LDS and
// leave with the tokens innermost: lanes of eight neighbouring slots write
// neighbouring addresses, whatever the slots' alignment.
//
// Eight tokens are a granule: with 16 a workgroup's LDS leaves too few of them
// on a compute unit (8191 tokens, 32 / 8 heads of 128: 48 us against 37), and
// a form with one token each for few tokens was slower there too (4 tokens of
// 24 / 4 heads of 256: 6.0 us against 5.2).  Workgroups with neighbouring
// tokens run on one XCD, so granules that two of them share meet in its L2
// (45 us without).  8191 tokens, 32 / 8 heads of 128, interleaved: 38 us,
// 5.3 TB/s, what a large copy reaches; split halves 44 us; 4 tokens 4.7 us.
template <typename T, int D, bool PAIRS>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(QkNormRopeArgs a) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  constexpr int VH = 1024 / D, VROW = D + 2;   // value heads in LDS at a time; odd dword rows
  __shared__ __attribute__((aligned(16))) float s_cos[TB][D / 2], s_sin[TB][D / 2];
  __shared__ __attribute__((aligned(16))) uint16_t s_v[VH * TB * VROW];
  const uint32_t each = gridDim.x / kXcds, more = gridDim.x % kXcds, xcd = blockIdx.x % kXcds;
  const int64_t first = (int64_t)(xcd * each + min(xcd, more) + blockIdx.x / kXcds) * TB;
  const int tokens = (int)min((int64_t)TB, a.tokens - first);
  const int tid = threadIdx.x, grp = tid / LANES, l = tid % LANES, d0 = l * 8;
  const int half = a.rotary / 2, P = 1 << a.page_log2;
  const int heads = a.heads_q + a.heads_kv;
  const int h0 = (int)((int64_t)heads * blockIdx.y / gridDim.y), h1 = (int)((int64_t)heads * (blockIdx.y + 1) / gridDim.y);
  const int v0 = (int)((int64_t)a.heads_kv * blockIdx.y / gridDim.y);
  const int v1 = (int)((int64_t)a.heads_kv * (blockIdx.y + 1) / gridDim.y);

  for (int x = tid; x < tokens * half; x += kThreads) {
    const int t = x / half, i = x - t * half;
    float s, c;
    turn(a.positions[first + t], a.inv_freq[i], c, s);
    s_cos[t][i] = c;
    s_sin[t][i] = s;
  }
  // where a token's slot lies: page and place, or a page outside the pool
  auto page_of = [&](int slot) { return (uint32_t)(slot >> a.page_log2); };
  auto cached = [&](int slot) { return slot >= 0 && page_of(slot) < a.pages; };

  // ---- values
  for (int hb = v0; hb < v1; hb += VH) {
    const int nh = min(VH, v1 - hb);
    if (hb != v0) __syncthreads();
    for (int x = grp; x < nh * TB; x += GROUPS) {
      const int h = x / TB, t = x % TB;
      if (t >= tokens) continue;
      const u32x4v raw = *reinterpret_cast<const u32x4v*>(a.v + (first + t) * a.v_stride + (hb + h) * D + d0);
      uint32_t* row = reinterpret_cast<uint32_t*>(s_v + x * VROW + d0);
#pragma unroll
      for (int w = 0; w < 4; ++w) row[w] = raw[w];
    }
    __syncthreads();
    const int t = tid % TB, slot = t < tokens ? a.slots[first + t] : -1, off = slot & (P - 1);
    if (cached(slot)) {
      uint16_t* dst = a.v_cache + ((int64_t)page_of(slot) * a.heads_kv + hb) * ((int64_t)D << a.page_log2) +
                      (int64_t)(off >> 3) * D * 8 + (off & 7);
#pragma unroll 4
      for (int x = tid / TB; x < nh * D; x += kThreads / TB) {
        const int h = x / D, d = x % D;
        dst[((int64_t)h * D << a.page_log2) + d * 8] = s_v[(h * TB + t) * VROW + d];
      }
    }
  }
  __syncthreads();

  // ---- queries and keys
  for (int x = grp; x < (h1 - h0) * TB; x += GROUPS) {
    const int h = h0 + x / TB, t = x % TB;
    if (t >= tokens) continue;
    const int64_t tok = first + t;
    const bool is_q = h < a.heads_q;
    const int hh = is_q ? h : h - a.heads_q;
    const uint16_t* src = (is_q ? a.q + tok * a.q_stride : a.k + tok * a.k_stride) + hh * D + d0;
    const uint16_t* weight = (is_q ? a.q_weight : a.k_weight) + d0;
    float y[8];
    norm_rotate<T, D, PAIRS>(*reinterpret_cast<const u32x4v*>(src), src, weight, d0, a.rotary, a.eps, s_cos[t], s_sin[t], y);
    u32x4v res;
#pragma unroll
    for (int w = 0; w < 4; ++w) res[w] = T::pack(y[2 * w], y[2 * w + 1]);
    if (is_q) {
      *reinterpret_cast<u32x4v*>(a.out + (tok * a.heads_q + hh) * D + d0) = res;
    } else {
      const int slot = a.slots[tok], off = slot & (P - 1);
      if (cached(slot))
        *reinterpret_cast<u32x4v*>(a.k_cache + ((int64_t)page_of(slot) * a.heads_kv + hh) * ((int64_t)D << a.page_log2) +
                                   ((int64_t)l * P + off) * 8) = res;
    }
  }
}

template <typename T, int D>
hipError_t launch_pairs(const QkNormRopeArgs& a, hipStream_t stream) {
  const int64_t blocks = (a.tokens + TB - 1) / TB;
  const int rounds = (a.heads_q + a.heads_kv) * TB * (D / 8) / kThreads;     // of a workgroup with all heads
  // heads are shared out until a compute unit has four workgroups (2048 tokens,
  // 24 / 4 heads of 256: 19 us; two 23, one 35)
  int64_t shares = 4 * (int64_t)device_cus() / blocks;
  if (shares > rounds) shares = rounds;
  const dim3 grid((unsigned)blocks, (unsigned)(shares < 1 ? 1 : shares > 64 ? 64 : shares));
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
