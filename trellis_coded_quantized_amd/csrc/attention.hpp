// attention.hpp -- device parts of the attention over the paged cache that
// both kernels use: which keys a sequence's rows read, who sees what, and one
// tile's step of the running softmax.
//
// Mathematics.  Row (token i, head): o = sum_j p_j v_j / sum_j p_j over its
// visible keys, p_j = 2^(c q.k_j - m) with c = scale log2(e) and m a running
// bound on the scores.  Scores are computed transposed, S^T = K Q^T, so a
// lane owns one row (MFMA column lane % 32) and its accumulators hold that
// row's keys; O^T = V^T P^T takes P^T straight from those registers:
//   accumulator r of lane half h is MFMA row 8 (r / 4) + 4 h + r % 4; the key
//   loaded as operand row R = 8 j + 4 h + i is key 16 (j / 2) + 8 h +
//   4 (j % 2) + i of the tile, so accumulators 8 s .. 8 s + 7 of half h are
//   keys 16 s + 8 h .. + 7: the B operand of contraction step s, and the
//   eight tokens of one value granule.
// No lane exchanges anything but the row maximum with lane ^ 32.
//
// Precision: scores, maxima, sums and outputs are f32.  P is rounded once to
// the values' 16-bit type for the second product (relative error half a step
// of that type per weight, as the output's own rounding); the sum uses the
// unrounded weights.
#pragma once

#include "internal.hpp"
#include "kv_common.hpp"

namespace trellis {

constexpr float kLog2e = 1.4426950408889634f;
// The bound m follows the row maximum only when that has grown by more than
// 2^8: weights stay below 2^8 (finite in fp16, the same relative precision),
// and most tiles skip the rescaling of O.
constexpr float kRescaleStep = 8.0f;

// operand row -> key of a 32-key tile (see above)
__device__ __forceinline__ int tile_key_of_row(int R) {
  return ((R >> 4) << 4) | (((R >> 2) & 1) << 3) | (((R >> 3) & 1) << 2) | (R & 3);
}

// One entry of the call: its tokens in q, its cached tokens, its page row.
struct Entry {
  int first, n;        // rows of q
  int ctx;             // tokens cached before this call
  int total;           // keys with storage: ctx + n, at most the table's
  const int32_t* pages;
};

__device__ __forceinline__ Entry load_entry(const AttnArgs& a, int e) {
  Entry r;
  const int64_t row = a.seq_ids ? a.seq_ids[e] : e;
  const bool known = row >= 0 && row < a.seqs;
  int b = a.q_start[e], f = a.q_start[e + 1];
  b = min(max(b, 0), (int)a.tokens);
  f = min(max(f, b), (int)a.tokens);
  const int64_t room = a.width << a.page_log2;
  const int len = known ? a.lengths[row] : 0;
  r.first = b;
  r.n = known ? min(f - b, a.max_q) : 0;
  r.ctx = (int)min((int64_t)max(len, 0), room);
  r.total = (int)min((int64_t)r.ctx + r.n, room);
  r.pages = a.table + (known ? row : 0) * a.width;
  return r;
}

// The key tiles (of KT keys) that tokens i0 .. i1 of an entry read, as a
// list: `lead` tiles of first tokens, then tiles from `from` on.
struct TileList {
  int lead, from, count;
  template <int KT>
  __device__ __forceinline__ int key(int u) const { return (u < lead ? u : u - lead + from) * KT; }
};

template <int KT, bool TREE>
__device__ __forceinline__ TileList tile_list(const AttnArgs& a, const Entry& e, int i0, int i1) {
  TileList t;
  t.lead = t.from = 0;
  int end = e.total;
  if (!TREE) {
    end = min(end, e.ctx + i1 + 1);
    if (a.window > 0) {
      const int lo = e.ctx + i0 - a.window + 1;
      const int from = lo > 0 ? lo / KT : 0;
      const int lead = (a.sinks + KT - 1) / KT;
      if (lead < from) {
        t.lead = lead;
        t.from = from;
      }
    }
  }
  t.count = t.lead + max(0, (end + KT - 1) / KT - t.from);
  return t;
}

// What one row sees: keys below `below` that are at least `from` or below
// `sinks`, and, in a tree, node bits from key `below` on.
struct RowMask {
  int below, from, sinks;
  uint64_t nodes;
  template <bool TREE>
  __device__ __forceinline__ bool sees(int key) const {
    if (TREE) {
      const int m = key - below;
      return m < 0 || (m < 64 && ((nodes >> (m & 63)) & 1));
    }
    return key < below && (key >= from || key < sinks);
  }
};

template <bool TREE>
__device__ __forceinline__ RowMask row_mask(const AttnArgs& a, const Entry& e, int i, bool live) {
  RowMask r;
  r.nodes = 0;
  r.sinks = 0;
  r.from = 0;
  r.below = 0;
  if (!live) return r;
  if (TREE) {
    r.below = e.ctx;
    // bits of nodes that have no token, or no room in the table, see nothing
    const int room = min(e.total - e.ctx, 64);
    const uint64_t have = room >= 64 ? ~0ull : ((1ull << room) - 1);
    r.nodes = (uint64_t)a.ancestors[e.first + i] & have;
  } else {
    const int pos = e.ctx + i;
    r.below = min(pos + 1, e.total);
    r.from = a.window > 0 ? pos - a.window + 1 : 0;
    r.sinks = a.sinks;
  }
  return r;
}

// Whether keys kb .. kb + KT - 1 are seen by every row of tokens i0 .. i1.
template <int KT, bool TREE>
__device__ __forceinline__ bool tile_open(const AttnArgs& a, const Entry& e, int i0, int i1, int kb) {
  if (TREE) return kb + KT <= e.ctx;
  if (kb + KT > min(e.ctx + i0 + 1, e.total)) return false;
  return a.window <= 0 || kb >= e.ctx + i1 - a.window + 1 || kb + KT <= a.sinks;
}

// The running softmax of the rows a wave owns.
struct Running {
  float m;     // bound on c * score (-inf: no visible key yet), equal in both lane halves
  float l;     // sum of weights over this lane's keys
};

// Scores of NS 32-key tiles -> weights in place (unrounded), and the running
// bound; `alpha` is what earlier sums and outputs are multiplied with, 1
// unless `moved` (the same answer in all lanes) is returned.
template <int NS>
__device__ __forceinline__ bool softmax_step(f32x16 (&s)[NS], float c, Running& st, float& alpha) {
  float top = s[0][0];
#pragma unroll
  for (int t = 0; t < NS; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) top = fmaxf(top, s[t][r]);
  top = fmaxf(top, __shfl_xor(top, 32)) * c;
  const bool grew = top > st.m + kRescaleStep;          // -inf + 8 = -inf: a first visible key grows it
  const bool moved = __any(grew);
  alpha = 1.0f;
  if (moved) {
    const float m = fmaxf(st.m, top);
    alpha = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
    st.m = m;
    st.l *= alpha;
  }
  const float bound = st.m == -INFINITY ? 0.0f : st.m;
  float sum = 0.0f;
#pragma unroll
  for (int t = 0; t < NS; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[t][r] = __builtin_amdgcn_exp2f(fmaf(s[t][r], c, -bound));
      sum += s[t][r];
    }
  st.l += sum;
  return moved;
}

// The B operands of the second product: weights of one tile, rounded.
template <typename T>
__device__ __forceinline__ void pack_weights(const f32x16& s, u32x4v (&p)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int w = 0; w < 4; ++w) p[h][w] = T::pack(s[8 * h + 2 * w], s[8 * h + 2 * w + 1]);
}

// Zero weights do not hide an infinity or NaN among the values (0 * inf =
// NaN), and such values may stand where a row does not look, or where nothing
// was ever written.  In a tile that some row sees in part they therefore
// enter the product as zeros (drop_nonfinite, which says whether there were
// any), and rows that do see one get it back from here: each lane walks the
// tile's keys and adds what its row sees to its own outputs.
template <typename T>
__device__ __forceinline__ bool drop_nonfinite(u32x4v& v) {
  bool any = false;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t x = v[w];
    const bool lo = (x & T::kExp) == T::kExp, hi = (x & (T::kExp << 16)) == (T::kExp << 16);
    v[w] = (lo ? 0u : x & 0xFFFFu) | (hi ? 0u : x & 0xFFFF0000u);
    any |= lo || hi;
  }
  return any;
}

template <typename T, int D, bool TREE>
__device__ __forceinline__ void add_nonfinite(const AttnArgs& a, const Entry& e, const RowMask& mask, int h, int kb,
                                              int keys, f32x16 (&o)[D / 32]) {
  const int half = (int)__lane_id() >> 5, P = 1 << a.page_log2;
  for (int key = kb; key < kb + keys; ++key) {
    if (!mask.sees<TREE>(key)) continue;
    const uint16_t* v = a.v + ((int64_t)page_in_pool(e.pages[key >> a.page_log2], a.pages) * a.heads_kv + h) *
                                  ((int64_t)D << a.page_log2) +
                        (int64_t)((key & (P - 1)) >> 3) * D * 8 + (key & 7);
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const uint16_t x = v[(d * 32 + 8 * (r >> 2) + 4 * half + (r & 3)) * 8];
        if ((x & T::kExp) == T::kExp) o[d][r] += T::to_f32(x);
      }
  }
}

}  // namespace trellis
