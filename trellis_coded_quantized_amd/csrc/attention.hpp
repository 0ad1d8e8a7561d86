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

// an address known to be in device memory (a pointer put together from integers is not)
typedef const __attribute__((address_space(1))) int32_t* GlobalInts;

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
  int total;           // keys with a place in the table: ctx + n, at most its room
  GlobalInts pages;
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
  r.pages = (GlobalInts)(a.table + (known ? row : 0) * a.width);
  return r;
}

__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(uint64_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// The same entry with its numbers in scalar registers (all lanes hold the same).
__device__ __forceinline__ Entry uniform(Entry e) {
  e.first = __builtin_amdgcn_readfirstlane(e.first);
  e.n = __builtin_amdgcn_readfirstlane(e.n);
  e.ctx = __builtin_amdgcn_readfirstlane(e.ctx);
  e.total = __builtin_amdgcn_readfirstlane(e.total);
  e.pages = (GlobalInts)uniform((int64_t)e.pages);
  return e;
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
// `sinks`, and, in a tree, node bits from key `below` on.  Keys whose page is
// not there are taken out by the kernels, a tile at a time: its pages are at
// hand when it is read.
struct RowMask {
  int below, from, sinks;
  uint64_t nodes;
  // bit j: key kb + j (of 64) is seen
  template <bool TREE>
  __device__ __forceinline__ uint64_t bits(int kb) const {
    const uint64_t under = ones(below - kb);
    if (TREE) {
      const int at = below - kb;                             // where node 0 stands
      const uint64_t drafted = at >= 64 || at <= -64 ? 0 : at >= 0 ? nodes << at : nodes >> -at;
      return under | drafted;
    }
    return under & (~ones(from - kb) | ones(sinks - kb));
  }
  // the n lowest bits
  static __device__ __forceinline__ uint64_t ones(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
  }
};

// Scores of keys that the row does not see become -inf.  `seen`: bits of the
// 32-key tile; a lane half holds keys 16 s + 8 half + 0 .. 7 in accumulators
// 8 s + 0 .. 7.
__device__ __forceinline__ void cut_scores(f32x16& s, uint32_t seen) {
  asm volatile("" : "+v"(seen));          // keeps the caller's branch: most tiles need none of this
  seen >>= ((int)__lane_id() >> 5) * 8;
#pragma unroll
  for (int r = 0; r < 16; ++r) s[r] = (seen >> ((r >> 3) * 16 + (r & 7))) & 1u ? s[r] : -INFINITY;
}

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
    r.nodes = (uint64_t)a.ancestors[e.first + i] & RowMask::ones(e.total - e.ctx);
  } else {
    const int pos = e.ctx + i;
    r.below = min(pos + 1, e.total);
    r.from = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
    r.sinks = a.sinks;
  }
  return r;
}

// The keys that every row of tokens i0 .. i1 sees if they have a page: from ..
// to - 1, and those below sinks.
struct OpenKeys {
  int from, to, sinks;
  __device__ __forceinline__ bool tile(int kb, int keys) const {
    return kb + keys <= to && (kb >= from || kb + keys <= sinks);
  }
};

template <bool TREE>
__device__ __forceinline__ OpenKeys open_keys(const AttnArgs& a, const Entry& e, int i0, int i1) {
  if (TREE) return {0, e.ctx, 0};
  return {a.window > 0 ? max(e.ctx + i1 - a.window + 1, 0) : 0, min(e.ctx + i0 + 1, e.total), a.sinks};
}

// x and the same of the lane 32 away, the larger of the two.
__device__ __forceinline__ float max_of_halves(float x) {
  const uint32_t v = __builtin_bit_cast(uint32_t, x);
  const auto both = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)both[0]), __builtin_bit_cast(float, (uint32_t)both[1]));
}

// The running softmax of the rows a wave owns.
struct Running {
  float m;     // bound on c * score (-inf: no visible key yet), equal in both lane halves
  float l;     // sum of weights over this lane's keys
};

// The largest score of a row over a 32-key tile, scaled.
__device__ __forceinline__ float row_top(const f32x16& s, float c) {
  float top = s[0];
#pragma unroll
  for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
  return max_of_halves(top) * c;
}

// Whether any row of the wave has to move its bound for that score (-inf + 8
// = -inf: a first visible key moves it).
__device__ __forceinline__ bool must_move(float top, const Running& st) {
  return __any(top > st.m + kRescaleStep);
}

// Moves the bound; returns what the lane's earlier sum (done here) and outputs
// have to be multiplied with.
__device__ __forceinline__ float move_bound(float top, Running& st) {
  const float m = fmaxf(st.m, top);
  const float alpha = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
  st.m = m;
  st.l *= alpha;
  return alpha;
}

// Scores -> weights under the current bound, rounded and packed as the B
// operands of the second product; returns their unrounded sum over this
// lane's keys.
template <typename T>
__device__ __forceinline__ float weigh(const f32x16& s, float c, const Running& st, u32x4v (&p)[2]) {
  const float bound = st.m == -INFINITY ? 0.0f : st.m;
  float sum[2] = {0.0f, 0.0f};
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float x = __builtin_amdgcn_exp2f(fmaf(s[8 * h + 2 * w], c, -bound));
      const float y = __builtin_amdgcn_exp2f(fmaf(s[8 * h + 2 * w + 1], c, -bound));
      sum[0] += x;
      sum[1] += y;
      p[h][w] = T::pack(x, y);
    }
  return sum[0] + sum[1];
}

// The same one score at a time, e = 0 .. 15 in order: a pair is packed with its
// second one.
template <typename T>
__device__ __forceinline__ void weigh_one(const f32x16& s, float c, const Running& st, int e, float& sum,
                                          u32x4v (&p)[2]) {
  const float bound = st.m == -INFINITY ? 0.0f : st.m;
  const float x = __builtin_amdgcn_exp2f(fmaf(s[e], c, -bound));
  sum += x;
  const int h = e >> 3, w = (e >> 1) & 3;
  p[h][w] = e & 1 ? T::pack(__builtin_bit_cast(float, (uint32_t)p[h][w]), x) : __builtin_bit_cast(uint32_t, x);
}

// At D = 256 a wave's outputs stay in accumulation registers; left alone, the
// allocator copies all of them to vector registers and back in every tile.
template <int DT>
__device__ __forceinline__ void settle(f32x16 (&o)[DT]) {
  if constexpr (DT == 8) {
#pragma unroll
    for (int d = 0; d < DT; ++d) asm volatile("" : "+a"(o[d]));
  }
}

// Zero weights do not hide an infinity or NaN among the values (0 * inf =
// NaN), and such values may stand where a row does not look, or where nothing
// was ever written.  In a tile that some row sees in part they therefore
// enter the product as zeros (drop_nonfinite, which says whether there were
// any), and rows that do see one get it back from here: each lane walks the
// tile's keys and adds what its row sees to its own outputs.  The walk ends
// with the table's room: the last tile may reach past it.  What the row sees is
// worked out once for the tile: key by key it costs the kernels that call this
// registers in their main loop (2 trees of 64 over 131000 keys, 24 / 4 heads of
// 256: 332 us against 343; 64 trees of 16 over 4096, 32 / 8 heads of 128: 212
// against 219; only heads of 64 would be faster so, 132 against 140).
template <typename T, int N>
__device__ __forceinline__ bool drop_nonfinite(u32x4v (&v)[N]) {
  // an exponent of all ones carries into the sign's place when its last bit is added
  constexpr uint32_t E = T::kExp * 0x10001u, L = (T::kExp & (0u - T::kExp)) * 0x10001u;
  uint32_t any = 0;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int w = 0; w < 4; ++w) any |= (v[n][w] & E) + L;
  if (!__any((any & 0x80008000u) != 0)) return false;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t x = v[n][w], hit = ((x & E) + L) & 0x80008000u;
      v[n][w] = x & ~((hit >> 15) * 0xFFFFu);
    }
  return (any & 0x80008000u) != 0;
}

template <typename T, int D, bool TREE>
__device__ __forceinline__ void add_nonfinite(const uint16_t* v_head, GlobalInts pages, int room, uint32_t pool,
                                              uint32_t page_elems, int page_log2, const RowMask& mask, int kb, int keys,
                                              f32x16 (&o)[D / 32]) {
  const int half = (int)__lane_id() >> 5, n = min(keys, room - kb);
  uint64_t seen = mask.bits<TREE>(kb);
  for (int j = 0; j < n; ++j, seen >>= 1) {
    const int key = kb + j;
    const int32_t page = pages[key >> page_log2];
    const uint16_t* v = v_head + (uint64_t)page_in_pool(page, pool) * page_elems +
                        ((key & ((1 << page_log2) - 1)) >> 3) * D * 8 + (key & 7);
    const uint32_t sees = (uint32_t)seen & (page_ok(page, pool) ? 1u : 0u);
#pragma unroll
    for (int d = 0; d < D / 32; ++d) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const uint16_t x = v[(d * 32 + 8 * (r >> 2) + 4 * half + (r & 3)) * 8];
        o[d][r] += (x & T::kExp) == T::kExp && sees ? T::to_f32(x) : 0.0f;
      }
      __builtin_amdgcn_sched_barrier(0);                     // rare code: few registers, not speed
    }
  }
}

}  // namespace trellis
