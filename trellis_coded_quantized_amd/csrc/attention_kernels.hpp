// attention_kernels.hpp -- attention of new tokens over the paged cache: the
// kernel for few rows per key head (decoding, small trees), the kernel for many
// (prompt chunks, wide trees), and the fold of split keys, for a cache of the
// queries' own type (Kv16, attention.hip) and one held in 8 bits (Kv8,
// attention_kv8.hip).  They differ in what a tile's loads bring and in how it
// gets into operand registers or LDS; scores, softmax and products are the same.
#pragma once

#include "attention.hpp"
#include "copy_ring.hpp"
#include <type_traits>

namespace trellis {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kFewRows = 32;              // rows of the few-row kernel: one MFMA tile
constexpr int kManyKeys = 64;             // keys of a tile of the many-row kernel
constexpr int kManyRun = 4;               // fewest tiles that it cuts the keys into

// ---- what the cache holds ------------------------------------------------
// The queries' own 16-bit type: granules are operands as they stand.
struct Kv16 {
  typedef AttnArgs Args;
  static constexpr int PACK = 1;                             // operands in 16 bytes
  static __device__ __forceinline__ int key_of_row(int R) { return tile_key_of_row(R); }
  static __device__ __forceinline__ void cut(f32x16& s, uint32_t seen) { cut_scores(s, seen); }
  template <typename T, int D, bool TREE>
  static __device__ __forceinline__ void put_back(const AttnArgs& a, uint32_t head_at, int, GlobalInts pages,
                                                  uint32_t page_elems, const RowMask& mask, int kb, int keys,
                                                  f32x16 (&o)[D / 32]) {
    add_nonfinite<T, D, TREE>(a.v + head_at, pages, (int)a.width << a.page_log2, a.pages, page_elems, a.page_log2,
                              mask, kb, keys, o);
  }
};

// e4m3, one power-of-two scale for 16 tokens of a head.  Elements become
// code * scale in the queries' type on their way into an operand, two in one
// instruction that takes the scale along: exact, since e4m3 has 4 significant
// bits (fp16 below its normal numbers: rounded once).  A granule is two
// operands: 16 dimensions of a token, or the 16 tokens of a block, so in the
// kernel for few rows a lane half owns a block of keys:
//   accumulator r of half h is key 16 h + r.
// 64 single tokens over 16383 keys, 32 / 8 heads of 128: 228 us a call, 5.3 TB/s
// of 1 byte an element, 422 at 16 bits; one over 200000, 24 / 4 of 256: 81 and 148.
// Windows of 2047 x 3 tokens take 222 us in either, 2 trees of 64 over 131000 at
// D = 256 312 against 321: the conversions are vector work, half as much is read.
struct Kv8 {
  typedef Attn8Args Args;
  static constexpr int PACK = 2;
  static __device__ __forceinline__ int key_of_row(int R) { return ((R >> 2) & 1) * 16 + (R >> 3) * 4 + (R & 3); }
  static __device__ __forceinline__ void cut(f32x16& s, uint32_t seen) {
    asm volatile("" : "+v"(seen));        // keeps the caller's branch, as in cut_scores
    seen >>= ((int)__lane_id() >> 5) * 16;
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = (seen >> r) & 1u ? s[r] : -INFINITY;
  }
  // 2^(byte - 127); the conversions look at the exponent alone
  static __device__ __forceinline__ float scale(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }
  template <typename T, bool HIGH>
  static __device__ __forceinline__ uint32_t two(uint32_t codes, float scale) {
    if constexpr (std::is_same<T, Bf16>::value)
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, HIGH));
    else
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, scale, HIGH));
  }
  // the first or second eight codes of a granule (or the eight there are) as an operand
  template <typename T, typename G>
  static __device__ __forceinline__ u32x4v widen(const G& g, int which, float scale) {
    const uint32_t x = g[2 * which], y = g[2 * which + 1];
    return u32x4v{two<T, false>(x, scale), two<T, true>(x, scale), two<T, false>(y, scale), two<T, true>(y, scale)};
  }
  // add_nonfinite (attention.hpp) over codes and scales
  template <typename T, int D, bool TREE>
  static __device__ __forceinline__ void put_back(const Attn8Args& a, uint32_t head_at, int h, GlobalInts pages,
                                                  uint32_t page_elems, const RowMask& mask, int kb, int keys,
                                                  f32x16 (&o)[D / 32]) {
    const int half = (int)__lane_id() >> 5, n = min(keys, ((int)a.width << a.page_log2) - kb);
    const uint8_t* pool = reinterpret_cast<const uint8_t*>(a.v) + head_at;
    uint64_t seen = mask.bits<TREE>(kb);
    for (int j = 0; j < n; ++j, seen >>= 1) {
      const int key = kb + j, at = key & ((1 << a.page_log2) - 1);
      const int32_t page = pages[key >> a.page_log2];
      const uint64_t in = page_in_pool(page, a.pages);
      const uint8_t* v = pool + in * page_elems + (at >> 4) * D * 16 + (at & 15);
      const float by = scale(a.v_scale[((in * a.heads_kv + h) << (a.page_log2 - 4)) + (at >> 4)]);
      const uint32_t sees = (uint32_t)seen & (page_ok(page, a.pages) ? 1u : 0u);
#pragma unroll
      for (int d = 0; d < D / 32; ++d) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const uint16_t x = (uint16_t)two<T, false>(v[(d * 32 + 8 * (r >> 2) + 4 * half + (r & 3)) * 16], by);
          o[d][r] += (x & T::kExp) == T::kExp && sees ? T::to_f32(x) : 0.0f;
        }
        __builtin_amdgcn_sched_barrier(0);                   // rare code: few registers, not speed
      }
    }
  }
};

// ---- cutting keys --------------------------------------------------------
// Units of work (all rows of an entry, or a tile of them) whose keys are cut
// into chunks of equally many tiles, so that the slots (unit, chunk) fill the
// `target` workgroups of a key head.  Every workgroup works the same cut out
// from the lengths, 64 entries at a time, one a lane.
constexpr int kRounds = 3;                // slots per workgroup where entries are many and unlike

struct Cut {
  int tiles, units;                       // this lane's entry of the first 64
  int chunk;
};

__device__ __forceinline__ int64_t wave_sum64(int64_t v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// sizes(e, tiles, units): how long the units of entry e are and how many.
// One slot a workgroup if a chunk little longer than the mean does it (the
// chunk grows until its slots fit), else kRounds of a third.  In the end all
// slots fit, or no unit is cut.
template <typename Sizes>
__device__ __forceinline__ Cut find_cut(const AttnArgs& a, int least, const Sizes& sizes) {
  const int lane = (int)__lane_id();
  Cut cut{0, 0, 0};
  if (lane < a.entries) sizes(lane, cut.tiles, cut.units);
  int64_t total = (int64_t)cut.tiles * cut.units;
  int longest = cut.tiles;
  for (int b = 64; b < a.entries; b += 64) {
    int t = 0, n = 0;
    if (b + lane < a.entries) sizes(b + lane, t, n);
    total += (int64_t)t * n;
    longest = max(longest, t);
  }
  total = uniform(wave_sum64(total));
#pragma unroll
  for (int d = 32; d; d >>= 1) longest = max(longest, __shfl_xor(longest, d));
  longest = __builtin_amdgcn_readfirstlane(longest);
  // whether one unit is all there is: the only entry's, which is lane 0's
  const bool single = a.entries == 1 && __builtin_amdgcn_readfirstlane(cut.units) == 1;
  auto slots = [&](int c) {
    int64_t n = (int64_t)((cut.tiles + c - 1) / c) * cut.units;
    for (int b = 64; b < a.entries; b += 64) {
      int t = 0, u = 0;
      if (b + lane < a.entries) sizes(b + lane, t, u);
      n += (int64_t)((t + c - 1) / c) * u;
    }
    return uniform(wave_sum64(n));
  };
  for (int rounds = 1;; rounds = a.rounds) {
    const int64_t room = (int64_t)rounds * a.target, mean = (total + room - 1) / room;
    int64_t c = mean < least ? least : mean;
    if (c >= longest) {
      cut.chunk = __builtin_amdgcn_readfirstlane(max(longest, 1));
      return cut;
    }
    if (single) {                                            // mean was rounded up: it fits
      cut.chunk = __builtin_amdgcn_readfirstlane((int)c);
      return cut;
    }
    bool fits = false;
    for (int tries = 0; tries < 5 && c < longest; ++tries) {
      const int64_t n = slots((int)c);
      if (n <= room) {
        fits = true;
        break;
      }
      c = max(c + 1, c * n / room);
    }
    if (rounds == a.rounds || (fits && c * 4 <= mean * 5)) {
      cut.chunk = __builtin_amdgcn_readfirstlane(fits ? (int)c : max(longest, 1));
      return cut;
    }
  }
}

// ---- few rows ------------------------------------------------------------
// All rows of an entry that share a key head (tokens x query heads per key
// head, at most 32) are one MFMA tile, so keys and values are read once,
// straight into operand registers; the four waves of a workgroup take the
// tiles of its chunk in turn.

struct Unit {
  int e, split, splits, chunk;
  int own_base, own_splits;               // the slots of entry number `slot`, whose note this workgroup writes
  bool live;
};

template <bool TREE>
__device__ __forceinline__ int entry_tiles(const AttnArgs& a, int e) {
  if (e >= a.entries) return 0;
  const Entry en = load_entry(a, e);
  if (en.n == 0) return 0;
  return max(1, tile_list<32, TREE>(a, en, 0, en.n - 1).count);
}

// Slot -> (entry, split); slot numbers reach past the entries' numbers.
template <bool TREE>
__device__ __forceinline__ Unit find_unit(const AttnArgs& a, int slot) {
  const int lane = (int)__lane_id();
  Unit u{};
  const Cut cut = find_cut(a, kWaves, [&](int e, int& tiles, int& units) {
    tiles = entry_tiles<TREE>(a, e);
    units = 1;
  });
  u.chunk = cut.chunk;
  int before = 0, tiles = cut.tiles;
  for (int b = 0; b < a.entries; b += 64) {
    if (b) tiles = entry_tiles<TREE>(a, b + lane);
    const int parts = (tiles + u.chunk - 1) / u.chunk;
    const int upto = wave_scan_add(parts);
    const uint64_t hit = __ballot(before + upto > slot);
    if (hit && !u.live) {
      const int at = __builtin_ctzll(hit);
      u.e = b + at;
      u.splits = __builtin_amdgcn_readlane(parts, at);
      u.split = slot - before - __builtin_amdgcn_readlane(upto, at) + u.splits;
      u.live = true;
    }
    if (slot >= b && slot < b + 64) {
      u.own_splits = __builtin_amdgcn_readlane(parts, slot - b);
      u.own_base = before + __builtin_amdgcn_readlane(upto, slot - b) - u.own_splits;
    }
    if (u.live && slot < b + 64) break;
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return u;
}

template <typename S, typename T, int D, bool TREE>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void attention_few_kernel(typename S::Args a) {
  constexpr int STEPS = D / 16, DT = D / 32;
  constexpr int JOIN = DT < 4 ? DT : 4;                      // 32-dimension tiles joined at a time
  __shared__ float s_m[kWaves][32], s_l[kWaves][32];
  __shared__ __align__(16) float s_o[kWaves][32][JOIN * 32 + 4];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, col = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = blockIdx.y, group = a.heads_q / a.heads_kv;
  const Unit u = find_unit<TREE>(a, blockIdx.x);
  if (h == 0 && tid == 0 && (int)blockIdx.x < a.entries) {   // for the fold
    PartNote note{u.own_splits > 1 ? u.own_splits : 0, 0, 0, u.own_base, 1};
    if (note.parts) {
      const Entry own = load_entry(a, blockIdx.x);
      note.first = own.first;
      note.rows = own.n * group;
    }
    a.part_note[blockIdx.x] = note;
  }
  if (!u.live) return;
  const Entry e = uniform(load_entry(a, __builtin_amdgcn_readfirstlane(u.e)));
  const int rows = e.n * group;
  const TileList list = tile_list<32, TREE>(a, e, 0, e.n - 1);
  const int t0 = __builtin_amdgcn_readfirstlane(u.split * u.chunk);
  const int t1 = __builtin_amdgcn_readfirstlane(min(list.count, t0 + u.chunk));
  const int P = 1 << a.page_log2, pmask = P - 1;
  const uint32_t page_elems = (uint32_t)(a.heads_kv * D) << a.page_log2, head_at = (uint32_t)(h * D) << a.page_log2;
  const int krow = S::key_of_row(col);

  // A wave takes every fourth tile.  Keys of the next one are under way while
  // the softmax and the second product of this one run, values while the next
  // one's scores are computed; page numbers are a tile further ahead.
  u32x4v kf[STEPS / S::PACK], vf[2 / S::PACK][DT];
  uint32_t ke = 0, ve = 0;                                   // Kv8: scales of the keys' and the values' blocks
  int page[2];                                               // of a tile's two halves of 16 keys
  auto load_pages = [&](int t) {
    const int kb = list.key<32>(min(t, t1 - 1));
    page[0] = e.pages[min(kb >> a.page_log2, (int)a.width - 1)];
    page[1] = e.pages[min((kb + 16) >> a.page_log2, (int)a.width - 1)];
  };
  uint64_t at[2];                                            // their elements in the pools
  uint32_t held = 0;                                         // the tile's keys whose page is there
  auto locate = [&]() {
    held = 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int32_t own = __builtin_amdgcn_readfirstlane(page[s]);
      held |= page_ok(own, a.pages) ? 0xFFFFu << (16 * s) : 0u;
      at[s] = (uint64_t)page_in_pool(own, a.pages) * page_elems + head_at;
    }
  };
  auto load_keys = [&](int t) {
    const int kb = list.key<32>(t);
    if constexpr (S::PACK == 1) {
      const uint16_t* kp = a.k + (krow >= 16 ? at[1] : at[0]) + (((kb + krow) & pmask) + half * P) * 8;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) kf[s] = *reinterpret_cast<const u32x4v*>(kp + s * 16 * P);
    } else {
      const uint64_t page = krow >= 16 ? at[1] : at[0];
      const int key = (kb + krow) & pmask;
      const uint8_t* kp = reinterpret_cast<const uint8_t*>(a.k) + page + (key + half * P) * 16;
      ke = a.k_scale[page / (D * 16) + (key >> 4)];
#pragma unroll
      for (int s = 0; s < STEPS / 2; ++s) kf[s] = *reinterpret_cast<const u32x4v*>(kp + s * 32 * P);
    }
  };
  auto load_values = [&](int t) {
    const int kb = list.key<32>(t);
    if constexpr (S::PACK == 1) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint16_t* vp = a.v + at[s] + (((kb + s * 16) & pmask) >> 3) * D * 8;
#pragma unroll
        for (int d = 0; d < DT; ++d)
          vf[s][d] = *reinterpret_cast<const u32x4v*>(vp + (uint32_t)((half * D + col) * 8 + d * 256));
      }
    } else {
      // a lane half has a block of 16 tokens: 16 bytes of one dimension
      const uint64_t page = half ? at[1] : at[0];
      const int block = ((kb + 16 * half) & pmask) >> 4;
      const uint8_t* vp = reinterpret_cast<const uint8_t*>(a.v) + page + (block * D + col) * 16;
      ve = a.v_scale[page / (D * 16) + block];
#pragma unroll
      for (int d = 0; d < DT; ++d) vf[0][d] = *reinterpret_cast<const u32x4v*>(vp + d * 512);
    }
  };
  int t = t0 + wave;
  if (t < t1) load_pages(t);

  const bool live = col < rows;
  const int i = live ? col / group : 0, hq = h * group + (live ? col % group : 0);
  u32x4v q[STEPS];
  {
    const uint16_t* src = a.q + (int64_t)(e.first + i) * a.q_stride + (int64_t)hq * D + half * 8 * S::PACK;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
      q[s] = *reinterpret_cast<const u32x4v*>(src + s / S::PACK * 16 * S::PACK + s % S::PACK * 8);
  }
  const RowMask mask = row_mask<TREE>(a, e, i, live);
  const OpenKeys seen_by_all = open_keys<TREE>(a, e, 0, e.n - 1);
  if (t < t1) {
    locate();
    load_keys(t);
    load_values(t);
    load_pages(t + kWaves);
  }

  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = f32x16{};
  Running st{-INFINITY, 0.0f};
  const float c = a.scale * kLog2e;
  for (; t < t1; t += kWaves) {
    const int kb = list.key<32>(t);
    const bool more = t + kWaves < t1;
    const uint32_t here = held;
    f32x16 sc = f32x16{};
    if constexpr (S::PACK == 1) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) sc = T::mfma(kf[s], q[s], sc);
    } else {
      const float scale = S::scale(ke);
#pragma unroll
      for (int s = 0; s < STEPS; ++s) sc = T::mfma(S::template widen<T>(kf[s / 2], s & 1, scale), q[s], sc);
    }
    if (more) {
      locate();
      load_keys(t + kWaves);
      load_pages(t + 2 * kWaves);
    }
    bool bad = false;
    const bool closed = !seen_by_all.tile(kb, 32) || here != ~0u;
    if (closed) {
      S::cut(sc, (uint32_t)mask.bits<TREE>(kb) & here);
      if constexpr (S::PACK == 1) {
        bad = drop_nonfinite<T>(vf[0]);
        bad |= drop_nonfinite<T>(vf[1]);
      }
    }
    const float top = row_top(sc, c);
    if (must_move(top, st)) {
      const float alpha = move_bound(top, st);
      settle(o);
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[d][r] *= alpha;
      settle(o);
    }
    u32x4v p[2];
    st.l += weigh<T>(sc, c, st, p);
    if constexpr (S::PACK == 1) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int s = 0; s < 2; ++s) o[d] = T::mfma(vf[s][d], p[s], o[d]);
    } else {
      const float scale = S::scale(ve);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        u32x4v v[2] = {S::template widen<T>(vf[0][d], 0, scale), S::template widen<T>(vf[0][d], 1, scale)};
        if (closed) bad |= drop_nonfinite<T>(v);
#pragma unroll
        for (int s = 0; s < 2; ++s) o[d] = T::mfma(v[s], p[s], o[d]);
      }
    }
    if (more) load_values(t + kWaves);
    settle(o);
    if (__any(bad)) {
      S::template put_back<T, D, TREE>(a, head_at, h, e.pages, page_elems, mask, kb, 32, o);
      settle(o);
    }
  }
  settle(o);

  // join the four waves
  st.l += __shfl_xor(st.l, 32);
  if (half == 0) {
    s_m[wave][col] = st.m;
    s_l[wave][col] = st.l;
  }
  __syncthreads();
  float top = s_m[0][col];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) top = fmaxf(top, s_m[w][col]);
  const float f = st.m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(st.m - top);
  const int orow = tid >> 3, od = (tid & 7) * 4;             // this thread's output row and dimensions
  float otop = s_m[0][orow], osum = 0.0f;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) otop = fmaxf(otop, s_m[w][orow]);
#pragma unroll
  for (int w = 0; w < kWaves; ++w)
    osum += s_l[w][orow] * (s_m[w][orow] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(s_m[w][orow] - otop));
  const bool whole = u.splits == 1;
  const float inv = whole ? (osum == 0.0f ? 0.0f : 1.0f / osum) : 1.0f;
  const int64_t slot = (int64_t)blockIdx.x * a.heads_kv + h;
  const bool owrite = orow < rows;
  uint16_t* dst = a.out + ((int64_t)(e.first + orow / group) * a.heads_q + h * group + orow % group) * D + od;
  float* part = a.part_o + (slot * kFewRows + orow) * D + od;
#pragma unroll
  for (int d0 = 0; d0 < DT; d0 += JOIN) {
    if (d0) __syncthreads();
#pragma unroll
    for (int d = 0; d < JOIN; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x16& x = o[d0 + d];
        *reinterpret_cast<f32x4v*>(&s_o[wave][col][d * 32 + 8 * j + 4 * half]) =
            f32x4v{x[4 * j] * f, x[4 * j + 1] * f, x[4 * j + 2] * f, x[4 * j + 3] * f};
      }
    __syncthreads();
    if (!owrite) continue;
#pragma unroll
    for (int d = 0; d < JOIN; ++d) {
      f32x4v sum = *reinterpret_cast<const f32x4v*>(&s_o[0][orow][d * 32 + od]);
#pragma unroll
      for (int w = 1; w < kWaves; ++w) sum += *reinterpret_cast<const f32x4v*>(&s_o[w][orow][d * 32 + od]);
      if (whole)
        *reinterpret_cast<u32x2v*>(dst + (d0 + d) * 32) =
            u32x2v{T::pack(sum[0] * inv, sum[1] * inv), T::pack(sum[2] * inv, sum[3] * inv)};
      else
        *reinterpret_cast<f32x4v*>(part + (d0 + d) * 32) = sum;
    }
  }
  if (!whole && owrite && (tid & 7) == 0)
    *reinterpret_cast<f32x2p*>(a.part_ml + (slot * kFewRows + orow) * 2) = f32x2p{otop, osum};
}

// ---- many rows -----------------------------------------------------------
// A workgroup takes 256 rows (token-major, the query heads of one key head
// innermost), 32 a wave, and walks its keys in tiles of 64 that all waves
// share through LDS, in the cache's own granule order, so LDS reads are
// contiguous across lanes and nothing is transposed.  At D = 256 a wave's
// outputs and queries fill a SIMD's registers alone, and it is 128 rows, as
// where no entry has more.
//
// A tile is two blocks of 32 keys.  The product with the values runs one tile
// behind the scores: a block's maximum is taken under the next block's scores,
// its weights under the product of the block before it, so all vector work
// has matrix work beside it, from the same wave at D = 256 where there is no
// other.  Loads of a tile are under way for a whole period.  The order is
// written out and pinned, an operand read four to six matrix instructions
// before its use; hints to the scheduler left most reads waited for at once
// (2048 tokens, 18432 keys, 24 / 4 heads of 256: 644 TFLOP/s against 889;
// 32 / 8 heads of 128: 906 against 985).  Two workgroups of 128 rows a compute
// unit were slower than one of 256 where both are full.
template <int W>
struct Many {
  static constexpr int kThreads = 64 * W, kRows = 32 * W;
};
// Waves of a workgroup, by the rows that an entry can have.  Where 128 rows do,
// two workgroups of four waves have twice the loads under way on a compute
// unit: 64 trees of 16 tokens over 4096 keys, 32 / 8 heads of 128, 212 us
// against 247 (heads of 64: 140 against 183).  A single entry loses to
// the doubled parts (32 tokens over 30000 keys: 43 us against 40).
constexpr int64_t kHalfRows = 128;
inline int many_waves(const AttnArgs& a) {
  return a.head_dim == 256 || (int64_t)a.max_q * (a.heads_q / a.heads_kv) <= kHalfRows ? 4 : 8;
}

// Weights that were taken before this point, not where they are used.
__device__ __forceinline__ void keep_here(u32x4v (&p)[2], float& sum) {
  asm volatile("" : "+v"(p[0]), "+v"(p[1]), "+v"(sum));
}

// Which workgroup does what.  A unit is (entry, row tile).
//
// Consecutive tokens: units of a head form one list, each as long as the key
// tiles it reads.  Every workgroup takes an equal run of that list, whatever
// the lengths and masks are: a run may end inside a unit, and the unit then
// goes on in the next workgroup.  Parts of units go to the workspace (a
// workgroup has at most two: the end of a unit it did not begin, in place 0 of
// its slot, and the beginning of one it does not end, in place 1).
//
// Trees: all row tiles of an entry read the same keys, far more of them than
// the caches hold, so workgroups that share keys should read them at the same
// time.  The units are cut into equal chunks of tiles, and slots run
// (entry, chunk, row tile) with the row tiles innermost.
//
// Parts are folded by the kernel after this one; whole units are written by
// the workgroup that has them.

template <int ROWS>
__device__ __forceinline__ int row_tiles_of(const Entry& e, int group) {
  return (e.n * group + ROWS - 1) / ROWS;
}

// The order of an entry's row tiles in the list: first, last, second, last but
// one, ...: under a causal mask short and long ones alternate, so no run is
// made of many short ones (each costs its start and its end).
__device__ __forceinline__ int row_tile_at(int u, int rts) { return u & 1 ? rts - 1 - (u >> 1) : u >> 1; }

template <int ROWS, bool TREE>
__device__ __forceinline__ int unit_tiles(const AttnArgs& a, const Entry& e, int rt, int group) {
  const int r0 = rt * ROWS;
  if (r0 >= e.n * group) return 0;
  // a unit without keys still writes its zeros: one empty tile
  return max(1, tile_list<kManyKeys, TREE>(a, e, r0 / group, min(e.n - 1, (r0 + ROWS - 1) / group)).count);
}

// Where the run of workgroup w begins: the u-th row tile of entry e, with
// `first` of its tiles in earlier runs.  The wave goes through the list 64
// units at a time: row tiles of one entry, or entries of a row tile count,
// whichever is fewer steps; a list of one step is gone through once.
struct Place {
  int e, u;
  int64_t first, run, left;               // left: tiles of the run, 0: none
};

template <int ROWS>
__device__ __forceinline__ Place find_place(const AttnArgs& a, int w) {
  const int lane = (int)__lane_id(), group = a.heads_q / a.heads_kv;
  const int most = (a.max_q * group + ROWS - 1) / ROWS;
  const bool by_entry = (int64_t)((a.entries + 63) / 64) * most < (int64_t)a.entries * ((most + 63) / 64);
  Place p{};
  auto entry_sum = [&](int e) {
    int n = 0;
    if (e < a.entries) {
      const Entry en = load_entry(a, e);
      const int rts = row_tiles_of<ROWS>(en, group);
      for (int rt = 0; rt < rts; ++rt) n += unit_tiles<ROWS, false>(a, en, rt, group);
    }
    return n;
  };
  auto unit_of = [&](const Entry& en, int u) {
    const int rts = row_tiles_of<ROWS>(en, group);
    return u < rts ? unit_tiles<ROWS, false>(a, en, row_tile_at(u, rts), group) : 0;
  };
  // the first step's lengths, and the length of the list
  const Entry e0 = uniform(load_entry(a, 0));
  const int mine0 = by_entry ? entry_sum(lane) : unit_of(e0, lane);
  int64_t total = 0;
  if (by_entry) {
    total = mine0;
    for (int b = 64; b < a.entries; b += 64) total += entry_sum(b + lane);
  } else {
    total = mine0;
    for (int e = 0; e < a.entries; ++e) {
      const Entry en = e ? uniform(load_entry(a, e)) : e0;
      for (int b = e ? 0 : 64; b < row_tiles_of<ROWS>(en, group); b += 64) total += unit_of(en, b + lane);
    }
  }
  total = uniform(wave_sum64(total));
  p.run = max((total + a.target - 1) / a.target, (int64_t)kManyRun);
  const int64_t want = w * p.run;
  if (want >= total) return p;
  p.left = min(p.run, total - want);
  int64_t before = 0;
  if (by_entry) {
    for (int b = 0; b < a.entries; b += 64) {
      const int mine = b ? entry_sum(b + lane) : mine0, upto = wave_scan_add(mine);
      const uint64_t hit = __ballot(before + upto > want);
      if (hit) {
        const int at = __builtin_ctzll(hit);
        p.e = b + at;
        before += __builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(mine, at);
        const Entry en = uniform(load_entry(a, p.e));
        for (; p.u < row_tiles_of<ROWS>(en, group); ++p.u) {
          const int n = unit_of(en, p.u);
          if (before + n > want) break;
          before += n;
        }
        break;
      }
      before += __builtin_amdgcn_readlane(upto, 63);
    }
  } else {
    for (; p.e < a.entries; ++p.e) {
      const Entry en = p.e ? uniform(load_entry(a, p.e)) : e0;
      bool found = false;
      for (int b = 0; b < row_tiles_of<ROWS>(en, group); b += 64) {
        const int mine = p.e + b ? unit_of(en, b + lane) : mine0, upto = wave_scan_add(mine);
        const uint64_t hit = __ballot(before + upto > want);
        if (hit) {
          const int at = __builtin_ctzll(hit);
          p.u = b + at;
          before += __builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(mine, at);
          found = true;
          break;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
      }
      if (found) break;
    }
  }
  p.first = want - before;
  return p;
}

// Slot `slot` of a tree call: entry, row tile, and which of the chunks.
struct Slot {
  int e, rt, part, parts;
  bool live;
};

template <int ROWS>
__device__ __forceinline__ int tree_tiles(const AttnArgs& a, int e, int& units) {
  const int group = a.heads_q / a.heads_kv;
  units = 0;
  if (e >= a.entries) return 0;
  const Entry en = load_entry(a, e);
  units = row_tiles_of<ROWS>(en, group);
  return units ? unit_tiles<ROWS, true>(a, en, 0, group) : 0;
}

template <int ROWS>
__device__ __forceinline__ Slot find_slot(const AttnArgs& a, const int (&tiles0)[64], const int (&units0)[64], int chunk,
                                          int64_t slot) {
  const int lane = (int)__lane_id();
  Slot s{};
  int64_t before = 0;
  for (int b = 0; b < a.entries; b += 64) {
    int tiles = tiles0[lane], units = units0[lane];
    if (b) tiles = tree_tiles<ROWS>(a, b + lane, units);
    const int parts = (tiles + chunk - 1) / chunk, mine = parts * units, upto = wave_scan_add(mine);
    const uint64_t hit = __ballot(before + upto > slot);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      const int in = (int)(slot - before) - __builtin_amdgcn_readlane(upto, at) + __builtin_amdgcn_readlane(mine, at);
      const int rts = __builtin_amdgcn_readlane(units, at);
      s.e = b + at;
      s.parts = __builtin_amdgcn_readlane(parts, at);
      s.part = __builtin_amdgcn_readfirstlane(in / rts);
      s.rt = in - s.part * rts;
      s.live = true;
      return s;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return s;
}

template <typename S, typename T, int D, int WAVES, bool TREE>
__global__ __launch_bounds__(64 * WAVES, D == 256 ? 1 : 2) void attention_many_kernel(typename S::Args a) {
  constexpr int STEPS = D / 16, DT = D / 32, KT = kManyKeys, THREADS = Many<WAVES>::kThreads;
  constexpr int ROWS = Many<WAVES>::kRows;
  constexpr int GRAN = KT * D / 8;                           // granules of one operand's tile
  constexpr int PER = GRAN / THREADS;
  // moves of a thread's share of one operand's tile: granules, or pairs of them
  // that 16 bytes of 8-bit elements hold; at one granule a thread, 8 bytes each
  constexpr int MOVES = S::PACK == 2 && PER > 1 ? PER / 2 : PER, PAIR = PER / MOVES;
  extern __shared__ __align__(16) u32x4v lds[];              // [2][keys, values][GRAN]
  __shared__ int s_bad[2];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, col = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = blockIdx.x % a.heads_kv, w = blockIdx.x / a.heads_kv, group = a.heads_q / a.heads_kv;
  const int P = 1 << a.page_log2, pmask = P - 1;
  const float c = a.scale * kLog2e;

  __shared__ int s_tiles[64], s_units[64];                   // trees: the first entries, kept out of registers
  int chunk = 1;
  Place at{};                                                // consecutive tokens
  Entry e{};
  int ei = -1;
  if constexpr (TREE) {
    const Cut cut = find_cut(a, kManyRun, [&](int x, int& tiles, int& units) { tiles = tree_tiles<ROWS>(a, x, units); });
    chunk = cut.chunk;
    if (wave == 0) {
      s_tiles[lane] = cut.tiles;
      s_units[lane] = cut.units;
    }
    lds_barrier();
  } else {
    at = find_place<ROWS>(a, w);
    at.first = uniform(at.first);
    at.left = uniform(at.left);
    at.e = __builtin_amdgcn_readfirstlane(at.e);
    at.u = __builtin_amdgcn_readfirstlane(at.u);
    // the fold reads a note of every run: none is left as the workspace had it, however the run ends
    if (h == 0 && tid == 0) a.part_note[w] = PartNote{0, 0, 0, 0, 0};
    if (at.left == 0) return;
  }
  for (int segment = 0;; ++segment) {
    int rt, first;                                           // the unit, and its tiles before this segment
    int64_t slot_at, upto;                                   // where a part goes, the tile that ends the segment
    if constexpr (TREE) {
      slot_at = w + (int64_t)segment * a.target;
      const Slot s = find_slot<ROWS>(a, s_tiles, s_units, chunk, slot_at);
      if (!s.live) {
        // notes are read for as many slots as can hold parts
        if (h == 0 && tid == 0 && segment < a.rounds) a.part_note[slot_at] = PartNote{0, 0, 0, 0, 0};
        if (segment + 1 >= a.rounds) return;
        continue;
      }
      ei = __builtin_amdgcn_readfirstlane(s.e);
      rt = __builtin_amdgcn_readfirstlane(s.rt);
      e = uniform(load_entry(a, ei));
      first = s.part * chunk;
      upto = first + chunk;
      if (h == 0 && tid == 0 && segment < a.rounds)
        a.part_note[slot_at] = s.part == 0 && s.parts > 1
                                   ? PartNote{s.parts, e.first, e.n * group, rt, row_tiles_of<ROWS>(e, group)}
                                   : PartNote{0, 0, 0, 0, 0};
    } else {
      if (at.left <= 0) return;
      if (ei < 0) e = uniform(load_entry(a, ei = at.e));
      while (at.u >= row_tiles_of<ROWS>(e, group)) {
        at.u = 0;
        if (++ei >= a.entries) return;                       // the lengths were changed under the call
        e = uniform(load_entry(a, ei));
      }
      rt = row_tile_at(at.u++, row_tiles_of<ROWS>(e, group));
      first = (int)at.first;
      at.first = 0;
      upto = first + at.left;
      slot_at = (int64_t)w * 2 + (segment != 0);
    }
    const int rows = e.n * group, r0 = rt * ROWS;
    const int i0 = r0 / group, i1 = min(e.n - 1, (r0 + ROWS - 1) / group);
    const TileList list = tile_list<KT, TREE>(a, e, i0, i1);
    const int count = max(1, list.count);
    const bool whole = first == 0 && count <= upto;
    const int t0 = __builtin_amdgcn_readfirstlane(first);
    const int t1 = __builtin_amdgcn_readfirstlane((int)min((int64_t)list.count, upto));
    if constexpr (!TREE) {
      // this run begins a unit and leaves it to others (its last segment)
      if (h == 0 && tid == 0 && first == 0 && count > upto)
        a.part_note[w] = PartNote{(int)((count - upto + at.run - 1) / at.run) + 1, e.first, e.n * group,
                                  rt << 1 | (segment != 0), 0};
      at.left -= min(upto, (int64_t)count) - first;
    }

    const int row = r0 + wave * 32 + col;
    RowMask mask;
    // What all rows of the workgroup see (their values need no cleaning), and
    // what all rows of the wave see.
    const OpenKeys seen_by_all = open_keys<TREE>(a, e, i0, i1);
    const int w0 = r0 + wave * 32, j0 = min(w0, rows - 1) / group, j1 = min(w0 + 31, rows - 1) / group;
    const OpenKeys seen_by_wave = open_keys<TREE>(a, e, j0, j1);
    u32x4v q[STEPS];
    {
      const bool live = row < rows;
      const int i = live ? row / group : 0, hq = h * group + (live ? row % group : 0);
      mask = row_mask<TREE>(a, e, i, live);
      const uint16_t* src = a.q + (int64_t)(e.first + i) * a.q_stride + (int64_t)hq * D + half * 8;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) q[s] = *reinterpret_cast<const u32x4v*>(src + s * 16);
    }
    f32x16 o[DT];
#pragma unroll
    for (int t = 0; t < DT; ++t) o[t] = f32x16{};
    Running st{-INFINITY, 0.0f};

    // A thread's granules on their way to LDS: of the keys one tile, of the
    // values the tile before it.
    typedef typename std::conditional<S::PACK == 1 || PAIR == 2, u32x4v, u32x2v>::type Move;
    Move in_k[MOVES], in_v[MOVES];
    // Kv8: the scale of each key's block, one key a lane, of the tiles in the
    // registers above and of the ones that are loaded next
    uint32_t ke = 0, ve = 0, next_ke = 0, next_ve = 0;
    // The page of each of a tile's keys, one key a lane.
    auto pages_of = [&](int t) {
      const int key = list.key<KT>(min(t, t1 - 1)) + lane;
      return e.pages[min(key >> a.page_log2, (int)a.width - 1)];
    };
    const uint32_t page_elems = (uint32_t)(a.heads_kv * D) << a.page_log2, head_at = (uint32_t)(h * D) << a.page_log2;
    // keys: granule g of the tile is dimension block g / 64 of key g % 64, so
    // a thread keeps its key
    auto keys_at = [&](int t, int32_t page) {
      const int key = (list.key<KT>(min(t, t1 - 1)) + lane) & pmask;
      const uint64_t head = (uint64_t)page_in_pool(page, a.pages) * page_elems + head_at;
      if constexpr (S::PACK == 1) {
        return a.k + head + (key + wave * P) * 8;
      } else {
        next_ke = a.k_scale[head / (D * 16) + (key >> 4)];
        const uint8_t* k = reinterpret_cast<const uint8_t*>(a.k) + head;
        return PAIR == 2 ? k + (key + wave * P) * 16 : k + (key + (wave >> 1) * P) * 16 + (wave & 1) * 8;
      }
    };
    auto load_keys = [&](auto at, int n) {
      in_k[n] = *reinterpret_cast<const Move*>(at + n * WAVES * P * 8 * S::PACK);
    };
    // values: granule g is token block g / D of dimension g % D, one token
    // block a wave, whose address the lane of the block's first key works out
    auto values_at = [&](int t, int32_t page) {
      const int key = (list.key<KT>(min(t, t1 - 1)) + lane) & pmask;
      const uint64_t head = (uint64_t)page_in_pool(page, a.pages) * page_elems + head_at;
      if constexpr (S::PACK == 1) {
        return (uint64_t)(a.v + head + (key >> 3) * D * 8);
      } else {
        next_ve = a.v_scale[head / (D * 16) + (key >> 4)];
        return (uint64_t)(reinterpret_cast<const uint8_t*>(a.v) + head + (key >> 4) * D * 16);
      }
    };
    auto load_values = [&](uint64_t at, int n) {
      const int g = n * THREADS + wave * 64, from = g / D * 8 * PAIR;
      const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)at, from);
      const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(at >> 32), from);
      const auto rsrc =
          __builtin_amdgcn_make_buffer_rsrc((void*)(((uint64_t)hi << 32) | lo), 0, D * 16, kRawBufferWord3);
      if constexpr (S::PACK == 1 || PAIR == 2)
        in_v[n] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, lane * 16, g % D * 16, 0);
      else
        in_v[n] = __builtin_amdgcn_raw_buffer_load_b64(rsrc, lane * 16, g % D * 16 + (g / D & 1) * 8, 0);
    };
    // a move into its tile's place in LDS
    auto store_keys = [&](u32x4v* tile, int n) __attribute__((always_inline)) {
      if constexpr (S::PACK == 1) {
        tile[n * THREADS + tid] = in_k[n];
      } else {
        const float scale = S::scale(ke);
        u32x4v* at = tile + (n * WAVES + wave) * PAIR * KT + lane;
#pragma unroll
        for (int x = 0; x < PAIR; ++x) at[x * KT] = S::template widen<T>(in_k[n], x, scale);
      }
    };
    auto store_values = [&](u32x4v* tile, int n) __attribute__((always_inline)) {
      if constexpr (S::PACK == 1) {
        tile[n * THREADS + tid] = in_v[n];
      } else {
        const int g = n * THREADS + wave * 64;
        const float scale = S::scale((uint32_t)__builtin_amdgcn_readlane((int)ve, g / D * 8 * PAIR));
        u32x4v* at = tile + g / D * PAIR * D + g % D + lane;
#pragma unroll
        for (int x = 0; x < PAIR; ++x) at[x * D] = S::template widen<T>(in_v[n], x, scale);
      }
    };
    auto rescale = [&](float alpha) {
      settle(o);
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[d][r] *= alpha;
      settle(o);
    };

    if (tid < 2) s_bad[tid] = -1;
    int32_t page_v = 0, page_k = 0;                          // pages of the tiles that are loaded next
    uint64_t held = 0;                                       // a tile's keys whose page is there
    if (t0 < t1) {
      const int32_t page = pages_of(t0), after = pages_of(t0 + 1);
      page_v = after;
      page_k = pages_of(t0 + 2);
      held = __ballot(page_ok(page, a.pages));
      auto kp = keys_at(t0, page);
      ke = next_ke;
#pragma unroll
      for (int n = 0; n < MOVES; ++n) load_keys(kp, n);
#pragma unroll
      for (int n = 0; n < MOVES; ++n) store_keys(lds, n);
      waitcnt_vm<0>();       // q has arrived too: waits inside the loop are for the tiles' loads only
      kp = keys_at(t0 + 1, after);
      const uint64_t vp = values_at(t0, page);
#pragma unroll
      for (int n = 0; n < MOVES; ++n) load_keys(kp, n);
#pragma unroll
      for (int n = 0; n < MOVES; ++n) load_values(vp, n);
      ke = next_ke;
      ve = next_ve;
    }
    lds_barrier();
    const int krow = tile_key_of_row(col);
    const bool has_rows = w0 < rows;
    f32x16 sa, sb;                                           // scores of a tile's first and second block
    u32x4v pa[2], pb[2];                                     // and their weights
    bool open = true;
    uint32_t seen_b = 0;
    // Period t: scores of tile t, the product with the values of tile t - 1.
    auto period = [&](int t, auto is_first, auto is_last) __attribute__((always_inline)) {
      constexpr bool FIRST = decltype(is_first)::value, LAST = decltype(is_last)::value;
      const int buf = (t - t0) & 1, kb = list.key<KT>(t);
      const u32x4v* kt = lds + buf * 2 * GRAN + half * KT + krow;              // [2 s + half][32 x + key]
      const u32x4v* vt = lds + ((buf ^ 1) * 2 + 1) * GRAN + half * D + col;    // [4 x + 2 s + half][dimension]
      // A quarter of the staging: tile t + 1's keys and tile t's values go to
      // LDS, and their registers take the loads of the tiles after them.
      // Past the end the last tile is read again.
      decltype(keys_at(0, 0)) kp = nullptr;
      uint64_t vp = 0;
      const uint64_t here = held;
      if constexpr (!LAST) {
        held = __ballot(page_ok(page_v, a.pages));
        kp = keys_at(t + 2, page_k);
        vp = values_at(t + 1, page_v);
        page_v = page_k;
        page_k = pages_of(t + 3);
      }
      auto stage = [&](int i) __attribute__((always_inline)) {
        if (i < MOVES) {
          store_keys(lds + (buf ^ 1) * 2 * GRAN, i);
          load_keys(kp, i);
        } else {
          store_values(lds + (buf * 2 + 1) * GRAN, i - MOVES);
          load_values(vp, i - MOVES);
        }
      };
      if (!has_rows) {
        if constexpr (!LAST) {
#pragma unroll
          for (int i = 0; i < 2 * MOVES; ++i) stage(i);
        }
      } else {
        // The period's matrix instructions in order, in quarters: scores of
        // this tile's first block, product of the first block before, scores
        // of the second block, product of the second block before.  A slot is
        // one of them, the operand read AHEAD slots later, and its share of
        // what else the quarter has to do.  The order is pinned: left to
        // itself every read is waited for where it stands.
        constexpr int N = STEPS, TOTAL = FIRST || LAST ? 2 * N : 4 * N, AHEAD = D == 256 ? 6 : 4;
        auto quarter = [](int j) { return FIRST ? j / N * 2 : LAST ? j / N * 2 + 1 : j / N; };
        auto read = [&](int j) __attribute__((always_inline)) {
          const int at = quarter(j), i = j % N, x = (at >> 1) * 32;
          return at & 1 ? vt[((at >> 1) * 4 + 2 * (i / DT)) * D + i % DT * 32] : kt[2 * i * KT + x];
        };
        u32x4v f[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) f[j] = read(j);
        auto run = [&](auto which, auto&& extra) __attribute__((always_inline)) {
          constexpr int Q = decltype(which)::value, FROM = (FIRST || LAST ? Q / 2 : Q) * N;
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int j = FROM + i;
            u32x4v& operand = f[j % AHEAD];
            if (Q == 0) sa = T::mfma(operand, q[i], sa);
            if (Q == 1) o[i % DT] = T::mfma(operand, pa[i / DT], o[i % DT]);
            if (Q == 2) sb = T::mfma(operand, q[i], sb);
            if (Q == 3) o[i % DT] = T::mfma(operand, pb[i / DT], o[i % DT]);
            if (j + AHEAD < TOTAL) operand = read(j + AHEAD);
            extra(i);
            if constexpr (!LAST) {
              // the moves of this quarter (two quarters where the others are left out)
              constexpr int M0 = (FIRST ? Q / 2 * 2 : Q) * MOVES / 2, M1 = (FIRST ? Q / 2 * 2 + 2 : Q + 1) * MOVES / 2;
#pragma unroll
              for (int m = M0 + i * (M1 - M0) / N; m < M0 + (i + 1) * (M1 - M0) / N; ++m) stage(m);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        };
        constexpr std::integral_constant<int, 0> Q0{};
        constexpr std::integral_constant<int, 1> Q1{};
        constexpr std::integral_constant<int, 2> Q2{};
        constexpr std::integral_constant<int, 3> Q3{};
        float top = -INFINITY, alpha = 1.0f, sum = 0.0f;
        bool moved = false;
        // the row maximum of a block, done after half a quarter
        auto maximum = [&](const f32x16& s, int i) __attribute__((always_inline)) {
          constexpr int E = 32 / N;
          if (i < N / 2) {
#pragma unroll
            for (int e = i * E; e < (i + 1) * E; e += 2) top = fmaxf(top, fmaxf(s[e], s[e + 1]));
          } else if (i == N / 2) {
            top = max_of_halves(top) * c;
          }
        };
        auto weights = [&](const f32x16& s, u32x4v (&p)[2], int i) __attribute__((always_inline)) {
          constexpr int E = 16 / N;
#pragma unroll
          for (int e = i * E; e < (i + 1) * E; ++e) weigh_one<T>(s, c, st, e, sum, p);
        };
        if (!FIRST && !open) cut_scores(sb, seen_b);
        if constexpr (!LAST) {
          sa = f32x16{};
          if constexpr (FIRST)
            run(Q0, [](int) {});
          else
            run(Q0, [&](int i) __attribute__((always_inline)) { maximum(sb, i); });
        } else {
          top = row_top(sb, c);
        }
        if constexpr (!FIRST) {
          moved = must_move(top, st);
          if (moved) alpha = move_bound(top, st);
          run(Q1, [&](int i) __attribute__((always_inline)) { weights(sb, pb, i); });
          keep_here(pb, sum);
          if (moved) rescale(alpha);                         // what went before was weighed with the earlier bound
          st.l += sum;
        }
        if constexpr (!LAST) {
          open = seen_by_wave.tile(kb, KT) && here == ~0ull;
          if (!open) {
            const uint64_t seen = mask.template bits<TREE>(kb) & here;
            cut_scores(sa, (uint32_t)seen);
            seen_b = (uint32_t)(seen >> 32);
          }
          sb = f32x16{};
          top = -INFINITY;
          alpha = 1.0f;
          sum = 0.0f;
          run(Q2, [&](int i) __attribute__((always_inline)) { maximum(sa, i); });
          moved = must_move(top, st);
          if (moved) alpha = move_bound(top, st);
        }
        if constexpr (FIRST) {
          sum = weigh<T>(sa, c, st, pa);
        } else if constexpr (LAST) {
          run(Q3, [](int) {});
        } else {
          run(Q3, [&](int i) __attribute__((always_inline)) { weights(sa, pa, i); });
        }
        if constexpr (!LAST) {
          keep_here(pa, sum);
          if (!FIRST && moved) rescale(alpha);
          st.l += sum;
        }
        settle(o);
        if constexpr (!FIRST) {
          if (s_bad[buf ^ 1] == t - 1) {
            S::template put_back<T, D, TREE>(a, head_at, h, e.pages, page_elems, mask, list.key<KT>(t - 1), KT, o);
            settle(o);
          }
        }
      }
      if constexpr (S::PACK == 2 && !LAST) {
        ke = next_ke;
        ve = next_ve;
      }
      lds_barrier();
      // A tile that some row does not see in full has its values cleaned in
      // place before they are used; s_bad: the last tile where that changed any.
      if constexpr (!LAST) {
        if (!seen_by_all.tile(kb, KT) || here != ~0ull) {
          u32x4v v[PER];
          u32x4v* own = lds + (buf * 2 + 1) * GRAN + tid;
#pragma unroll
          for (int n = 0; n < PER; ++n) v[n] = own[n * THREADS];
          if (drop_nonfinite<T>(v)) s_bad[buf] = t;
#pragma unroll
          for (int n = 0; n < PER; ++n) own[n * THREADS] = v[n];
          lds_barrier();
        }
      }
    };
    if (t0 < t1) {
      constexpr std::true_type yes{};
      constexpr std::false_type no{};
      period(t0, yes, no);
      for (int t = t0 + 1; t < t1; ++t) period(t, no, no);
      period(t1, no, yes);
    }

    settle(o);
    const float l = st.l + __shfl_xor(st.l, 32);
    // Outputs of whole units go through LDS, where a wave's rows lie as they do
    // in memory (granules of 16 bytes, turned by the row against bank
    // conflicts), and leave as whole rows.  Parts are only read by the fold:
    // they lie as the registers do, a wave's 64 lanes side by side.
    int olane = lane;
    asm volatile("" : "+v"(olane));          // the lane's addresses are worked out here, not kept through the loop
    const int ocol = olane & 31, ohalf = olane >> 5;
    if (has_rows && whole) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      constexpr int GRANS = D / 8;
      uint16_t* tile = reinterpret_cast<uint16_t*>(lds) + wave * 32 * D;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<u32x2v*>(tile + ocol * D + ((d * 4 + j) ^ (ocol & 7)) * 8 + ohalf * 4) =
              u32x2v{T::pack(o[d][4 * j] * inv, o[d][4 * j + 1] * inv), T::pack(o[d][4 * j + 2] * inv, o[d][4 * j + 3] * inv)};
#pragma unroll
      for (int n = 0; n < GRANS / 2; ++n) {
        const int r = (n * 64 + olane) / GRANS, g = (n * 64 + olane) % GRANS, at = w0 + r;
        const u32x4v x = *reinterpret_cast<const u32x4v*>(tile + r * D + (g ^ (r & 7)) * 8);
        const int i = at / group;
        if (at < rows)
          *reinterpret_cast<u32x4v*>(a.out + ((int64_t)(e.first + i) * a.heads_q + h * group + at - i * group) * D + g * 8) = x;
      }
    } else if (has_rows) {
      const int64_t slot = (slot_at * a.heads_kv + h) * ROWS + wave * 32;
      if (ohalf == 0) *reinterpret_cast<f32x2p*>(a.part_ml + (slot + ocol) * 2) = f32x2p{st.m, l};
      float* part = a.part_o + slot * D + olane * 4;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<f32x4v*>(part + (d * 4 + j) * 256) =
              f32x4v{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
    }
    lds_barrier();                                           // the next segment's tiles take the same place
  }
}

// ---- fold ----------------------------------------------------------------
// o = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s over the parts s of a row.
// A part with m_s = -inf has a factor of zero, but is not left out: o_s and l_s
// are zeros where the row sees no key of it, and NaN where every score that it
// sees there is NaN (the maximum passes over those).

// Few rows: notes by entry; parts are consecutive slots of 32 rows a head.  One
// row a workgroup; D / 4 lanes take its dimensions and read its (m, l) pairs
// side by side, and the 1024 / D groups of lanes take the parts in turn.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attention_fold_few_kernel(AttnArgs a) {
  constexpr int LANES = D / 4, GROUPS = kThreads / LANES, BATCH = 8;
  const PartNote note = a.part_note[blockIdx.x];
  if (note.parts == 0) return;
  const int gl = threadIdx.x % LANES, g = threadIdx.x / LANES, d = gl * 4;
  const int h = blockIdx.z, group = a.heads_q / a.heads_kv, row = blockIdx.y;
  if (row >= note.rows) return;
  auto slot = [&](int s) -> int64_t { return ((int64_t)(note.place + s) * a.heads_kv + h) * kFewRows + row; };
  float top = -INFINITY;
  for (int s = gl; s < note.parts; s += LANES) top = fmaxf(top, a.part_ml[slot(s) * 2]);
#pragma unroll
  for (int x = LANES / 2; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
  f32x4v acc = {};
  float sum = 0.0f;
  for (int base = 0; base < note.parts; base += LANES) {
    float f = 0.0f;
    if (base + gl < note.parts) {
      const f32x2p ml = *reinterpret_cast<const f32x2p*>(a.part_ml + slot(base + gl) * 2);
      f = ml[0] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml[0] - top);
      sum += f * ml[1];
    }
    const int n = min(LANES, note.parts - base);
    for (int s0 = 0; s0 < n; s0 += GROUPS * BATCH) {
      f32x4v x[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int s = s0 + k * GROUPS + g;
        x[k] = f32x4v{};
        if (s < n) x[k] = *reinterpret_cast<const f32x4v*>(a.part_o + slot(base + s) * D + d);
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int s = s0 + k * GROUPS + g;
        const float got = __shfl(f, s % LANES, LANES), fs = s < n ? got : 0.0f;
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[v] += fs * x[k][v];
      }
    }
  }
#pragma unroll
  for (int x = LANES / 2; x; x >>= 1) sum += __shfl_xor(sum, x);
  __shared__ f32x4v s_acc[kThreads];
  s_acc[threadIdx.x] = acc;
  __syncthreads();
  if (g) return;
  for (int o = 1; o < GROUPS; ++o) acc += s_acc[o * LANES + gl];
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint16_t* dst = a.out + ((int64_t)(note.first + row / group) * a.heads_q + h * group + row % group) * D + d;
  *reinterpret_cast<u32x2v*>(dst) = u32x2v{T::pack(acc[0] * inv, acc[1] * inv), T::pack(acc[2] * inv, acc[3] * inv)};
}

// Many rows, trees: notes by the slot of the first part, parts every `step`
// slots.  Consecutive tokens: notes by the run that begins the unit; the first
// part is in place 0 or 1 of that run, the others in place 0 of the runs after
// it.  A wave takes 32 rows and one granule of 8 dimensions, as its lanes lie
// in the parts; the workgroup's four granules leave together.  Notes are the
// slowest dimension of the grid: most of a short call's are empty, and as the
// fastest they left its work to one XCD (one tree of 64 tokens, 4096 keys,
// 32 / 8 heads of 128: 34 us).
template <typename T, int D, int WAVES, bool TREE>
__global__ __launch_bounds__(kThreads) void attention_fold_many_kernel(AttnArgs a) {
  constexpr int ROWS = Many<WAVES>::kRows, BATCH = 8;
  const PartNote note = a.part_note[blockIdx.z];
  if (note.parts == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 31, half = lane >> 5;
  const int h = blockIdx.y, group = a.heads_q / a.heads_kv;
  const int block = blockIdx.x / (D / 32), gran = blockIdx.x % (D / 32) * 4 + wave;
  const int r0 = (TREE ? note.place : note.place >> 1) * ROWS + block * 32;
  if (r0 >= note.rows) return;
  auto slot = [&](int s) -> int64_t {
    const int64_t at = TREE ? (int64_t)blockIdx.z + (int64_t)s * note.step
                            : ((int64_t)blockIdx.z + s) * 2 + (s ? 0 : note.place & 1);
    return (at * a.heads_kv + h) * ROWS + block * 32;
  };
  f32x4v acc = {};
  float top = -INFINITY, sum = 0.0f;
  const bool live = r0 + col < note.rows;                    // rows past the end were not written
  for (int s0 = 0; s0 < note.parts; s0 += BATCH) {
    f32x2p ml[BATCH];
    f32x4v x[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      ml[k] = f32x2p{-INFINITY, 0.0f};
      x[k] = f32x4v{};
      if (s0 + k >= note.parts) continue;
      const int64_t at = slot(s0 + k);
      ml[k] = *reinterpret_cast<const f32x2p*>(a.part_ml + (at + col) * 2);
      x[k] = *reinterpret_cast<const f32x4v*>(a.part_o + at * D + gran * 256 + lane * 4);
    }
    float up = top;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) up = fmaxf(up, ml[k][0]);
    const float down = up == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(top - up);
    top = up;
    sum *= down;
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] *= down;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const float f = ml[k][0] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml[k][0] - up);
      sum += f * ml[k][1];
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[v] += f * x[k][v];
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  __shared__ u32x2v s_out[32][8 + 1];
  if (live)
    s_out[col][wave * 2 + half] =
        u32x2v{T::pack(acc[0] * inv, acc[1] * inv), T::pack(acc[2] * inv, acc[3] * inv)};
  __syncthreads();
  const int r = tid >> 3, g = tid & 7, i = (r0 + r) / group;
  if (r0 + r < note.rows)
    *reinterpret_cast<u32x2v*>(a.out + ((int64_t)(note.first + i) * a.heads_q + h * group + r0 + r - i * group) * D +
                               blockIdx.x % (D / 32) * 32 + g * 4) = s_out[r][g];
}

bool few_rows(const AttnArgs& a) { return (int64_t)a.max_q * (a.heads_q / a.heads_kv) <= kFewRows; }

// Workgroups per key head that the few-row kernel's cut aims at: as many as
// run at once, over the heads.
int few_target(const AttnArgs& a) {
  const int resident = device_cus() * (a.head_dim == 256 ? 1 : 2);
  return resident / a.heads_kv > 1 ? resident / a.heads_kv : 1;
}
// Rounds of slots: more than one only where entries are many against the target.
int rounds_of(const AttnArgs& a, int target) { return 2 * (int64_t)a.entries > target ? kRounds : 1; }

int64_t few_slots(const AttnArgs& a) {
  const int64_t slots = (int64_t)rounds_of(a, few_target(a)) * few_target(a);
  return slots > a.entries ? slots : a.entries;
}

// Runs per key head of the many-row kernel: the workgroups that run at once,
// over the heads.  (At D = 64 two of eight waves would fit the LDS but not the
// registers; cut for two, 64 tokens over 30000 keys, 32 / 8 heads, took 56 us
// against 44.)
int many_target(const AttnArgs& a) {
  const int resident = device_cus() * (a.head_dim != 256 && many_waves(a) == 4 ? 2 : 1);
  return resident / a.heads_kv > 1 ? resident / a.heads_kv : 1;
}
size_t round256(size_t v) { return (v + 255) / 256 * 256; }

// The workspace: partial outputs, (m, l) pairs, notes.
struct Parts {
  size_t o, ml, notes;
};

Parts part_bytes(const AttnArgs& a) {
  int64_t slots, rows;                                       // notes; rows of partial outputs a head
  if (few_rows(a)) {
    slots = few_slots(a);
    rows = slots * kFewRows;
  } else {
    const int64_t of_slot = 32 * many_waves(a);
    slots = (int64_t)many_target(a) * (a.tree ? rounds_of(a, many_target(a)) : 1);
    rows = slots * (a.tree ? 1 : 2) * of_slot;
  }
  rows *= a.heads_kv;
  return {round256((size_t)rows * a.head_dim * 4), round256((size_t)rows * 8), round256((size_t)slots * sizeof(PartNote))};
}

template <typename S, typename T, int D, int WAVES, bool TREE>
hipError_t launch_many(typename S::Args& a, hipStream_t stream) {
  constexpr size_t lds = 2 * 2 * (size_t)kManyKeys * D * 2;
  static LdsLimit limit;
  const hipError_t e = limit.raise(reinterpret_cast<const void*>(&attention_many_kernel<S, T, D, WAVES, TREE>), lds);
  if (e != hipSuccess) return e;
  a.target = many_target(a);
  a.rounds = rounds_of(a, a.target);
  attention_many_kernel<S, T, D, WAVES, TREE><<<(unsigned)(a.target * a.heads_kv), Many<WAVES>::kThreads, lds, stream>>>(a);
  const unsigned notes = (unsigned)(TREE ? a.target * a.rounds : a.target);
  attention_fold_many_kernel<T, D, WAVES, TREE><<<dim3(Many<WAVES>::kRows * D / (4 * kThreads), a.heads_kv, notes), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename S, typename T, int D, bool TREE>
hipError_t launch_typed(typename S::Args& a, hipStream_t stream) {
  if (few_rows(a)) {
    a.target = few_target(a);
    a.rounds = rounds_of(a, a.target);
    const unsigned slots = (unsigned)few_slots(a), rows = (unsigned)(a.max_q * (a.heads_q / a.heads_kv));
    attention_few_kernel<S, T, D, TREE><<<dim3(slots, a.heads_kv), kThreads, 0, stream>>>(a);
    attention_fold_few_kernel<T, D><<<dim3(a.entries, rows, a.heads_kv), kThreads, 0, stream>>>(a);
    return hipGetLastError();
  }
  if constexpr (D != 256)
    if (many_waves(a) == 8) return launch_many<S, T, D, 8, TREE>(a, stream);
  return launch_many<S, T, D, 4, TREE>(a, stream);
}

template <typename S, typename T, int D>
hipError_t launch_masked(typename S::Args& a, hipStream_t stream) {
  return a.tree ? launch_typed<S, T, D, true>(a, stream) : launch_typed<S, T, D, false>(a, stream);
}

template <typename S, typename T>
hipError_t launch_dim(typename S::Args& a, hipStream_t stream) {
  switch (a.head_dim) {
    case 64: return launch_masked<S, T, 64>(a, stream);
    case 128: return launch_masked<S, T, 128>(a, stream);
    default: return launch_masked<S, T, 256>(a, stream);
  }
}

// Fills in the workspace's parts and launches.
template <typename S>
hipError_t launch_store(typename S::Args& a, void* workspace, hipStream_t stream) {
  const Parts p = part_bytes(a);
  char* w = reinterpret_cast<char*>(workspace);
  a.part_o = reinterpret_cast<float*>(w);
  a.part_ml = reinterpret_cast<float*>(w + p.o);
  a.part_note = reinterpret_cast<PartNote*>(w + p.o + p.ml);
  return a.fp16 ? launch_dim<S, F16>(a, stream) : launch_dim<S, Bf16>(a, stream);
}

}  // namespace

}  // namespace trellis
