// attention.hip -- attention of new tokens over the paged cache: the kernel
// for few rows per key head (decoding, small trees), the kernel for many
// (prompt chunks, wide trees), and the fold of split keys.
#include "attention.hpp"
#include "copy_ring.hpp"

namespace trellis {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kFewRows = 32;              // rows of the few-row kernel: one MFMA tile
constexpr int kManyRows = 128;            // rows of a many-row workgroup: 32 a wave
constexpr int kManyKeys = 64;             // keys of a tile of the many-row kernel

// ---- few rows ------------------------------------------------------------
// All rows of an entry that share a key head (tokens x query heads per key
// head, at most 32) are one MFMA tile, so keys and values are read once,
// straight into operand registers.  The keys of all entries are cut into
// chunks of `chunk` tiles, chosen from the sum of the entries' tiles so that
// about `target` workgroups per key head have equal work however unlike the
// lengths are.  Every workgroup computes the same cut from the lengths.

struct Unit {
  int e, split, splits, chunk, base;
  bool live;
};

template <bool TREE>
__device__ __forceinline__ int entry_tiles(const AttnArgs& a, int e) {
  if (e >= a.entries) return 0;
  const Entry en = load_entry(a, e);
  if (en.n == 0) return 0;
  return max(1, tile_list<32, TREE>(a, en, 0, en.n - 1).count);
}

// Slot -> (entry, split), or with by_entry: entry -> its slots.
template <bool TREE>
__device__ __forceinline__ Unit find_unit(const AttnArgs& a, int want, bool by_entry) {
  const int lane = (int)__lane_id();
  Unit u;
  u.live = false;
  u.e = u.split = u.splits = u.base = 0;
  int tiles = entry_tiles<TREE>(a, lane);
  int total = wave_sum(tiles);
  for (int b = 64; b < a.entries; b += 64) total += wave_sum(entry_tiles<TREE>(a, b + lane));
  u.chunk = max(kWaves, (total + a.target - 1) / a.target);
  int before = 0;
  for (int b = 0; b < a.entries; b += 64) {
    if (b) tiles = entry_tiles<TREE>(a, b + lane);
    const int parts = (tiles + u.chunk - 1) / u.chunk;
    const int upto = wave_scan_add(parts);
    const int last = __shfl(upto, 63);
    const uint64_t hit = by_entry ? (want - b < 64 ? 1ull << (want - b) : 0ull)
                                  : __ballot(before + upto > want);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      u.e = b + at;
      u.splits = __shfl(parts, at);
      u.base = before + __shfl(upto, at) - u.splits;
      u.split = by_entry ? 0 : want - u.base;
      u.live = u.splits > 0;
      return u;
    }
    before += last;
  }
  return u;
}

template <typename T, int D, bool TREE>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void attention_few_kernel(AttnArgs a) {
  constexpr int STEPS = D / 16, DT = D / 32;
  __shared__ float s_m[kWaves][32], s_l[kWaves][32];
  __shared__ __align__(16) float s_o[kWaves][32][36];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, col = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Unit u = find_unit<TREE>(a, blockIdx.x, false);
  if (!u.live) return;
  const Entry e = uniform(load_entry(a, u.e));
  const int h = blockIdx.y, group = a.heads_q / a.heads_kv, rows = e.n * group;
  const TileList list = tile_list<32, TREE>(a, e, 0, e.n - 1);
  const int t0 = u.split * u.chunk, t1 = min(list.count, t0 + u.chunk);
  const int P = 1 << a.page_log2, pmask = P - 1;

  const bool live = col < rows;
  const int i = live ? col / group : 0, hq = h * group + (live ? col % group : 0);
  const RowMask mask = row_mask<TREE>(a, e, i, live);
  const OpenKeys seen_by_all = open_keys<TREE>(a, e, 0, e.n - 1);
  u32x4v q[STEPS];
  {
    const uint16_t* src = a.q + (int64_t)(e.first + i) * a.q_stride + (int64_t)hq * D + half * 8;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) q[s] = *reinterpret_cast<const u32x4v*>(src + s * 16);
  }

  f32x16 o[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t) o[t] = f32x16{};
  Running st{-INFINITY, 0.0f};
  const float c = a.scale * kLog2e;
  const int64_t head_elems = (int64_t)D << a.page_log2;      // one head's page
  const int krow = tile_key_of_row(col);

  for (int t = t0 + wave; t < t1; t += kWaves) {
    const int kb = list.key<32>(t);
    const int p0 = kb >> a.page_log2, p1 = (kb + 16) >> a.page_log2;
    const int64_t g0 = ((int64_t)page_in_pool(e.pages[min(p0, (int)a.width - 1)], a.pages) * a.heads_kv + h) * head_elems;
    const int64_t g1 = ((int64_t)page_in_pool(e.pages[min(p1, (int)a.width - 1)], a.pages) * a.heads_kv + h) * head_elems;
    const uint16_t* kp = a.k + (krow >= 16 ? g1 : g0) + (((kb + krow) & pmask) + half * P) * 8;
    u32x4v kf[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) kf[s] = *reinterpret_cast<const u32x4v*>(kp + (int64_t)s * 16 * P);
    u32x4v vf[2][DT];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int key = kb + s * 16 + half * 8;
      const uint16_t* vp = a.v + (s ? g1 : g0) + (int64_t)((key & pmask) >> 3) * D * 8 + col * 8;
#pragma unroll
      for (int d = 0; d < DT; ++d) vf[s][d] = *reinterpret_cast<const u32x4v*>(vp + d * 256);
    }
    f32x16 sc[1] = {f32x16{}};
#pragma unroll
    for (int s = 0; s < STEPS; ++s) sc[0] = T::mfma(kf[s], q[s], sc[0]);
    const bool open = seen_by_all.tile(kb, 32);
    if (!open) cut_scores(sc[0], (uint32_t)mask.bits<TREE>(kb));
    float alpha;
    if (move_bound(sc, c, st, alpha)) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[d][r] *= alpha;
    }
    weigh(sc, c, st);
    bool bad = false;
    if (!open) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int d = 0; d < DT; ++d) bad |= drop_nonfinite<T>(vf[s][d]);
    }
    u32x4v p[2];
    pack_weights<T>(sc[0], p);
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int s = 0; s < 2; ++s) o[d] = T::mfma(vf[s][d], p[s], o[d]);
    if (__any(bad))
      add_nonfinite<T, D, TREE>(a.v + h * head_elems, e.pages, a.pages, (uint32_t)(a.heads_kv * head_elems),
                                a.page_log2, mask, kb, 32, o);
  }

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
    osum += s_m[w][orow] == -INFINITY ? 0.0f : s_l[w][orow] * __builtin_amdgcn_exp2f(s_m[w][orow] - otop);
  const bool whole = u.splits == 1;
  const float inv = whole ? (osum == 0.0f ? 0.0f : 1.0f / osum) : 1.0f;
  const int64_t slot = (int64_t)blockIdx.x * a.heads_kv + h;
  const bool owrite = orow < rows;
  uint16_t* dst = a.out + ((int64_t)(e.first + orow / group) * a.heads_q + h * group + orow % group) * D + od;
  float* part = a.part_o + (slot * kFewRows + orow) * D + od;
#pragma unroll
  for (int d = 0; d < DT; ++d) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<f32x4v*>(&s_o[wave][col][8 * j + 4 * half]) =
          f32x4v{o[d][4 * j] * f, o[d][4 * j + 1] * f, o[d][4 * j + 2] * f, o[d][4 * j + 3] * f};
    __syncthreads();
    f32x4v sum = *reinterpret_cast<const f32x4v*>(&s_o[0][orow][od]);
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += *reinterpret_cast<const f32x4v*>(&s_o[w][orow][od]);
    if (owrite) {
      if (whole)
        *reinterpret_cast<u32x2v*>(dst + d * 32) =
            u32x2v{T::pack(sum[0] * inv, sum[1] * inv), T::pack(sum[2] * inv, sum[3] * inv)};
      else
        *reinterpret_cast<f32x4v*>(part + d * 32) = sum;
    }
    __syncthreads();
  }
  if (!whole && owrite && (tid & 7) == 0)
    *reinterpret_cast<f32x2p*>(a.part_ml + (slot * kFewRows + orow) * 2) = f32x2p{otop, osum};
}

// ---- many rows -----------------------------------------------------------
// A workgroup takes 128 rows (token-major, the query heads of one key head
// innermost), 32 a wave, and walks its keys in tiles of 64 that all waves
// share through LDS, in the cache's own granule order, so LDS reads are
// contiguous across lanes and nothing is transposed.
//
// A tile is two blocks of 32 keys.  The second block's scores are computed
// under the first block's exponentials, and the first block's product with the
// values under the second's: the vector work of the softmax (over half of it
// exponentials) is about as long as the matrix instructions at D = 128.

// Let every matrix instruction of a block be followed by vector ones (a
// scheduling hint for the code around it).
template <int MFMAS, int VALU, int TRANS>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < MFMAS; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
    __builtin_amdgcn_sched_group_barrier(0x400, TRANS, 0);
  }
}

template <typename T, int D, bool TREE>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void attention_many_kernel(AttnArgs a) {
  constexpr int STEPS = D / 16, DT = D / 32, KT = kManyKeys;
  constexpr int GRAN = KT * D / 8;                           // granules of one operand's tile
  constexpr int PER = GRAN / kThreads;
  extern __shared__ __align__(16) u32x4v lds[];              // [2][keys, values][GRAN]
  __shared__ int s_bad[2];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, col = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int split = blockIdx.x % a.splits, rt = gridDim.x / a.splits - 1 - blockIdx.x / a.splits;
  const int h = blockIdx.y, group = a.heads_q / a.heads_kv;
  const Entry e = uniform(load_entry(a, blockIdx.z));
  const int rows = e.n * group, r0 = rt * kManyRows;
  if (r0 >= rows) return;
  const int i0 = r0 / group, i1 = min(e.n - 1, (r0 + kManyRows - 1) / group);
  const TileList list = tile_list<KT, TREE>(a, e, i0, i1);
  const int chunk = (list.count + a.splits - 1) / a.splits;
  const int t0 = split * chunk, t1 = min(list.count, t0 + chunk);
  const int P = 1 << a.page_log2, pmask = P - 1;

  const int row = r0 + wave * 32 + col;
  const bool live = row < rows;
  const int i = live ? row / group : 0, hq = h * group + (live ? row % group : 0);
  const RowMask mask = row_mask<TREE>(a, e, i, live);
  const OpenKeys seen_by_all = open_keys<TREE>(a, e, i0, i1);
  const bool wave_live = r0 + wave * 32 < rows;              // else it only carries tiles
  u32x4v q[STEPS];
  {
    const uint16_t* src = a.q + (int64_t)(e.first + i) * a.q_stride + (int64_t)hq * D + half * 8;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) q[s] = *reinterpret_cast<const u32x4v*>(src + s * 16);
  }
  f32x16 o[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t) o[t] = f32x16{};
  Running st{-INFINITY, 0.0f};
  const float c = a.scale * kLog2e;

  u32x4v in[PER];                                            // a thread's granules of one operand on their way
  // The page of each of a tile's keys, one key a lane.
  auto pages_of = [&](int t) {
    const int key = list.key<KT>(min(t, t1 - 1)) + lane;
    return e.pages[min(key >> a.page_log2, (int)a.width - 1)];
  };
  const uint32_t page_elems = (uint32_t)(a.heads_kv * D) << a.page_log2, head_at = (uint32_t)(h * D) << a.page_log2;
  // keys: granule g of the tile is dimension block g / 64 of key g % 64, so
  // a thread keeps its key
  auto fetch_keys = [&](int t, int32_t pk) {
    const uint16_t* kp = a.k + (uint64_t)page_in_pool(pk, a.pages) * page_elems + head_at +
                         (((list.key<KT>(t) + lane) & pmask) + wave * P) * 8;
#pragma unroll
    for (int n = 0; n < PER; ++n) in[n] = *reinterpret_cast<const u32x4v*>(kp + n * kWaves * P * 8);
  };
  // values: granule g is token block g / D of dimension g % D, one token
  // block a wave, whose address the lane of the block's first key works out
  auto fetch_values = [&](int t, int32_t pk) {
    const uint64_t block = (uint64_t)(a.v + (uint64_t)page_in_pool(pk, a.pages) * page_elems + head_at +
                                      (((list.key<KT>(t) + lane) & pmask) >> 3) * D * 8);
#pragma unroll
    for (int n = 0; n < PER; ++n) {
      const int g = n * kThreads + wave * 64, at = g / D * 8;
      const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)block, at);
      const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(block >> 32), at);
      in[n] = reinterpret_cast<const __attribute__((address_space(1))) u32x4v*>(((uint64_t)hi << 32) | lo)[g % D + lane];
    }
  };
  auto store_keys = [&](int buf) {
#pragma unroll
    for (int n = 0; n < PER; ++n) lds[buf * 2 * GRAN + n * kThreads + tid] = in[n];
  };
  // s_bad: the last tile whose values had to be cleaned
  auto store_values = [&](int buf, int t) {
    if (!seen_by_all.tile(list.key<KT>(t), KT)) {
      bool bad = false;
#pragma unroll
      for (int n = 0; n < PER; ++n) bad |= drop_nonfinite<T>(in[n]);
      if (bad) s_bad[buf] = t;
    }
#pragma unroll
    for (int n = 0; n < PER; ++n) lds[(buf * 2 + 1) * GRAN + n * kThreads + tid] = in[n];
  };
  auto rescale = [&](float alpha) {
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[d][r] *= alpha;
  };

  if (tid < 2) s_bad[tid] = -1;
  lds_barrier();
  int32_t page = 0;
  if (t0 < t1) {
    page = pages_of(t0);
    fetch_keys(t0, page);
    store_keys(0);
    fetch_values(t0, page);
    page = pages_of(t0 + 1);
    store_values(0, t0);
  }
  lds_barrier();
  const int krow = tile_key_of_row(col);
  waitcnt_vm<0>();         // q has arrived: waits inside the loop are for the tiles' loads only
  for (int t = t0; t < t1; ++t) {
    const int buf = (t - t0) & 1, kb = list.key<KT>(t);
    const bool more = t + 1 < t1;
    const u32x4v* kt = lds + buf * 2 * GRAN + half * KT + krow;        // [2 s + half][32 x + key]
    const u32x4v* vt = lds + (buf * 2 + 1) * GRAN + half * D + col;    // [4 x + 2 s + half][dimension]
    if (more) fetch_keys(t + 1, page);
    const bool open = seen_by_all.tile(kb, KT);
    uint64_t seen = 0;
    f32x16 s0[1] = {f32x16{}}, s1[1] = {f32x16{}};
    u32x4v p0[2], p1[2];
    float alpha;
    bool moved = false;
    if (wave_live) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) s0[0] = T::mfma(kt[2 * s * KT], q[s], s0[0]);
      if (!open) {
        seen = mask.bits<TREE>(kb);
        cut_scores(s0[0], (uint32_t)seen);
      }
      if (move_bound(s0, c, st, alpha)) rescale(alpha);
#pragma unroll
      for (int s = 0; s < STEPS; ++s) s1[0] = T::mfma(kt[2 * s * KT + 32], q[s], s1[0]);
      weigh(s0, c, st);
      pack_weights<T>(s0[0], p0);
      interleave<STEPS, 56 / STEPS, 16 / STEPS>();
    }
    if (more) {
      store_keys(buf ^ 1);
      fetch_values(t + 1, page);
      page = pages_of(t + 2);
    }
    if (wave_live) {
      if (!open) cut_scores(s1[0], (uint32_t)(seen >> 32));
      moved = move_bound(s1, c, st, alpha);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = T::mfma(vt[2 * s * D + d * 32], p0[s], o[d]);
      weigh(s1, c, st);
      pack_weights<T>(s1[0], p1);
      interleave<2 * DT, 56 / (2 * DT), 16 / (2 * DT)>();
      if (moved) rescale(alpha);                             // the first block was weighed with the earlier bound
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = T::mfma(vt[(4 + 2 * s) * D + d * 32], p1[s], o[d]);
      if (!open && s_bad[buf] == t)
        add_nonfinite<T, D, TREE>(a.v + head_at, e.pages, a.pages, page_elems, a.page_log2, mask, kb, KT, o);
    }
    if (more) store_values(buf ^ 1, t + 1);
    lds_barrier();
  }

  const float l = st.l + __shfl_xor(st.l, 32);
  if (!live) return;
  if (a.splits == 1) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t* dst = a.out + ((int64_t)(e.first + i) * a.heads_q + hq) * D + 4 * half;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<u32x2v*>(dst + d * 32 + 8 * j) =
            u32x2v{T::pack(o[d][4 * j] * inv, o[d][4 * j + 1] * inv), T::pack(o[d][4 * j + 2] * inv, o[d][4 * j + 3] * inv)};
    return;
  }
  const int64_t at = ((int64_t)(e.first + i) * a.heads_q + hq) * a.splits + split;
  if (half == 0) *reinterpret_cast<f32x2p*>(a.part_ml + at * 2) = f32x2p{st.m, l};
  if (st.m == -INFINITY) return;
  float* part = a.part_o + at * D + 4 * half;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<f32x4v*>(part + d * 32 + 8 * j) =
          f32x4v{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
}

// ---- fold ----------------------------------------------------------------
// o = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s, one wave per output row.
template <typename T, int D, bool TREE, bool FEW>
__global__ __launch_bounds__(64) void attention_fold_kernel(AttnArgs a) {
  constexpr int V = D / 64;
  const int lane = threadIdx.x;
  int64_t ml, step;                                          // first (m, l) pair, distance between parts
  int splits;
  int64_t out_row;
  if (FEW) {
    const Unit u = find_unit<TREE>(a, blockIdx.z, true);
    if (!u.live || u.splits == 1) return;
    const Entry e = load_entry(a, u.e);
    const int h = blockIdx.y, group = a.heads_q / a.heads_kv, row = blockIdx.x;
    if (row >= e.n * group) return;
    splits = u.splits;
    ml = ((int64_t)u.base * a.heads_kv + h) * kFewRows + row;
    step = (int64_t)a.heads_kv * kFewRows;
    out_row = (int64_t)(e.first + row / group) * a.heads_q + h * group + row % group;
  } else {
    const Entry e = load_entry(a, blockIdx.z);
    if ((int)blockIdx.x >= e.n) return;
    splits = a.splits;
    out_row = (int64_t)(e.first + blockIdx.x) * a.heads_q + blockIdx.y;
    ml = out_row * splits;
    step = 1;
  }
  float top = -INFINITY;
  for (int s = lane; s < splits; s += 64) top = fmaxf(top, a.part_ml[(ml + s * step) * 2]);
#pragma unroll
  for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  float acc[V] = {}, sum = 0.0f;
  if (top != -INFINITY) {
    for (int s = 0; s < splits; ++s) {
      const float m = a.part_ml[(ml + s * step) * 2], l = a.part_ml[(ml + s * step) * 2 + 1];
      if (m == -INFINITY) continue;
      const float f = __builtin_amdgcn_exp2f(m - top);
      sum += f * l;
      const float* src = a.part_o + (ml + s * step) * D + lane * V;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += f * src[v];
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint16_t* dst = a.out + out_row * D + lane * V;
#pragma unroll
  for (int v = 0; v < V; ++v) dst[v] = (uint16_t)T::pack(acc[v] * inv, 0.0f);
}

bool few_rows(const AttnArgs& a) { return (int64_t)a.max_q * (a.heads_q / a.heads_kv) <= kFewRows; }

// Workgroups per key head that the few-row kernel's cut aims at: as many as
// run at once, over the heads.
int few_target(const AttnArgs& a) {
  const int resident = device_cus() * (a.head_dim == 256 ? 1 : 2);
  return resident / a.heads_kv > 1 ? resident / a.heads_kv : 1;
}
int64_t few_slots(const AttnArgs& a) { return (int64_t)few_target(a) + a.entries; }

int64_t row_tiles(const AttnArgs& a) {
  return ((int64_t)a.max_q * (a.heads_q / a.heads_kv) + kManyRows - 1) / kManyRows;
}

// Parts of every unit's keys in the many-row kernel: enough that the grid
// holds two workgroups a compute unit, none shorter than four tiles.
int many_splits(const AttnArgs& a) {
  const int64_t units = row_tiles(a) * a.heads_kv * a.entries;
  int64_t s = 2 * (int64_t)device_cus() / (units > 0 ? units : 1);
  int64_t keys = a.width << a.page_log2;
  const int64_t reach = (int64_t)a.window + a.max_q + a.sinks;
  if (a.window > 0 && reach < keys) keys = reach;
  const int64_t most = keys / (4 * kManyKeys);
  if (s > most) s = most;
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

// (partial outputs, (m, l) pairs) in bytes
void part_bytes(const AttnArgs& a, size_t* o, size_t* ml) {
  int64_t rows;
  if (few_rows(a)) {
    rows = few_slots(a) * a.heads_kv * kFewRows;
  } else {
    const int s = many_splits(a);
    rows = s == 1 ? 0 : a.tokens * a.heads_q * s;
  }
  *o = round256((size_t)rows * a.head_dim * 4);
  *ml = round256((size_t)rows * 8);
}

template <typename T, int D, bool TREE>
hipError_t launch_typed(AttnArgs& a, hipStream_t stream) {
  if (few_rows(a)) {
    a.target = few_target(a);
    attention_few_kernel<T, D, TREE><<<dim3((unsigned)few_slots(a), a.heads_kv), kThreads, 0, stream>>>(a);
    attention_fold_kernel<T, D, TREE, true>
        <<<dim3(a.max_q * (a.heads_q / a.heads_kv), a.heads_kv, a.entries), 64, 0, stream>>>(a);
    return hipGetLastError();
  }
  constexpr size_t lds = 2 * 2 * (size_t)kManyKeys * D * 2;
  static hipError_t ready = hipFuncSetAttribute((const void*)&attention_many_kernel<T, D, TREE>,
                                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (ready != hipSuccess) return ready;
  a.splits = many_splits(a);
  attention_many_kernel<T, D, TREE>
      <<<dim3((unsigned)(row_tiles(a) * a.splits), a.heads_kv, a.entries), kThreads, lds, stream>>>(a);
  if (a.splits > 1)
    attention_fold_kernel<T, D, TREE, false><<<dim3(a.max_q, a.heads_q, a.entries), 64, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_masked(AttnArgs& a, hipStream_t stream) {
  return a.ancestors ? launch_typed<T, D, true>(a, stream) : launch_typed<T, D, false>(a, stream);
}

template <typename T>
hipError_t launch_dim(AttnArgs& a, hipStream_t stream) {
  switch (a.head_dim) {
    case 64: return launch_masked<T, 64>(a, stream);
    case 128: return launch_masked<T, 128>(a, stream);
    default: return launch_masked<T, 256>(a, stream);
  }
}

}  // namespace

size_t attention_workspace_bytes(const AttnArgs& a) {
  size_t o, ml;
  part_bytes(a, &o, &ml);
  return o + ml;
}

hipError_t launch_attention(AttnArgs a, void* workspace, hipStream_t stream) {
  size_t o, ml;
  part_bytes(a, &o, &ml);
  a.part_o = reinterpret_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + o);
  return a.fp16 ? launch_dim<F16>(a, stream) : launch_dim<Bf16>(a, stream);
}

}  // namespace trellis
