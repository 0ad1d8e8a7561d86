// cache.hip -- the pages of the key/value cache: reserving, forking, accepting
// drafted rows (compaction), freeing.
//
// The state is three device arrays: table [seqs, width] of page numbers (-1:
// none), lengths [seqs], refs [pages].  A page is free when refs is 0, and the
// lowest free pages are taken first, in the order of the call's list; there
// is no free list whose order could depend on which workgroup came first, so
// every outcome is determined by the arguments, and a step that changes the
// cache can be captured into a graph without the host knowing any length.
#include "internal.hpp"
#include "kv8_common.hpp"

namespace trellis {
namespace {

constexpr int kPlan = 1024;               // threads of the one workgroup that hands out pages
constexpr int kPlanWaves = kPlan / 64;

// Whether entry b of a list names a sequence of the state that no earlier
// entry names.  Called by a whole wave, whose lanes compare 64 entries at a
// time: one lane by itself waits a memory latency for each (8 us of a
// reservation for 16 of 48 sequences).
__device__ __forceinline__ bool first_of_its_name(const int32_t* ids, int b, int64_t seqs) {
  const int32_t id = ids[b];
  bool known = false;
  for (int j = threadIdx.x & 63; j < b; j += 64) known |= ids[j] == id;
  return id >= 0 && id < seqs && __ballot(known) == 0;
}

// Exclusive sum over the workgroup's threads; `total` for all.
__device__ __forceinline__ int block_scan(int v, int* sums, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int upto = wave_scan_add(v);
  __syncthreads();
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    const int s = sums[w];
    before += w < wave ? s : 0;
    all += s;
  }
  total = all;
  return before + upto - v;
}

// The lowest `want` free pages, ascending, into list; returns how many there
// are (at most want).  Called by the whole workgroup.
__device__ __forceinline__ int find_free(const int32_t* refs, uint32_t pages, int want, int32_t* list, int* sums) {
  constexpr int PER = 16;
  int found = 0;
  for (int64_t base = 0; base < pages && found < want; base += (int64_t)kPlan * PER) {
    const int64_t first = base + (int64_t)threadIdx.x * PER;
    uint32_t free = 0;
    if (first + PER <= pages) {
#pragma unroll
      for (int j = 0; j < PER; j += 4) {
        const u32x4v r = *reinterpret_cast<const u32x4v*>(refs + first + j);
#pragma unroll
        for (int x = 0; x < 4; ++x) free |= (r[x] == 0 ? 1u : 0u) << (j + x);
      }
    } else {
      for (int j = 0; j < PER && first + j < pages; ++j) free |= (refs[first + j] == 0 ? 1u : 0u) << j;
    }
    int total;
    int rank = found + block_scan(__popc(free), sums, total);
    for (; free; free &= free - 1, ++rank)
      if (rank < want) list[rank] = (int32_t)(first + __builtin_ctz(free));
    found += total;
  }
  __syncthreads();
  return min(found, want);
}

// ---- reserve -------------------------------------------------------------

// The slot of token t: the last entry that starts at or before it owns it.
__device__ __forceinline__ int32_t slot_of(const CacheArgs& c, const int32_t* seq_ids, int n, const int32_t* q_start,
                                           const int32_t* granted, int64_t t) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (q_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  if (!granted[lo] || t < q_start[lo] || t >= q_start[lo + 1]) return -1;
  const int64_t at = max(c.lengths[seq_ids[lo]], 0) + t - max(q_start[lo], 0);
  const int32_t page = c.table[(int64_t)seq_ids[lo] * c.width + (at >> c.page_log2)];
  return page_ok(page, c.pages) ? (int32_t)(((int64_t)page << c.page_log2) + (at & ((1 << c.page_log2) - 1))) : -1;
}

// One workgroup hands out the pages.  With SLOTS it writes the tokens' slots
// too, which saves a launch for a step that decodes.
template <bool SLOTS>
__global__ __launch_bounds__(kPlan) void reserve_plan_kernel(CacheArgs c, const int32_t* seq_ids, int n,
                                                             const int32_t* q_start, int64_t tokens, int32_t* granted,
                                                             int32_t* list, int32_t* slots) {
  __shared__ int s_need[kCacheMaxEntries], s_at[kCacheMaxEntries], s_sums[kPlanWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t room = c.width << c.page_log2;
  // pages without storage among those the entry's new tokens fall on; -1: refused
  for (int b = wave; b < n; b += kPlanWaves) {
    int need = -1;
    if (first_of_its_name(seq_ids, b, c.seqs)) {
      const int64_t len = max(c.lengths[seq_ids[b]], 0);
      const int64_t count = max(min((int64_t)q_start[b + 1], tokens) - max(q_start[b], 0), (int64_t)0);
      if (len + count <= room) {
        const int32_t* row = c.table + (int64_t)seq_ids[b] * c.width;
        const int64_t end = count ? (len + count + (1 << c.page_log2) - 1) >> c.page_log2 : 0;
        int mine = 0;
        for (int64_t p = (len >> c.page_log2) + lane; p < end; p += 64) mine += !page_ok(row[p], c.pages);
        need = wave_sum(mine);
      }
    }
    if (lane == 0) s_need[b] = need;
  }
  __syncthreads();
  int total;
  const int mine = tid < n ? max(s_need[tid], 0) : 0;
  const int at = block_scan(mine, s_sums, total);
  if (tid < n) s_at[tid] = at;
  const int have = find_free(c.refs, c.pages, total, list, s_sums);
  for (int b = wave; b < n; b += kPlanWaves) {
    const int need = s_need[b];
    const bool ok = need >= 0 && s_at[b] + need <= have;
    if (lane == 0) granted[b] = ok;
    if (!ok || need == 0) continue;
    const int64_t len = max(c.lengths[seq_ids[b]], 0);
    const int64_t count = min((int64_t)q_start[b + 1], tokens) - max(q_start[b], 0);
    int32_t* row = c.table + (int64_t)seq_ids[b] * c.width;
    const int64_t end = (len + count + (1 << c.page_log2) - 1) >> c.page_log2;
    int next = s_at[b];
    for (int64_t base = len >> c.page_log2; base < end; base += 64) {
      const int64_t p = base + lane;
      const bool take = p < end && !page_ok(row[p], c.pages);
      const uint64_t votes = __ballot(take);
      if (take) {
        const int32_t page = list[next + __popcll(votes & ((1ull << lane) - 1))];
        row[p] = page;
        c.refs[page] = 1;
      }
      next += __popcll(votes);
    }
  }
  if (SLOTS) {
    __syncthreads();
    for (int64_t t = tid; t < tokens; t += kPlan) slots[t] = slot_of(c, seq_ids, n, q_start, granted, t);
  }
}

__global__ __launch_bounds__(256) void reserve_slots_kernel(CacheArgs c, const int32_t* seq_ids, int n,
                                                            const int32_t* q_start, int64_t tokens,
                                                            const int32_t* granted, int32_t* slots) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= tokens) return;
  slots[t] = slot_of(c, seq_ids, n, q_start, granted, t);
}

// ---- fork ----------------------------------------------------------------
// Workspace per entry: its parent's row as it was before the call, and what
// the plan decided.
enum ForkState : int32_t {
  kForkIgnored = 0,    // a repeated or unknown child: nothing of it changes
  kForkSame = 1,       // its own parent: left as it is
  kForkDone = 2,
  kForkEmptied = 3,    // no such parent, or a page of its length is missing: the child is left empty
  kForkNoPage = 4,     // no page was left for its partial page: left empty
};
struct ForkEntry {
  int32_t state, length, src, page;
};

// Before any page is handed out: copy the parents' rows, count the shared
// pages for the children, hold on to the partial pages that will be copied,
// and let go of the children's old pages.  All of it is additions, so the
// order does not matter, and what the call still needs keeps refs > 0 even
// where a parent is itself replaced.
__global__ __launch_bounds__(256) void fork_snapshot_kernel(CacheArgs c, const int32_t* parents,
                                                            const int32_t* children, ForkEntry* entries,
                                                            int32_t* rows) {
  const int b = blockIdx.x, tid = threadIdx.x;
  const int32_t par = parents[b], kid = children[b];
  ForkEntry f{kForkIgnored, 0, -1, -1};
  if (first_of_its_name(children, b, c.seqs)) {
    if (par == kid) {
      f.state = kForkSame;
    } else {
      f.state = kForkEmptied;
      int full = 0;
      if (par >= 0 && par < c.seqs) {
        f.length = max(c.lengths[par], 0);
        full = f.length >> c.page_log2;
        const bool part = (f.length & ((1 << c.page_log2) - 1)) != 0;
        bool missing = (int64_t)full + part > c.width;
        const int32_t src = part && !missing ? c.table[(int64_t)par * c.width + full] : -1;
        missing |= part && !page_ok(src, c.pages);
        for (int64_t p = tid; !missing && p < full; p += 256)
          missing = !page_ok(c.table[(int64_t)par * c.width + p], c.pages);
        if (!__syncthreads_or(missing)) {
          f.state = kForkDone;
          f.src = src;
        }
      }
      for (int64_t p = tid; p < c.width; p += 256) {
        if (f.state == kForkDone && p < full) {
          const int32_t page = c.table[(int64_t)par * c.width + p];
          rows[(int64_t)b * c.width + p] = page;
          if (page_ok(page, c.pages)) atomicAdd(c.refs + page, 1);
        }
        const int32_t old = c.table[(int64_t)kid * c.width + p];
        if (page_ok(old, c.pages)) atomicSub(c.refs + old, 1);
      }
      if (tid == 0 && f.src >= 0) atomicAdd(c.refs + f.src, 1);
    }
  }
  if (tid == 0) entries[b] = f;
}

__global__ __launch_bounds__(kPlan) void fork_plan_kernel(CacheArgs c, int n, ForkEntry* entries, int32_t* list) {
  __shared__ int s_sums[kPlanWaves];
  const int tid = threadIdx.x;
  const bool part = tid < n && entries[tid].state == kForkDone && entries[tid].src >= 0;
  int total;
  const int at = block_scan(part ? 1 : 0, s_sums, total);
  const int have = find_free(c.refs, c.pages, total, list, s_sums);
  if (!part) return;
  if (at < have) {
    entries[tid].page = list[at];
    c.refs[list[at]] = 1;
  } else {
    entries[tid].state = kForkNoPage;
  }
}

// Children's rows and lengths; the copy of the partial page in every layer
// (blockIdx.y: layer), of 8-bit caches (SCALED) with its scales.
template <bool SCALED>
__global__ __launch_bounds__(256) void fork_write_kernel(CacheArgs c, const int32_t* children, const ForkEntry* entries,
                                                         const int32_t* rows, int32_t* granted, Scales scales) {
  const int b = blockIdx.x, tid = threadIdx.x;
  const ForkEntry f = entries[b];
  if (blockIdx.y == 0) {
    const int32_t kid = children[b];
    if (tid == 0) {
      granted[b] = f.state == kForkSame || f.state == kForkDone;
      if (f.src >= 0) atomicSub(c.refs + f.src, 1);
    }
    if (f.state >= kForkDone) {
      const int full = f.length >> c.page_log2;
      for (int64_t p = tid; p < c.width; p += 256) {
        int32_t page = -1;
        if (f.state != kForkEmptied && p < full) {
          page = rows[(int64_t)b * c.width + p];
          if (!page_ok(page, c.pages)) page = -1;
          if (f.state == kForkNoPage && page >= 0) {
            atomicSub(c.refs + page, 1);
            page = -1;
          }
        } else if (f.state == kForkDone && p == full) {
          page = f.page;
        }
        c.table[(int64_t)kid * c.width + p] = page;
      }
      if (tid == 0) c.lengths[kid] = f.state == kForkDone ? f.length : 0;
    }
  }
  if (f.state != kForkDone || f.page < 0) return;
  const int64_t granules = ((int64_t)c.heads * c.head_dim << c.page_log2) / (SCALED ? 16 : 8);   // one page of one layer
  const int64_t layer = (int64_t)blockIdx.y * c.pages;
  const u32x4v* ks = reinterpret_cast<const u32x4v*>(c.k) + (layer + f.src) * granules;
  const u32x4v* vs = reinterpret_cast<const u32x4v*>(c.v) + (layer + f.src) * granules;
  u32x4v* kd = reinterpret_cast<u32x4v*>(c.k) + (layer + f.page) * granules;
  u32x4v* vd = reinterpret_cast<u32x4v*>(c.v) + (layer + f.page) * granules;
  for (int64_t g = tid; g < granules; g += 256) {
    const u32x4v x = ks[g], y = vs[g];
    kd[g] = x;
    vd[g] = y;
  }
  if constexpr (SCALED) {
    const int64_t blocks = (int64_t)c.heads << (c.page_log2 - 4), src = (layer + f.src) * blocks, dst = (layer + f.page) * blocks;
    for (int64_t x = tid; x < blocks; x += 256) {
      scales.k[dst + x] = scales.k[src + x];
      scales.v[dst + x] = scales.v[src + x];
    }
  }
}

// ---- accept --------------------------------------------------------------
// Row length + j becomes what row length + path[j] was: one workgroup per
// (sequence, layer, head) reads all its rows into LDS before it writes any.
// Where the new lengths go to an array of their own, the workgroups past the
// list's end write them; in place that has to wait for all readers.
__device__ __forceinline__ void accept_lengths(const CacheArgs& c, const int32_t* seq_ids, int n, int max_path,
                                               const int32_t* counts, int32_t* new_lengths) {
  const int waves = blockDim.x >> 6;
  if (new_lengths != c.lengths) {
    for (int64_t s = threadIdx.x; s < c.seqs; s += blockDim.x) new_lengths[s] = c.lengths[s];
    __syncthreads();
  }
  for (int b = threadIdx.x >> 6; b < n; b += waves) {
    if (!first_of_its_name(seq_ids, b, c.seqs) || (threadIdx.x & 63)) continue;
    const int64_t len = max(c.lengths[seq_ids[b]], 0);
    new_lengths[seq_ids[b]] = (int32_t)min(len + min(max(counts[b], 0), max_path), c.width << c.page_log2);
  }
}

__global__ __launch_bounds__(256) void accept_kernel(CacheArgs c, const int32_t* seq_ids, int n, const int32_t* path,
                                                     int max_path, const int32_t* counts, int32_t* new_lengths) {
  if ((int)blockIdx.x == n) {
    if (blockIdx.y == 0 && blockIdx.z == 0) accept_lengths(c, seq_ids, n, max_path, counts, new_lengths);
    return;
  }
  extern __shared__ __align__(16) u32x4v lds[];              // keys [row][D / 8], values [row][D / 8]
  const int b = blockIdx.x, layer = blockIdx.y, h = blockIdx.z, tid = threadIdx.x;
  const int count = min(max(counts[b], 0), max_path);
  if (count == 0 || !first_of_its_name(seq_ids, b, c.seqs)) return;
  const int64_t row = seq_ids[b], len = max(c.lengths[row], 0), P = 1 << c.page_log2;
  const int gran = c.head_dim / 8;
  const int64_t head_elems = (int64_t)c.head_dim << c.page_log2;
  // base of the head's page that holds a token, or -1
  auto base = [&](int64_t at) -> int64_t {
    const int64_t p = at >> c.page_log2;
    if (at < 0 || p >= c.width) return -1;
    const int32_t page = c.table[row * c.width + p];
    if (!page_ok(page, c.pages)) return -1;
    return (((int64_t)layer * c.pages + page) * c.heads + h) * head_elems;
  };
  u32x4v* lk = lds;
  uint16_t* lv = reinterpret_cast<uint16_t*>(lds + max_path * gran);
  for (int x = tid; x < count * gran; x += 256) {
    const int j = x / gran, g = x % gran, from = path[(int64_t)b * max_path + j];
    const int64_t at = len + from, src = base(at);
    if (from == j || from < 0 || src < 0) continue;
    lk[x] = *reinterpret_cast<const u32x4v*>(c.k + src + ((int64_t)g * P + (at & (P - 1))) * 8);
    const uint16_t* vs = c.v + src + ((at & (P - 1)) >> 3) * c.head_dim * 8 + g * 64 + (at & 7);
#pragma unroll
    for (int e = 0; e < 8; ++e) lv[x * 8 + e] = vs[e * 8];
  }
  __syncthreads();
  for (int x = tid; x < count * gran; x += 256) {
    const int j = x / gran, g = x % gran, from = path[(int64_t)b * max_path + j];
    const int64_t at = len + j, dst = base(at);
    if (from == j || from < 0 || dst < 0 || base(len + from) < 0) continue;
    *reinterpret_cast<u32x4v*>(c.k + dst + ((int64_t)g * P + (at & (P - 1))) * 8) = lk[x];
    uint16_t* vd = c.v + dst + ((at & (P - 1)) >> 3) * c.head_dim * 8 + g * 64 + (at & 7);
#pragma unroll
    for (int e = 0; e < 8; ++e) vd[e * 8] = lv[x * 8 + e];
  }
}

// The same over 8-bit blocks.  All rows that move, and their scales, are in LDS
// before any block changes; then a thread owns a granule of the blocks that
// rows move into: it sets the rows that arrive and rounds the others again
// where the block's scale grew.  The scales are written at the end, from what
// all threads read at the start.  A chain of latencies, as in 16 bits: 8 x 16
// rows, 32 layers 10.6 us either way.
constexpr int kAcceptBlocks = kCacheMaxPath / 16 + 1;
__global__ __launch_bounds__(256) void accept_kv8_kernel(CacheArgs c, Scales scales, const int32_t* seq_ids, int n,
                                                         const int32_t* path, int max_path, const int32_t* counts,
                                                         int32_t* new_lengths) {
  if ((int)blockIdx.x == n) {
    if (blockIdx.y == 0 && blockIdx.z == 0) accept_lengths(c, seq_ids, n, max_path, counts, new_lengths);
    return;
  }
  extern __shared__ __align__(16) u32x4v lds[];              // keys [row][D / 16], values [row][D / 16]
  __shared__ int s_moves[kCacheMaxPath];
  __shared__ uint32_t s_from[2][kCacheMaxPath], s_old[2][kAcceptBlocks], s_new[2][kAcceptBlocks];
  const int b = blockIdx.x, layer = blockIdx.y, h = blockIdx.z, tid = threadIdx.x;
  const int count = min(max(counts[b], 0), max_path);
  if (count == 0 || !first_of_its_name(seq_ids, b, c.seqs)) return;
  const int64_t row = seq_ids[b], len = max(c.lengths[row], 0), P = 1 << c.page_log2;
  const int D = c.head_dim, gran = D / 16;
  const uint8_t *k8 = reinterpret_cast<const uint8_t*>(c.k), *v8 = reinterpret_cast<const uint8_t*>(c.v);
  // the head's page that holds a token, counted over the pool, or -1
  auto page_of = [&](int64_t at) -> int64_t {
    const int64_t p = at >> c.page_log2;
    if (at < 0 || p >= c.width) return -1;
    const int32_t page = c.table[row * c.width + p];
    if (!page_ok(page, c.pages)) return -1;
    return ((int64_t)layer * c.pages + page) * c.heads + h;
  };
  auto scale_at = [&](int64_t page, int64_t at) { return (page << (c.page_log2 - 4)) + ((at & (P - 1)) >> 4); };
  const int64_t head_bytes = (int64_t)D << c.page_log2;
  const int64_t from_block = len >> 4;                       // the first that a row can move into
  const int blocks = (int)(((len + count - 1) >> 4) - from_block) + 1;
  for (int j = tid; j < count; j += 256) {
    const int from = path[(int64_t)b * max_path + j];
    const int64_t src = page_of(len + from);
    const bool moves = from != j && from >= 0 && src >= 0 && page_of(len + j) >= 0;
    s_moves[j] = moves;
    s_from[0][j] = moves ? scales.k[scale_at(src, len + from)] : 0;
    s_from[1][j] = moves ? scales.v[scale_at(src, len + from)] : 0;
  }
  for (int x = tid; x < 2 * blocks; x += 256) {
    const int64_t at = (from_block + (x >> 1)) << 4, page = page_of(at);
    s_old[x & 1][x >> 1] = s_new[x & 1][x >> 1] = page < 0 ? 0u : (x & 1 ? scales.v : scales.k)[scale_at(page, at)];
  }
  __syncthreads();
  for (int j = tid; j < 2 * count; j += 256)
    if (s_moves[j >> 1])
      atomicMax(&s_new[j & 1][((len + (j >> 1)) >> 4) - from_block], s_from[j & 1][j >> 1]);
  u32x4v* lk = lds;
  uint8_t* lv = reinterpret_cast<uint8_t*>(lds + max_path * gran);
  for (int x = tid; x < count * gran; x += 256) {
    const int j = x / gran, g = x % gran;
    if (!s_moves[j]) continue;
    const int64_t at = len + path[(int64_t)b * max_path + j], in = at & (P - 1), src = page_of(at) * head_bytes;
    lk[x] = *reinterpret_cast<const u32x4v*>(k8 + src + (g * P + in) * 16);
    const uint8_t* vs = v8 + src + ((in >> 4) * D + g * 16) * 16 + (in & 15);
#pragma unroll
    for (int e = 0; e < 16; ++e) lv[x * 16 + e] = vs[e * 16];
  }
  __syncthreads();
  // keys: granules [block][D / 16][16 rows]; values: [block][D]
  for (int x = tid; x < 2 * blocks * D; x += 256) {
    const bool is_v = x >= blocks * D;
    const int y = is_v ? x - blocks * D : x, blk = y / D, z = y % D;
    const uint32_t old = s_old[is_v][blk], now = s_new[is_v][blk];
    const int64_t base = (from_block + blk) << 4, page = page_of(base);
    if (page < 0) continue;
    const int64_t in = base & (P - 1);
    if (!is_v) {
      const int r = z & 15, g = z >> 4;
      const int64_t j = base + r - len;
      const bool arrives = j >= 0 && j < count && s_moves[j];
      if (!arrives && now == old) continue;
      u32x4v* at = reinterpret_cast<u32x4v*>(c.k) + (page * head_bytes >> 4) + g * P + in + r;
      *at = rescaled(arrives ? lk[j * gran + g] : *at, arrives ? s_from[0][j] : old, now);
    } else {
      u32x4v* at = reinterpret_cast<u32x4v*>(c.v) + (page * head_bytes >> 4) + (in >> 4) * D + z;
      u32x4v v = *at;
      if (now != old) v = rescaled(v, old, now);
      for (int r = 0; r < 16; ++r) {
        const int64_t j = base + r - len;
        if (j < 0 || j >= count || !s_moves[j]) continue;
        const int by = (r & 3) * 8;
        const uint32_t code = rescaled4(lv[j * D + z], s_from[1][j], now) & 0xFFu;
#pragma unroll
        for (int w = 0; w < 4; ++w) v[w] = r >> 2 == w ? (v[w] & ~(0xFFu << by)) | code << by : v[w];
      }
      *at = v;
    }
  }
  for (int x = tid; x < 2 * blocks; x += 256) {
    const int64_t at = (from_block + (x >> 1)) << 4, page = page_of(at);
    const uint32_t now = s_new[x & 1][x >> 1];
    if (page >= 0 && now != s_old[x & 1][x >> 1]) (x & 1 ? scales.v : scales.k)[scale_at(page, at)] = (uint8_t)now;
  }
}

__global__ __launch_bounds__(kPlan) void accept_lengths_kernel(CacheArgs c, const int32_t* seq_ids, int n,
                                                               int max_path, const int32_t* counts,
                                                               int32_t* new_lengths) {
  accept_lengths(c, seq_ids, n, max_path, counts, new_lengths);
}

// ---- free ----------------------------------------------------------------
// The exchange hands every table entry to one of the list's entries only, so
// a sequence named twice is freed once.
__global__ __launch_bounds__(256) void free_kernel(CacheArgs c, const int32_t* seq_ids) {
  const int64_t row = seq_ids[blockIdx.x];
  if (row < 0 || row >= c.seqs) return;
  for (int64_t p = threadIdx.x; p < c.width; p += 256) {
    const int32_t page = atomicExch(c.table + row * c.width + p, -1);
    if (page_ok(page, c.pages)) atomicSub(c.refs + page, 1);
  }
  if (threadIdx.x == 0) c.lengths[row] = 0;
}

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// the free pages that are handed out: never more than the pool has, nor than the list can want
size_t cache_reserve_workspace_bytes(const CacheArgs& c, int n) {
  const int64_t want = (int64_t)n * c.width;
  return round256((size_t)(want < (int64_t)c.pages ? want : (int64_t)c.pages) * 4);
}

hipError_t launch_cache_reserve(const CacheArgs& c, const int32_t* seq_ids, int n, const int32_t* q_start,
                                int64_t tokens, int32_t* slots, int32_t* granted, void* workspace,
                                hipStream_t stream) {
  int32_t* list = reinterpret_cast<int32_t*>(workspace);
  if (tokens <= kPlan) {
    reserve_plan_kernel<true><<<1, kPlan, 0, stream>>>(c, seq_ids, n, q_start, tokens, granted, list, slots);
  } else {
    reserve_plan_kernel<false><<<1, kPlan, 0, stream>>>(c, seq_ids, n, q_start, tokens, granted, list, slots);
    reserve_slots_kernel<<<(unsigned)((tokens + 255) / 256), 256, 0, stream>>>(c, seq_ids, n, q_start, tokens, granted,
                                                                               slots);
  }
  return hipGetLastError();
}

size_t cache_fork_workspace_bytes(const CacheArgs& c, int n) {
  return round256((size_t)n * sizeof(ForkEntry)) + round256((size_t)n * 4) + round256((size_t)n * (size_t)c.width * 4);
}

namespace {

template <bool SCALED>
hipError_t launch_fork(const CacheArgs& c, const Scales& s, const int32_t* parents, const int32_t* children, int n,
                       int32_t* granted, void* workspace, hipStream_t stream) {
  char* w = reinterpret_cast<char*>(workspace);
  ForkEntry* entries = reinterpret_cast<ForkEntry*>(w);
  int32_t* list = reinterpret_cast<int32_t*>(w + round256((size_t)n * sizeof(ForkEntry)));
  int32_t* rows = reinterpret_cast<int32_t*>(w + round256((size_t)n * sizeof(ForkEntry)) + round256((size_t)n * 4));
  fork_snapshot_kernel<<<n, 256, 0, stream>>>(c, parents, children, entries, rows);
  fork_plan_kernel<<<1, kPlan, 0, stream>>>(c, n, entries, list);
  fork_write_kernel<SCALED><<<dim3(n, c.layers), 256, 0, stream>>>(c, children, entries, rows, granted, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_fork(const CacheArgs& c, const int32_t* parents, const int32_t* children, int n,
                             int32_t* granted, void* workspace, hipStream_t stream) {
  return launch_fork<false>(c, Scales{}, parents, children, n, granted, workspace, stream);
}

hipError_t launch_cache_fork_kv8(const CacheArgs& c, const Scales& s, const int32_t* parents, const int32_t* children,
                                 int n, int32_t* granted, void* workspace, hipStream_t stream) {
  return launch_fork<true>(c, s, parents, children, n, granted, workspace, stream);
}

hipError_t launch_cache_accept(const CacheArgs& c, const int32_t* seq_ids, int n, const int32_t* path, int max_path,
                               const int32_t* counts, int32_t* new_lengths, hipStream_t stream) {
  const size_t lds = (size_t)max_path * c.head_dim * 4;
  const bool in_place = new_lengths == c.lengths;
  accept_kernel<<<dim3(n + !in_place, c.layers, c.heads), 256, lds, stream>>>(c, seq_ids, n, path, max_path, counts,
                                                                              new_lengths);
  if (in_place)
    accept_lengths_kernel<<<1, kPlan, 0, stream>>>(c, seq_ids, n, max_path, counts, new_lengths);
  return hipGetLastError();
}

hipError_t launch_cache_accept_kv8(const CacheArgs& c, const Scales& s, const int32_t* seq_ids, int n,
                                   const int32_t* path, int max_path, const int32_t* counts, int32_t* new_lengths,
                                   hipStream_t stream) {
  const size_t lds = (size_t)max_path * c.head_dim * 2;
  const bool in_place = new_lengths == c.lengths;
  accept_kv8_kernel<<<dim3(n + !in_place, c.layers, c.heads), 256, lds, stream>>>(c, s, seq_ids, n, path, max_path,
                                                                                  counts, new_lengths);
  if (in_place)
    accept_lengths_kernel<<<1, kPlan, 0, stream>>>(c, seq_ids, n, max_path, counts, new_lengths);
  return hipGetLastError();
}

hipError_t launch_cache_free(const CacheArgs& c, const int32_t* seq_ids, int n, hipStream_t stream) {
  free_kernel<<<n, 256, 0, stream>>>(c, seq_ids);
  return hipGetLastError();
}

}  // namespace trellis
