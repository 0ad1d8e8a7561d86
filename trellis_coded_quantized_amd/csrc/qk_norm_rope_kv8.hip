// qk_norm_rope_kv8.hip -- RMS norm of every query and key head, rotation by
// position, and the append of keys and values to the cache held in 8 bits.
#include "internal.hpp"
#include "kv8_common.hpp"
#include "norm_rope.hpp"

namespace trellis {
namespace {

constexpr int TB = 8;             // tokens of a workgroup that has queries

// The largest number of the 16-bit type with 4 significant bits: a larger one
// could not come back from e4m3 and a scale.
template <typename T>
__device__ __forceinline__ float type_top() {
  return __builtin_bit_cast(float, T::kExp == 0x7F80u ? 0x7F700000u : 0x47700000u);   // 1.875 2^127, 61440
}

// Infinities become NaN, magnitudes end at the type's top; returns the largest
// finite one.  Few waves have either, and a sum tells.
template <typename T>
__device__ __forceinline__ float tame(float (&y)[8]) {
  float top = 0.0f, sum = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    top = fmaxf(top, fabsf(y[e]));
    sum += fabsf(y[e]);
  }
  if (!__any(!(sum < INFINITY) || top > type_top<T>())) return top;
  top = 0.0f;
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

// The largest over eight neighbouring lanes, in the last of them (x >= 0).
__device__ __forceinline__ float max_of_eight(float x) {
  int v = __builtin_bit_cast(int, x);                        // magnitudes order as their bits
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true));   // row_shr:1
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true));   // row_shr:2
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true));   // row_shr:4
  return __builtin_bit_cast(float, v);
}

// Rows a, b, c, d of four bytes each -> out[i]: byte i of all four.
__device__ __forceinline__ void turn_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&out)[4]) {
  const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x05010400u), cd = __builtin_amdgcn_perm(d, c, 0x05010400u);
  const uint32_t AB = __builtin_amdgcn_perm(b, a, 0x07030602u), CD = __builtin_amdgcn_perm(d, c, 0x07030602u);
  out[0] = __builtin_amdgcn_perm(cd, ab, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(cd, ab, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(CD, AB, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(CD, AB, 0x07060302u);
}

template <int D>
struct Shape {
  static constexpr int THREADS = D == 256 ? 512 : 256, LANES = D / 8, GROUPS = THREADS / LANES;
  static constexpr int PER = 2, UNITS = GROUPS * PER;        // (head, token) pairs at a time
  static constexpr int WINDOW = 16, MOST = WINDOW + 15;      // tokens of the list, tokens of its runs
  static_assert(UNITS >= MOST, "one head of all runs");
};

// Queries.  As in the 16-bit append: a workgroup takes TB tokens and a share of
// the heads, D / 8 lanes a head.
template <typename T, int D, bool PAIRS>
__device__ void queries(const QkNormRope8Args& a, int64_t first, int share, int shares, float (*s_cos)[D / 2],
                        float (*s_sin)[D / 2]) {
  constexpr int LANES = Shape<D>::LANES, GROUPS = Shape<D>::GROUPS;
  const int tokens = (int)min((int64_t)TB, a.tokens - first), half = a.rotary / 2;
  const int tid = threadIdx.x, grp = tid / LANES, d0 = tid % LANES * 8;
  const int h0 = (int)((int64_t)a.heads_q * share / shares), h1 = (int)((int64_t)a.heads_q * (share + 1) / shares);
  for (int x = tid; x < tokens * half; x += Shape<D>::THREADS) {
    const int t = x / half, i = x - t * half;
    turn(a.positions[first + t], a.inv_freq[i], s_cos[t][i], s_sin[t][i]);
  }
  __syncthreads();
  // four heads of a group at a time: their loads go together
  constexpr int AHEAD = 4;
  const int all = (h1 - h0) * TB;
  auto source = [&](int x) { return a.q + (first + x % TB) * a.q_stride + (h0 + x / TB) * D + d0; };
  for (int x0 = grp; x0 < all; x0 += AHEAD * GROUPS) {
    u32x4v raw[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int x = x0 + k * GROUPS;
      raw[k] = u32x4v{};
      if (x < all && x % TB < tokens) raw[k] = *reinterpret_cast<const u32x4v*>(source(x));
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int x = x0 + k * GROUPS, h = h0 + x / TB, t = x % TB;
      if (x >= all || t >= tokens) continue;
      float y[8];
      norm_rotate<T, D, PAIRS>(raw[k], source(x), a.q_weight + d0, d0, a.rotary, a.eps, s_cos[t], s_sin[t], y);
      u32x4v res;
#pragma unroll
      for (int w = 0; w < 4; ++w) res[w] = T::pack(y[2 * w], y[2 * w + 1]);
      *reinterpret_cast<u32x4v*>(a.out + ((first + t) * a.heads_q + h) * D + d0) = res;
    }
  }
}

// Keys and values.  A block of 16 slots has one owner, so that its scale and
// its rows change together: the workgroup that has the first of the block's
// tokens (a run; at most 16) in its window of the list.  All runs of a window
// are worked on at once, some heads at a time, one (head, token) to D / 8 lanes:
// values in registers, the blocks' largest magnitudes through LDS, codes
// through LDS into the cache's order, so that whole blocks leave as whole
// granules.  Of other blocks new tokens are written alone, and all of a block
// that has to be rounded again.
// One run: its block and what it gets.
struct Run {
  int first, n;                   // tokens, counted from the window's first
  uint32_t places;                // of the block's 16
  int64_t keys, values, scales;   // bytes of head 0 of the block in the pools; its scale
};

template <typename T, int D, bool PAIRS>
__device__ void keys_values(const QkNormRope8Args& a, int64_t first, int window, int share, int shares,
                            float (*s_cos)[D / 2], float (*s_sin)[D / 2]) {
  typedef Shape<D> S;
  constexpr int LANES = S::LANES, GROUPS = S::GROUPS, PER = S::PER, UNITS = S::UNITS, THREADS = S::THREADS;
  // by unit: keys [D/16][16], values [D]; of the units of a whole block, keys
  // [D/16][place][16] and values [place][D] of a head
  __shared__ __align__(16) uint8_t s_code[2][UNITS * D];
  __shared__ uint32_t s_top[2][UNITS], s_old[2][UNITS], s_new[2][UNITS];      // by (run, head)
  __shared__ Run s_run[S::WINDOW];
  __shared__ uint32_t s_full;                                // runs that are whole blocks, a bit each
  __shared__ int s_of[S::MOST], s_place[S::MOST];            // a token's run (-1: none), its place in the block
  const int tid = threadIdx.x, lane = tid & 63, grp = tid / LANES, l = tid % LANES, d0 = l * 8;
  const int half = a.rotary / 2, P = 1 << a.page_log2;
  const int v0 = (int)((int64_t)a.heads_kv * share / shares), v1 = (int)((int64_t)a.heads_kv * (share + 1) / shares);
  const int64_t head_bytes = (int64_t)D << a.page_log2;

  // lane j of every wave looks at token first - 1 + j: which begin a run, which go on with one
  const int64_t tok = first - 1 + lane;
  const int slot = tok >= 0 && tok < a.tokens ? a.slots[tok] : -1;
  const bool cached = slot >= 0 && (uint32_t)(slot >> a.page_log2) < a.pages;
  const int block = cached ? slot >> 4 : -1;
  const int before = __shfl_up(block, 1);
  const uint64_t goes_on = __ballot(cached && lane > 0 && block == before);
  const uint64_t begins = __ballot(cached && lane > 0 && lane <= window && block != before);
  if (begins == 0) return;
  const int runs = __builtin_popcountll(begins);
  // the run that begins at lane j: its tokens
  auto length = [&](int j) { return min(16, 1 + __builtin_ctzll(~(goes_on >> (j + 1)))); };
  const int j0 = __builtin_ctzll(begins), j1 = 63 - __builtin_clzll(begins);
  const int n = j1 + length(j1) - j0;                        // tokens from the first run's first to the last one's last
  const int64_t t0 = first - 1 + j0;
  if (tid < 64) {
    // a token is in the last run that began, if that is not over
    const uint64_t upto = begins & (~0ull >> (63 - lane));
    const int mine = upto ? 63 - __builtin_clzll(upto) : 0;
    const bool in = cached && upto && lane < mine + length(mine);
    if (lane >= j0 && lane < j0 + n) {
      s_of[lane - j0] = in ? __builtin_popcountll(upto) - 1 : -1;
      s_place[lane - j0] = slot & 15;
    }
    if (lane < S::WINDOW) s_run[lane].places = 0;
    if ((begins >> lane) & 1) {
      Run& r = s_run[__builtin_popcountll(upto) - 1];
      const int64_t page = slot >> a.page_log2;
      const int in_page = (slot & (P - 1)) >> 4;
      r.first = lane - j0;
      r.n = length(lane);
      r.keys = page * a.heads_kv * head_bytes + in_page * 256;
      r.values = page * a.heads_kv * head_bytes + in_page * D * 16;
      r.scales = ((page * a.heads_kv) << (a.page_log2 - 4)) + in_page;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    if (in && lane >= j0 && lane < j0 + n) atomicOr(&s_run[__builtin_popcountll(upto) - 1].places, 1u << (slot & 15));
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    const uint32_t full = (uint32_t)__ballot(lane < runs && s_run[lane % S::WINDOW].places == 0xFFFFu);
    if (lane == 0) s_full = full;
  }
  for (int x = tid; x < n * half; x += THREADS) {
    const int t = x / half, i = x - t * half;
    turn(a.positions[t0 + t], a.inv_freq[i], s_cos[t][i], s_sin[t][i]);
  }
  const int batch = min(UNITS / n, v1 - v0);                 // heads at a time
  const int64_t scale_heads = (int64_t)P >> 4;               // scales from a head to the next
  for (int hb = v0; hb < v1; hb += batch) {
    const int heads = min(batch, v1 - hb), units = heads * n, blocks = heads * runs;
    // unit -> head and token of the window
    auto head_of = [&](int u) { return n == 16 ? u >> 4 : u / n; };
    u32x4v rk[PER], rv[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int u = min(grp + i * GROUPS, units - 1), h = head_of(u), t = u - h * n;
      rk[i] = *reinterpret_cast<const u32x4v*>(a.k + (t0 + t) * a.k_stride + (hb + h) * D + d0);
      rv[i] = *reinterpret_cast<const u32x4v*>(a.v + (t0 + t) * a.v_stride + (hb + h) * D + d0);
    }
    __syncthreads();                                         // the runs are there; the batch before is done with LDS
    int grown = 0;
    const uint32_t full = s_full;
    for (int x = tid; x < 2 * blocks; x += THREADS) {
      const int which = x & 1, r = (x >> 1) / heads, h = (x >> 1) - r * heads;
      s_top[which][x >> 1] = 0;
      s_old[which][x >> 1] =
          s_run[r].places & 1u ? 0u : (which ? a.v_scale : a.k_scale)[s_run[r].scales + (hb + h) * scale_heads];
    }
    __syncthreads();
    float yk[PER][8], yv[PER][8];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int u = grp + i * GROUPS;
      if (u >= units) continue;
      const int h = head_of(u), t = u - h * n, r = s_of[t];
      norm_rotate<T, D, PAIRS>(rk[i], a.k + (t0 + t) * a.k_stride + (hb + h) * D + d0, a.k_weight + d0, d0, a.rotary,
                               a.eps, s_cos[t], s_sin[t], yk[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) yv[i][e] = T::to_f32((uint16_t)(rv[i][e >> 1] >> (16 * (e & 1))));
      const float kt = max_of_eight(tame<T>(yk[i])), vt = max_of_eight(tame<T>(yv[i]));
      if ((l & 7) == 7 && r >= 0) {
        atomicMax(&s_top[0][r * heads + h], __builtin_bit_cast(uint32_t, kt));
        atomicMax(&s_top[1][r * heads + h], __builtin_bit_cast(uint32_t, vt));
      }
    }
    __syncthreads();
    for (int x = tid; x < 2 * blocks; x += THREADS) {
      const int which = x & 1, r = (x >> 1) / heads, h = (x >> 1) - r * heads;
      const uint32_t old = s_old[which][x >> 1], now = max(old, scale_byte(s_top[which][x >> 1]));
      s_new[which][x >> 1] = now;
      grown |= !(s_run[r].places & 1u) && now != old;
      if ((s_run[r].places & 1u) || now != old)
        (which ? a.v_scale : a.k_scale)[s_run[r].scales + (hb + h) * scale_heads] = (uint8_t)now;
    }
    grown = __syncthreads_or(grown);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int u = grp + i * GROUPS;
      if (u >= units) continue;
      const int h = head_of(u), t = u - h * n, r = s_of[t];
      if (r < 0) continue;
      const float ki = inverse_scale(s_new[0][r * heads + h]), vi = inverse_scale(s_new[1][r * heads + h]);
      const u32x2v kc = {codes4(yk[i][0] * ki, yk[i][1] * ki, yk[i][2] * ki, yk[i][3] * ki),
                         codes4(yk[i][4] * ki, yk[i][5] * ki, yk[i][6] * ki, yk[i][7] * ki)};
      const u32x2v vc = {codes4(yv[i][0] * vi, yv[i][1] * vi, yv[i][2] * vi, yv[i][3] * vi),
                         codes4(yv[i][4] * vi, yv[i][5] * vi, yv[i][6] * vi, yv[i][7] * vi)};
      if ((full >> r) & 1) {
        const int base = (h * n + s_run[r].first) * D;       // of the block's units
        *reinterpret_cast<u32x2v*>(&s_code[0][base + ((l >> 1) * 16 + s_place[t]) * 16 + (l & 1) * 8]) = kc;
        *reinterpret_cast<u32x2v*>(&s_code[1][base + s_place[t] * D + d0]) = vc;
      } else {
        *reinterpret_cast<u32x2v*>(&s_code[0][u * D + d0]) = kc;
        *reinterpret_cast<u32x2v*>(&s_code[1][u * D + d0]) = vc;
      }
    }
    __syncthreads();

    for (uint32_t left = full; left; left &= left - 1) {     // whole blocks
      const Run& run = s_run[__builtin_ctz(left)];
      uint8_t* const kd = a.k8 + run.keys + hb * head_bytes;
      uint8_t* const vd = a.v8 + run.values + hb * head_bytes;
      const uint8_t *kc = &s_code[0][run.first * D], *vc = &s_code[1][run.first * D];
      for (int x = tid; x < heads * D; x += THREADS)
        *reinterpret_cast<u32x4v*>(kd + x / D * head_bytes + (x % D >> 4) * P * 16 + (x & 15) * 16) =
            *reinterpret_cast<const u32x4v*>(kc + x / D * (n * D) + x % D * 16);
      for (int x = tid; x < heads * D / 4; x += THREADS) {
        const int d = x % (D / 4) * 4, h = x / (D / 4);
        u32x4v g[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t row[4], out[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) row[e] = *reinterpret_cast<const uint32_t*>(vc + (h * n + w * 4 + e) * D + d);
          turn_bytes(row[0], row[1], row[2], row[3], out);
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e][w] = out[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<u32x4v*>(vd + h * head_bytes + (d + e) * 16) = g[e];
      }
    }
    // new tokens of the others: granules of keys, bytes of values (a lane has one
    // dimension of all a run's tokens: 8 trees of 5 tokens 6.5 us, a byte a lane 7.6)
    const bool rest = full != (1u << runs) - 1;
    for (int x = tid; rest && x < units * (D / 16); x += THREADS) {
      const int u = x / (D / 16), g = x % (D / 16), h = head_of(u), t = u - h * n, r = s_of[t];
      if (r < 0 || (full >> r) & 1) continue;
      *reinterpret_cast<u32x4v*>(a.k8 + s_run[r].keys + (hb + h) * head_bytes + (g * P + s_place[t]) * 16) =
          *reinterpret_cast<const u32x4v*>(&s_code[0][x * 16]);
    }
    for (int x = tid; rest && x < blocks * D; x += THREADS) {
      const int b = x / D, d = x % D, r = b / heads, h = b - r * heads;
      const Run& run = s_run[r];
      if ((full >> r) & 1 || (!(run.places & 1u) && s_new[1][b] != s_old[1][b])) continue;   // grew: below
      uint8_t* const at = a.v8 + run.values + (hb + h) * head_bytes + d * 16;
      const uint8_t* const code = &s_code[1][h * n * D + d];
      for (int t = run.first, end = t + run.n; t < end; ++t) at[s_place[t]] = code[t * D];
    }
    // blocks whose scale grew: their other keys, and values as whole granules
    for (int x = tid; grown && x < blocks * D; x += THREADS) {
      const int b = x / D, y = x % D, r = b / heads, h = b - r * heads;
      const Run& run = s_run[r];
      if (run.places & 1u) continue;
      const uint32_t k0 = s_old[0][b], k1 = s_new[0][b], w0 = s_old[1][b], w1 = s_new[1][b];
      if (k1 != k0 && !((run.places >> (y & 15)) & 1)) {
        u32x4v* at = reinterpret_cast<u32x4v*>(a.k8 + run.keys + (hb + h) * head_bytes + ((y >> 4) * P + (y & 15)) * 16);
        *at = rescaled(*at, k0, k1);
      }
      if (w1 != w0) {
        u32x4v* at = reinterpret_cast<u32x4v*>(a.v8 + run.values + (hb + h) * head_bytes + y * 16);
        u32x4v g = rescaled(*at, w0, w1);
        for (int t = run.first; t < run.first + run.n; ++t) {
          const int off = s_place[t], by = (off & 3) * 8;
          const uint32_t c = (uint32_t)s_code[1][(h * n + t) * D + y] << by, out = ~(0xFFu << by);
#pragma unroll
          for (int w = 0; w < 4; ++w) g[w] = off >> 2 == w ? (g[w] & out) | c : g[w];
        }
        *at = g;
      }
    }
  }
}

template <typename T, int D, bool PAIRS>
__global__ __launch_bounds__(Shape<D>::THREADS, 4) void qk_norm_rope_kv8_kernel(QkNormRope8Args a, int window, int kv_blocks,
                                                                               int kv_shares, int q_shares) {
  __shared__ __align__(16) float s_cos[Shape<D>::MOST][D / 2], s_sin[Shape<D>::MOST][D / 2];
  // the two kinds in turn, so that queries' loads and stores go on while keys
  // and values wait at their barriers (8191 tokens, 32 / 8 heads of 128: one
  // after the other in two launches 48 us, in turn 45; 185 MB at the copy's rate
  // are 36).  Bound by vector work: it issues in 80 % of the cycles (norms, angles,
  // conversions and largest magnitudes, weights converted for every head).
  // Registers for more waves spill (96 of them: 57.1 against 56.8 us in a graph,
  // 68 against 63 at 256 dimensions, 28 against 26 at 64; 80: 71, 83, 44), and
  // so do the next heads' loads ahead of this batch's stores (57 us either way,
  // 256 dimensions 72 against 66).
  const uint64_t b = blockIdx.x;
  const int k = (int)(b * (uint64_t)kv_blocks / gridDim.x), q = (int)b - k;
  if ((int)((b + 1) * (uint64_t)kv_blocks / gridDim.x) > k)
    keys_values<T, D, PAIRS>(a, (int64_t)(k / kv_shares) * window, window, k % kv_shares, kv_shares, s_cos, s_sin);
  else
    queries<T, D, PAIRS>(a, (int64_t)(q / q_shares) * TB, q % q_shares, q_shares, s_cos, s_sin);
}

template <typename T, int D, bool PAIRS>
hipError_t launch(const QkNormRope8Args& a, hipStream_t stream) {
  typedef Shape<D> S;
  const int cus = device_cus();
  auto shared = [](int64_t have, int64_t want, int64_t most) {
    const int64_t s = want / have;
    return (int)(s > most ? most : s < 1 ? 1 : s);
  };
  const int64_t q_groups = (a.tokens + TB - 1) / TB;
  const int rounds = a.heads_q * TB * S::LANES / S::THREADS; // of a workgroup with all query heads
  const int q_shares = shared(q_groups, 4 * cus, rounds < 1 ? 1 : rounds > 64 ? 64 : rounds);
  // Few tokens: a workgroup each, which may find that its run began before.  Of
  // 32 / 8 heads of 128 (a workgroup each / 16 together, us): 64 single tokens
  // 6.8 / 9.3, 128 7.8 / 10.0, 192 10.0 / 10.4, 256 11.9 / 11.3; one of 64 8.6 / 9.7,
  // 160 9.8 / 9.7, 256 11.9 / 9.9, 512 20 / 11; heads of 64 even out at 128 already
  // (7.9 / 7.7), 8 / 1 of 128 past 512.
  const int window = a.tokens > 128 ? S::WINDOW : 1;
  const int64_t windows = (a.tokens + window - 1) / window;
  // Many windows: enough workgroups for 512 / D a compute unit (8191 tokens:
  // 16 / 16 heads of 64 37 us with 2 shares a window, 30 with 4; 32 / 8 of 128
  // 57 with 2, 70 with 1; 24 / 4 of 256 81 with 2, 66 with 1).  Few: a share a
  // head, since the batches of a window take turns (300 tokens: 12.2 us with 8
  // shares, 19.5 with 4, when tokens of open blocks were slower; 10.0 now); but where a window is one token, not fewer heads than
  // fill a workgroup (64 tokens, 16 heads of 64: 6.6 us with 4, 9.7 with 16).
  const int64_t most = window == 1 ? (a.heads_kv * 16 + S::UNITS - 1) / S::UNITS : a.heads_kv;
  const int kv_shares = shared(windows, cus * (512 / D), most);
  const int64_t kv = windows * kv_shares, blocks = kv + q_groups * q_shares;
  if (blocks >= ((int64_t)1 << 31) / S::THREADS * 2) return hipErrorInvalidValue;
  qk_norm_rope_kv8_kernel<T, D, PAIRS><<<(unsigned)blocks, S::THREADS, 0, stream>>>(a, window, (int)kv, kv_shares, q_shares);
  return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_pairs(const QkNormRope8Args& a, hipStream_t stream) {
  return a.interleaved ? launch<T, D, true>(a, stream) : launch<T, D, false>(a, stream);
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
