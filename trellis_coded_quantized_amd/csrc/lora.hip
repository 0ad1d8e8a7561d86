// lora.hip -- low-rank adapters of many requests beside shared projections.
//
// Row m of entry e with adapter a:  t = A_a x_m,  y'_m = y_m + s_a B_a t.
// The first product reads x and A once and leaves f32 partial sums of its
// column chunks in the workspace; the second one adds them up, reads B and y
// and writes y'.  Two launches: every output needs the whole of t.
//
// Bound by memory where entries are long: 8191 rows, 6144 -> 5120, rank 16,
// 21 + 40 us traced, 4.8 and 4.2 TB/s of the copy's 5.1.  Gate and up of 5120
// -> 17408 for 2047 rows, rank 64, bf16: 15 + 65 us (239 MB and 7.7 GFLOP
// least); the second product has two workgroups a compute unit for its
// registers and LDS, which wait 41 % of their time, while nothing is saturated
// (vector issue 47 %, matrix units 18 %).  64 rows, 48 adapters of rank 32, three
// matrices: 10 + 10 us over 45 MB; a wave has two or three steps of work behind
// a chain of dependent loads (starts, adapter, rank).  One row: 4.7 + 5.5 us,
// latencies.
#include "internal.hpp"
#include "kv_common.hpp"
#include <type_traits>

namespace trellis {
namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr unsigned kXcds = 8;
constexpr int kCols = 32 * kWaves;    // columns that a workgroup's waves take at a time

// Rows of one entry that a workgroup takes: one MFMA tile where entries are
// short, two (first product) and four (second product) where they are long:
// gate and up of 2047 rows, rank 64, with 32 / 64 / 128 rows in the second
// product 125 / 89 / 148 us (operands of B read for each tile; registers), 8191
// rows of rank 16 78 / 72 / 84, though three matrices in f32 of 2047 rows 47 / 51 /
// 56; tiles of 16 rows in the first one 2 - 7 % faster up to 1024 rows, and from
// 2047 on between 1 % faster and 5 % slower.
constexpr int kShort = 16, kLongShrink = 32, kLongExpand = 64;

struct Tile {
  int e, first, rows;             // entry, its first row of the tile, rows
  int adapter, rank;
  bool live;
};

// Slot -> entry and row tile, 64 entries at a time, one a lane; `bare`: entries
// without an adapter have tiles too.
__device__ __forceinline__ Tile find_tile(const LoraArgs& a, int slot, int tile, bool bare) {
  const int lane = threadIdx.x & 63;
  Tile t{};
  int before = 0;
  for (int b = 0; b < a.entries; b += 64) {
    const int e = b + lane;
    int first = 0, rows = 0, adapter = -1, rank = 0;
    if (e < a.entries) {
      const int from = a.starts[e], to = a.starts[e + 1];
      adapter = a.adapters[e];
      first = min(max(from, 0), (int)a.M);
      rows = min(max(to, first), (int)a.M) - first;
      if (adapter < 0 || adapter >= a.pool) adapter = -1;
      if (adapter >= 0) rank = a.ranks ? min(max(a.ranks[adapter], 0), a.r) : a.r;
      if (rank == 0) adapter = -1;
      if (adapter < 0 && !bare) rows = 0;
    }
    const int tiles = (rows + tile - 1) / tile, upto = wave_scan_add(tiles);
    const uint64_t hit = __ballot(before + upto > slot);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      const int u = slot - before - __builtin_amdgcn_readlane(upto, at) + __builtin_amdgcn_readlane(tiles, at);
      t.e = b + at;
      t.first = __builtin_amdgcn_readlane(first, at) + u * tile;
      t.rows = min(tile, __builtin_amdgcn_readlane(rows, at) - u * tile);
      t.adapter = __builtin_amdgcn_readlane(adapter, at);
      t.rank = __builtin_amdgcn_readlane(rank, at);
      t.live = true;
      return t;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return t;
}

__device__ __forceinline__ f32x4v mfma16(u32x4v a, u32x4v b, f32x4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// ---- t = A x -------------------------------------------------------------
// N matrices (from `first_target` on) over one x, RT tiles of 16 ranks each, RM
// tiles of 16 rows, a chunk of columns a workgroup, whose four waves take steps
// of WIDE columns in turn.  The result has the row of x in the lane and four
// ranks in its registers.
//
// Operands have neighbouring lanes on neighbouring rows, C elements apart.
// Loaded like that, every lane of 16 bytes is a request of its own to the L1
// (counted: 63 of them a load; the second product, whose loads were like that,
// was bound by them: 2047 rows of gate and up 109 us then, 84 with both
// products' loads along rows).  So a tile is loaded with neighbouring lanes along its
// rows, and turned in LDS, a wave's own: granule g of row r lies at g ^ turn(r),
// which keeps 16 rows' granules on different banks.  Its registers are free for
// the next step's loads before this one's products run.
template <int WIDE>
struct Turn {
  static constexpr int GRANS = WIDE / 8, ROWS = 64 / GRANS, LOADS = 16 / ROWS;   // a row's granules, rows of a load
  static __device__ __forceinline__ int at(int row, int g) {
    return row * GRANS + (g ^ (GRANS == 8 ? (row & 7) ^ (row >> 3) : row >> 2));
  }
};

template <int N, int RT, int RM>
__global__ __launch_bounds__(kThreads, 2) void lora_shrink_kernel(LoraArgs a) {
  constexpr int NT = N * RT, TILES = RM + NT, WIDE = TILES <= 5 ? 64 : 32;    // 40 KB of LDS at most
  typedef Turn<WIDE> T;
  __shared__ __align__(16) u32x4v s_tile[kWaves][TILES][16 * T::GRANS];
  static_assert(sizeof(s_tile) <= 40960 && sizeof(f32x4v) * 64 * RM * NT <= sizeof(s_tile[0]) * 2, "LDS of the sums");
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.x / a.splits, split = blockIdx.x - slot * a.splits;
  const Tile t = find_tile(a, slot, RM * 16, false);
  if (!t.live) return;
  const int lr = lane / T::GRANS, lg = lane % T::GRANS;      // this lane's row of a load, and its granule
  const uint16_t* src[TILES][T::LOADS];
#pragma unroll
  for (int l = 0; l < T::LOADS; ++l) {
#pragma unroll
    for (int m = 0; m < RM; ++m)
      src[m][l] = a.x + (int64_t)(t.first + min(m * 16 + l * T::ROWS + lr, t.rows - 1)) * a.x_stride + lg * 8;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      // ranks past the adapter's are read as its last: nothing reads their sums
      src[RM + n][l] = a.target[a.first_target + n / RT].a +
                       ((int64_t)t.adapter * a.r + min(n % RT * 16 + l * T::ROWS + lr, t.rank - 1)) * a.C + lg * 8;
  }
  const int64_t c0 = (int64_t)split * a.chunk, c1 = min(a.C, c0 + a.chunk);
  u32x4v in[TILES][T::LOADS];
  auto load = [&](int64_t c) __attribute__((always_inline)) {
    if (c + WIDE <= c1) {
#pragma unroll
      for (int k = 0; k < TILES; ++k)
#pragma unroll
        for (int l = 0; l < T::LOADS; ++l) in[k][l] = *reinterpret_cast<const u32x4v*>(src[k][l] + c);
    } else {
      const bool have = c + lg * 8 < c1;                     // whole granules: C and chunks are multiples of 8
#pragma unroll
      for (int k = 0; k < TILES; ++k)
#pragma unroll
        for (int l = 0; l < T::LOADS; ++l) {
          in[k][l] = u32x4v{};
          if (have) in[k][l] = *reinterpret_cast<const u32x4v*>(src[k][l] + c);
        }
    }
  };
  f32x4v acc[RM][NT] = {};
  int64_t c = c0 + wave * WIDE;
  if (c < c1) load(c);
  for (; c < c1; c += kWaves * WIDE) {
#pragma unroll
    for (int k = 0; k < TILES; ++k)
#pragma unroll
      for (int l = 0; l < T::LOADS; ++l) s_tile[wave][k][T::at(l * T::ROWS + lr, lg)] = in[k][l];
    if (c + kWaves * WIDE < c1) load(c + kWaves * WIDE);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
#pragma unroll
    for (int s = 0; s < WIDE / 32; ++s) {
      u32x4v x[RM];
#pragma unroll
      for (int m = 0; m < RM; ++m) x[m] = s_tile[wave][m][T::at(col, s * 4 + grp)];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const u32x4v w = s_tile[wave][RM + n][T::at(col, s * 4 + grp)];
#pragma unroll
        for (int m = 0; m < RM; ++m) acc[m][n] = mfma16(w, x[m], acc[m][n]);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  }
  // the waves' sums, two waves at a time: waves 2 and 3 give theirs to 0 and 1, then 1 to 0
  f32x4v* const sums = reinterpret_cast<f32x4v*>(s_tile);
#pragma unroll
  for (int half = 2; half; half >>= 1) {
    __syncthreads();
    if (wave >= half && wave < 2 * half)
#pragma unroll
      for (int k = 0; k < RM * NT; ++k) sums[((wave - half) * RM * NT + k) * 64 + lane] = acc[k / NT][k % NT];
    __syncthreads();
    if (wave < half)
#pragma unroll
      for (int k = 0; k < RM * NT; ++k) acc[k / NT][k % NT] += sums[(wave * RM * NT + k) * 64 + lane];
  }
  if (wave) return;
#pragma unroll
  for (int k = 0; k < RM * NT; ++k) {
    const int m = k / NT * 16 + col, n = k % NT, j = n % RT * 16 + grp * 4;
    if (m < t.rows && j < a.r)
      *reinterpret_cast<f32x4v*>(a.part + ((int64_t)split * a.M + t.first + m) * (a.n * a.r) +
                                 (a.first_target + n / RT) * a.r + j) = acc[k / NT][n];
  }
}

// ---- y + s B t -----------------------------------------------------------
// t enters as three bf16 numbers, which hold its 24 bits.  Two hold 16, too few
// for bf16 outputs also: where y or another rank's product cancels the rest,
// the dropped bits are what is left (gate and up of 2047 rows, rank 64: 84.6 us
// with two, 87.6 with three; 8191 rows, rank 16: 72.5 and 72.9).  The
// contraction is (part, rank), in units of eight ranks, four units a matrix
// instruction, and an operand of B serves all parts.  MFMA row 4 g + e of
// instruction q is output 8 g + 4 q + e, so two instructions leave eight
// neighbouring outputs of a row in a lane.
//
// 32 rows of B are one stretch of memory; they are loaded as that and turned
// into operands in LDS, a wave's own: unit k of row i lies at k ^ turn(i), which
// keeps the rows of an instruction on different banks.
//
// Infinities and NaN of B meet the first part alone, which has t's sign: a
// lower part is often zero or of the other sign, and inf * 0 and inf - inf are
// NaN where B t is infinite.  Whether a wave's rows of B hold any is seen as
// they enter LDS (64 rows, rank 64: 3 % of a call; others 1 %).
constexpr int PARTS = 3;

template <int NB>
struct Units {
  static constexpr int LOADS = NB < 2 ? 1 : NB / 2;          // of a wave, for 32 rows
  static __device__ __forceinline__ int at(int i, int k) {
    const int turn = NB == 8 ? (i >> 3) * 2 + ((i >> 1) & 1) : NB == 4 ? i >> 3 : NB == 2 ? (i >> 3) & 1 : 0;
    return i * NB + (k ^ turn);
  }
  static constexpr int MFMAS = (PARTS * NB + 3) / 4, OPERANDS = NB < 4 ? 1 : NB / 4;
  static __device__ __forceinline__ int block(int q, int grp) { return NB < 4 ? grp % NB : q % OPERANDS * 4 + grp; }
  static __device__ __forceinline__ int part(int q, int grp) { return (4 * q + grp) / NB; }
};

// A finite number past bf16's largest becomes that, and the next part the rest;
// rounded, it would be an infinity.
__device__ __forceinline__ float within_bf16(float v) {
  constexpr float kTop = 0x1.FEp127f;
  return fabsf(v) < INFINITY ? fminf(fmaxf(v, -kTop), kTop) : v;
}

// The signs' places of two bf16 numbers, set where one is an infinity or NaN:
// an exponent of all ones carries there when its last bit is added.
__device__ __forceinline__ uint32_t nonfinite(uint32_t two) { return ((two & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ bool any_nonfinite(u32x4v v) {
  return (nonfinite(v[0]) | nonfinite(v[1]) | nonfinite(v[2]) | nonfinite(v[3])) != 0;
}
// the same numbers, those as zeros
__device__ __forceinline__ u32x4v finite_ones(u32x4v v) {
#pragma unroll
  for (int w = 0; w < 4; ++w) v[w] &= ~((nonfinite(v[w]) >> 15) * 0xFFFFu);
  return v;
}

// g u / (1 + e^-g).  e^-g overflows from g = -88.7 on, and its reciprocal is lost
// from -87.3 on, where the product may still be far from zero.  So gates below
// -64, where it is g u e^g to f32, become -64 with what that leaves out in u.
// Waves that have none skip it (2047 rows, rank 64: 88.9 us, 87.7 without; with
// e^(g/2) on both factors and no branch 91.4).
__device__ __forceinline__ float silu_times(float g, float u) { return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u; }
__device__ __forceinline__ bool far_gate(float g) { return g < -64.0f; }
__device__ __forceinline__ void near_gate(float& g, float& u) {
  u *= far_gate(g) ? g * (-1.0f / 64) * __expf(g + 64.0f) : 1.0f;
  g = far_gate(g) ? -64.0f : g;
}

__device__ __forceinline__ float get_one(const float* p) { return *p; }
__device__ __forceinline__ float get_one(const uint16_t* p) { return Bf16::to_f32(*p); }
__device__ __forceinline__ void put_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void put_one(uint16_t* p, float v) { *p = (uint16_t)Bf16::pack(v, 0.0f); }

// 16 bytes of outputs as floats, and E floats as outputs
__device__ __forceinline__ void unpack(u32x4v w, float (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = __builtin_bit_cast(float, (uint32_t)w[e]);
}
__device__ __forceinline__ void unpack(u32x4v w, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = Bf16::to_f32((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
}
__device__ __forceinline__ void put(float* p, const float (&v)[4]) {
  *reinterpret_cast<f32x4v*>(p) = f32x4v{v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ void put(uint16_t* p, const float (&v)[4]) {
  *reinterpret_cast<u32x2v*>(p) = u32x2v{Bf16::pack(v[0], v[1]), Bf16::pack(v[2], v[3])};
}
__device__ __forceinline__ void put(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<u32x4v*>(p) =
      u32x4v{Bf16::pack(v[0], v[1]), Bf16::pack(v[2], v[3]), Bf16::pack(v[4], v[5]), Bf16::pack(v[6], v[7])};
}

// A wave takes MT tiles of 16 rows and SUB neighbouring blocks of 32 columns at
// a time; the workgroup's waves stand side by side.  Rows of B and of y are
// asked for together, the first ones before t is put together.  y is read and
// written with neighbouring lanes along a row, 64 or 128 bytes of it: the
// adapter's part of 16 rows goes there from the product's layout through LDS,
// a wave's own.
// WHOLE: rows of all matrices are 16-byte aligned and whole granules of eight;
// else outputs are read and written one by one.
// SWIGLU: targets 0 and 1 are gate and up, outputs go to target 0's out.
template <typename Y, int NB, int MT, int SUB, bool WHOLE, bool SWIGLU>
__global__ __launch_bounds__(kThreads, 2) void lora_expand_kernel(LoraArgs a) {
  typedef Units<NB> U;
  typedef typename std::conditional<SWIGLU, uint16_t, Y>::type Out;
  constexpr int R = NB * 8, G = SWIGLU ? 2 : 1, ROWS = MT * 16, STEP = SUB * 32 * kWaves;
  constexpr int E = 16 / sizeof(Y), ITEMS = 32 / E, Q = 16 * ITEMS / 64;      // outputs of a lane's item, items a row, a lane
  __shared__ __align__(16) uint16_t s_t[G][PARTS][ROWS][R + 8];               // padded: rows on different banks
  __shared__ __align__(16) float s_part[kWaves][16][32 + 4];
  __shared__ __align__(16) u32x4v s_b[kWaves][32 * NB];
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Workgroups of an XCD (every eighth) take neighbouring units, row tiles
  // innermost: what they read of B at a time is one column block's, which stays
  // in its L2.
  const int unit = (int)(blockIdx.x % kXcds * (gridDim.x / kXcds) + blockIdx.x / kXcds);
  int k = 0, block = unit / a.slots;                         // target and its column block
  const int slot = unit - block * a.slots;
  if (block >= a.blocks) return;
  if (!SWIGLU)
    while (block >= a.target[k].blocks) block -= a.target[k++].blocks;
  const Tile t = find_tile(a, slot, ROWS, a.bare);
  if (!t.live) return;
  const LoraTarget* const target = a.target + k;
  const bool on = t.adapter >= 0;
  if (!on && !SWIGLU && target->in_place) return;
  const int64_t out_n = target->R, end = min(out_n, (int64_t)(block + 1) * a.cols);
  int64_t c = (int64_t)block * a.cols + wave * 32 * SUB;

  // item q of this lane: row of a tile, first output of a block
  auto item_row = [&](int q) { return (q * 64 + lane) / ITEMS; };
  const int item_at = lane % ITEMS * E;
  struct Ahead {
    u32x4v b[G][SUB][U::LOADS], y[G][SUB][MT][Q];
  };
  auto load = [&](Ahead& to, int64_t c) __attribute__((always_inline)) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        if constexpr (WHOLE) {
          const int64_t i = min(c + u * 32 + item_at, out_n - E);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int q = 0; q < Q; ++q)
              to.y[g][u][m][q] = *reinterpret_cast<const u32x4v*>(
                  reinterpret_cast<const Y*>(target[g].y) +
                  (int64_t)(t.first + min(m * 16 + item_row(q), t.rows - 1)) * target[g].y_stride + i);
        }
        if (on) {
#pragma unroll
          for (int q = 0; q < U::LOADS; ++q) {
            // what B holds past the adapter's rank is cut below; the address stays inside the matrix
            const int64_t i = min(c + u * 32 + (q * 64 + lane) % (32 * NB) / NB, out_n - 1);
            to.b[g][u][q] = *reinterpret_cast<const u32x4v*>(target[g].b + ((int64_t)t.adapter * out_n + i) * R + lane % NB * 8);
          }
        }
      }
  };
  Ahead now, next;
  load(now, c);

  u32x4v keep[U::OPERANDS];
  if (on) {
    // the column chunks' sums, four ranks at a time: short entries may have many
    // chunks, and 16 lanes share them; long ones have few
    constexpr int SHARE = MT == 1 ? 16 : 1, QUADS = G * ROWS * R / 4;
    const float scale = a.scales[t.adapter];
    const int lead = tid % SHARE;
    for (int x = tid / SHARE; x < QUADS; x += kThreads / SHARE) {
      const int g = x / (ROWS * R / 4), m = x / (R / 4) % ROWS, j = x % (R / 4) * 4;
      if (m >= t.rows) continue;                             // those columns of the product are not looked at
      const float* part = a.part + (int64_t)(t.first + m) * (a.n * R) + (k + g) * R + j;
      const int64_t step = a.M * (a.n * R);
      f32x4v v = {};
#pragma unroll 4
      for (int s = lead; s < a.splits; s += SHARE) v += *reinterpret_cast<const f32x4v*>(part + s * step);
#pragma unroll
      for (int d = SHARE / 2; d; d >>= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += __shfl_xor(v[e], d);
      if (lead) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = j + e < t.rank ? v[e] * scale : 0.0f;
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
        float c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = p ? v[e] : within_bf16(v[e]);
        const u32x2v w = {Bf16::pack(c[0], c[1]), Bf16::pack(c[2], c[3])};
        *reinterpret_cast<u32x2v*>(&s_t[g][p][m][j]) = w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float rest = v[e] - Bf16::to_f32((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
          v[e] = fabsf(rest) < INFINITY ? rest : 0.0f;       // an infinity or NaN stands in the first part alone
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < U::OPERANDS; ++q) {                  // bits of the ranks that the adapter has
      const int have = t.rank - U::block(q, grp) * 8;
#pragma unroll
      for (int w = 0; w < 4; ++w) keep[q][w] = (have > 2 * w ? 0xFFFFu : 0u) | (have > 2 * w + 1 ? 0xFFFF0000u : 0u);
    }
  }

  auto block_of = [&](Ahead& from, int64_t c, const int u) __attribute__((always_inline)) {
    u32x4v b[G][U::OPERANDS][2];
    bool bad = false;                                        // infinities or NaN in these rows of B
    if (on) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int q = 0; q < U::LOADS; ++q) {
          const int unit = q * 64 + lane;
          bad |= any_nonfinite(from.b[g][u][q]);
          if (NB > 1 || unit < 32) s_b[wave][U::at(unit / NB, unit % NB)] = from.b[g][u][q];
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
#pragma unroll
        for (int q = 0; q < U::OPERANDS; ++q)
#pragma unroll
          for (int z = 0; z < 2; ++z)
            b[g][q][z] = s_b[wave][U::at((col >> 2) * 8 + z * 4 + (col & 3), U::block(q, grp))] & keep[q];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
      }
      bad = __any(bad);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m * 16 >= t.rows) continue;
      float d[Q][G][E];
#pragma unroll
      for (int x = 0; x < Q * G * E; ++x) d[x / (G * E)][x / E % G][x % E] = -0.0f;   // rows without an adapter: y + -0 is y
      if (on) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          f32x4v acc[2] = {};
          auto product = [&](auto careful) __attribute__((always_inline)) {
#pragma unroll
            for (int q = 0; q < U::MFMAS; ++q) {
              const int part = U::part(q, grp);
              u32x4v v = *reinterpret_cast<const u32x4v*>(&s_t[g][part < PARTS ? part : 0][m * 16 + col][U::block(q, grp) * 8]);
              if (PARTS * NB % 4 && part >= PARTS) v = u32x4v{};             // units past the last part
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                u32x4v w = b[g][q % U::OPERANDS][z];
                if (careful && part > 0) w = finite_ones(w);
                acc[z] = mfma16(w, v, acc[z]);
              }
            }
          };
          if (bad) product(std::true_type{});
          else product(std::false_type{});
#pragma unroll
          for (int z = 0; z < 2; ++z) *reinterpret_cast<f32x4v*>(&s_part[wave][col][grp * 8 + z * 4]) = acc[z];
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
#pragma unroll
          for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int e = 0; e < E; e += 4) {
              const f32x4v w = *reinterpret_cast<const f32x4v*>(&s_part[wave][item_row(q)][item_at + e]);
              d[q][g][e] = w[0], d[q][g][e + 1] = w[1], d[q][g][e + 2] = w[2], d[q][g][e + 3] = w[3];
            }
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
        }
      }
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int r = item_row(q);
        const int64_t i = c + u * 32 + item_at, row = t.first + m * 16 + r;
        if (i < end && m * 16 + r < t.rows) {
          Out* out = reinterpret_cast<Out*>(target->out) + row * target->out_stride + i;
          if constexpr (WHOLE) {
            float v[E];
            unpack(from.y[0][u][m][q], v);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] += d[q][0][e];
            if constexpr (SWIGLU) {
              float w[E];
              unpack(from.y[G - 1][u][m][q], w);
#pragma unroll
              for (int e = 0; e < E; ++e) w[e] += d[q][G - 1][e];
              float low = v[0];
#pragma unroll
              for (int e = 1; e < E; ++e) low = fminf(low, v[e]);
              if (__any(far_gate(low))) {
#pragma unroll
                for (int e = 0; e < E; ++e) near_gate(v[e], w[e]);
              }
#pragma unroll
              for (int e = 0; e < E; ++e) v[e] = silu_times(v[e], w[e]);
            }
            put(out, v);
          } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (i + e < out_n) {
                float v = get_one(reinterpret_cast<const Y*>(target->y) + row * target->y_stride + i + e) + d[q][0][e];
                if constexpr (SWIGLU) {
                  float w = get_one(reinterpret_cast<const Y*>(target[1].y) + row * target[1].y_stride + i + e) +
                            d[q][G - 1][e];
                  near_gate(v, w);
                  v = silu_times(v, w);
                }
                put_one(out + e, v);
              }
          }
        }
      }
    }
  };
  auto work = [&](Ahead& from, int64_t c) __attribute__((always_inline)) {
    block_of(from, c, 0);
    if constexpr (SUB > 1) block_of(from, c, 1);
    if constexpr (SUB > 2) block_of(from, c, 2), block_of(from, c, 3);
  };
  if constexpr (MT > 1 && !(SWIGLU && sizeof(Y) == 4)) {     // there registers do not reach for two sets
    // the next loads are asked for before this step's stores: loads and stores
    // are waited for in order
    while (c < end) {
      if (c + STEP < end) load(next, c + STEP);
      work(now, c);
      c += STEP;
      if (c >= end) break;
      if (c + STEP < end) load(now, c + STEP);
      work(next, c);
      c += STEP;
    }
  } else {
    while (c < end) {
      work(now, c);
      c += STEP;
      if (c < end) load(now, c);
    }
  }
}

// ---- launch --------------------------------------------------------------
int64_t slots_of(int64_t M, int entries, int rows) {
  const int64_t most = (M + rows - 1) / rows + entries;      // every entry's last tile may be a short one
  return M < most ? M : most;
}

}  // namespace

LoraPlan lora_plan(int64_t M, int entries, int64_t C, int n, int r) {
  LoraPlan p;
  // Short tiles read A and B once for 16 rows, in many column chunks; long ones
  // keep what they read for more rows.  Which is faster turns with the mean of
  // rows and with the rank, at about 16, 8, 4, 2 rows for 8, 16, 32, 64 (us, short
  // / long tiles, 5120 -> 6144 + 1024 + 1024 in bf16):
  //   rank 16, 256 entries of 1, 4, 8 rows: 34 / 53, 49 / 58, 56 / 64;
  //            32 of 8, 16, 24: 16.6 / 16.5, 20.3 / 17.9, 24.6 / 20.4
  //   rank 64, 16 of 1, 4, 8: 24.5 / 31.9, 27.9 / 31.6, 32.4 / 31.8
  // and gate and up, 5120 -> 17408:
  //   rank 16, 64 of 1, 8: 31 / 37, 40 / 43;  rank 64, 16 of 1, 2, 8: 28 / 31,
  //   31 / 32, 69 / 33, but 64 of 1 84 / 68.
  // A prompt among single tokens is cut as the mean says, up to a fifth slower than
  // the other way: rank 16, 1000 + 255 x 1 56 / 63, 1000 + 63 x 1 30 / 29,
  // 500 + 63 x 1 23 / 27; gate and up, rank 64, 4000 + 31 x 1 365 / 259, 500 + 255 x 1
  // 292 / 349.
  p.few = M * r <= 128 * (int64_t)entries;
  p.shrink_slots = slots_of(M, entries, p.few ? kShort : kLongShrink);
  p.expand_slots = slots_of(M, entries, p.few ? kShort : kLongExpand);
  // column chunks until the compute units have two workgroups, none shorter
  // than two steps of every wave.  Long entries: at most four, which every
  // workgroup of the second product adds up again (2047 rows of gate and up,
  // rank 64: 15 chunks 100 us, four 89).
  const int64_t want = 4 * (int64_t)device_cus() / (p.shrink_slots ? p.shrink_slots : 1), most = p.few ? 32 : 4;
  int64_t splits = (C + 255) / 256;
  if (splits > want) splits = want;
  if (splits > most) splits = most;
  if (splits < 1) splits = 1;
  p.chunk = ((C + splits - 1) / splits + 127) / 128 * 128;           // whole steps of all waves
  p.splits = (int)((C + p.chunk - 1) / p.chunk);
  p.bytes = ((size_t)p.splits * (size_t)M * n * r * 4 + 255) / 256 * 256;
  return p;
}

namespace {

template <int N, int RT>
void shrink(const LoraArgs& a, const LoraPlan& p, hipStream_t stream) {
  const unsigned grid = (unsigned)(p.shrink_slots * p.splits);
  if (p.few)
    lora_shrink_kernel<N, RT, kShort / 16><<<grid, kThreads, 0, stream>>>(a);
  else
    lora_shrink_kernel<N, RT, kLongShrink / 16><<<grid, kThreads, 0, stream>>>(a);
}

template <int RT>
void shrink_n(const LoraArgs& a, int n, const LoraPlan& p, hipStream_t stream) {
  switch (n) {
    case 1: return shrink<1, RT>(a, p, stream);
    case 2: return shrink<2, RT>(a, p, stream);
    case 3:
      if constexpr (RT <= 2) return shrink<3, RT>(a, p, stream);
      break;
    default:
      if constexpr (RT <= 2) return shrink<4, RT>(a, p, stream);
  }
}

template <typename Y, int NB, bool SWIGLU>
void expand(const LoraArgs& a, const LoraPlan& p, hipStream_t stream) {
  constexpr int LONG = kLongExpand / 16;
  const unsigned grid = (unsigned)((p.expand_slots * a.blocks + kXcds - 1) / kXcds * kXcds);
  auto kernel = lora_expand_kernel<Y, NB, LONG, 1, true, SWIGLU>;
  if (!a.whole)
    kernel = p.few ? lora_expand_kernel<Y, NB, 1, 1, false, SWIGLU> : lora_expand_kernel<Y, NB, LONG, 1, false, SWIGLU>;
  else if (p.few)
    kernel = a.cols % (4 * kCols) ? lora_expand_kernel<Y, NB, 1, 1, true, SWIGLU>
                                  : lora_expand_kernel<Y, NB, 1, SWIGLU && NB == 8 ? 2 : 4, true, SWIGLU>;
  kernel<<<grid, kThreads, 0, stream>>>(a);
}

template <typename Y, bool SWIGLU>
void expand_r(const LoraArgs& a, const LoraPlan& p, hipStream_t stream) {
  switch (a.r) {
    case 8: return expand<Y, 1, SWIGLU>(a, p, stream);
    case 16: return expand<Y, 2, SWIGLU>(a, p, stream);
    case 32: return expand<Y, 4, SWIGLU>(a, p, stream);
    default: return expand<Y, 8, SWIGLU>(a, p, stream);
  }
}

}  // namespace

hipError_t launch_lora(LoraArgs a, bool swiglu, hipStream_t stream) {
  const LoraPlan p = lora_plan(a.M, a.entries, a.C, a.n, a.r);
  a.splits = p.splits;
  a.chunk = p.chunk;
  // at most eight tiles of ranks in one launch: two matrices of rank 64
  const int most = a.r == 64 ? 2 : 4;
  for (a.first_target = 0; a.first_target < a.n; a.first_target += most) {
    const int n = a.n - a.first_target < most ? a.n - a.first_target : most;
    switch (a.r) {
      case 8:
      case 16: shrink_n<1>(a, n, p, stream); break;
      case 32: shrink_n<2>(a, n, p, stream); break;
      default: shrink_n<4>(a, n, p, stream); break;
    }
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // columns of a workgroup: as many as leave the compute units four workgroups
  int64_t all = 0;
  for (int k = 0; k < (swiglu ? 1 : a.n); ++k) all += a.target[k].R;
  int64_t cols = p.expand_slots * all / ((swiglu && !p.few ? 2 : 4) * (int64_t)device_cus());
  // short entries: four blocks a wave, or one
  const int unit = p.few && cols >= 3 * kCols ? 4 * kCols : kCols;
  a.cols = (int)(((cols < kCols ? kCols : cols > 4096 ? 4096 : cols) + unit - 1) / unit * unit);
  a.slots = (int)p.expand_slots;
  a.bare = swiglu;
  for (;; a.cols *= 2) {                                     // a grid holds fewer than 2^32 threads
    a.blocks = 0;
    for (int k = 0; k < (swiglu ? 1 : a.n); ++k) {
      a.target[k].blocks = (int)((a.target[k].R + a.cols - 1) / a.cols);
      a.blocks += a.target[k].blocks;
      if (!a.target[k].in_place) a.bare = true;
    }
    if (p.expand_slots * a.blocks < (1 << 23)) break;
  }
  if (swiglu)
    a.f32 ? expand_r<float, true>(a, p, stream) : expand_r<uint16_t, true>(a, p, stream);
  else
    a.f32 ? expand_r<float, false>(a, p, stream) : expand_r<uint16_t, false>(a, p, stream);
  return hipGetLastError();
}

}  // namespace trellis
