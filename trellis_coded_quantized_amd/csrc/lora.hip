// lora.hip -- low-rank adapters of many requests beside shared projections.
//
// Row m of entry e with adapter a:  t = A_a x_m,  y'_m = y_m + s_a B_a t.
// The first product reads x and A once and leaves f32 partial sums of its
// column chunks in the workspace; the second one adds them up, reads B and y
// and writes y'.  Two launches: every output needs the whole of t.
#include "internal.hpp"
#include "kv_common.hpp"
#include <type_traits>

namespace trellis {
namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr int kCols = 32 * kWaves;    // columns that a workgroup's waves take at a time

// Rows of one entry that a workgroup takes: one MFMA tile where entries are
// short, two (first product) and four (second product) where they are long.
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
// N matrices over one x, RT tiles of 16 ranks each, RM tiles of 16 rows, a
// chunk of columns a workgroup, whose four waves take them in turn.  Both
// operands contract along their rows in memory: a lane's 16 bytes are eight
// columns of one row, nothing goes through LDS.  The result has the row of x in
// the lane and four ranks in its registers.  The next step's loads are under
// way while this one's products run.
constexpr int shrink_registers(int nt, int rm, int steps) { return ((nt + rm) * steps * 2 + rm * nt) * 4; }

template <int N, int RT, int RM>
__global__ __launch_bounds__(kThreads, 2) void lora_shrink_kernel(LoraArgs a) {
  // steps of 32 columns whose loads go together, and two sets of them, as registers allow
  constexpr int NT = N * RT, STEPS = shrink_registers(NT, RM, 4) <= 216 ? 4 : shrink_registers(NT, RM, 2) <= 216 ? 2 : 1;
  constexpr int WIDE = 32 * STEPS;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.x / a.splits, split = blockIdx.x - slot * a.splits;
  const Tile t = find_tile(a, slot, RM * 16, false);
  if (!t.live) return;
  const uint16_t *x[RM], *w[NT];
#pragma unroll
  for (int m = 0; m < RM; ++m) x[m] = a.x + (int64_t)(t.first + min(m * 16 + col, t.rows - 1)) * a.x_stride + grp * 8;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    // ranks past the adapter's are read as its last: nothing reads their sums
    const int j = min(n % RT * 16 + col, t.rank - 1);
    w[n] = a.target[n / RT].a + ((int64_t)t.adapter * a.r + j) * a.C + grp * 8;
  }
  struct Step {
    u32x4v x[RM][STEPS], w[NT][STEPS];
  };
  // columns past `end` count as zeros
  auto load = [&](Step& to, int64_t c, int64_t end, bool check) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int64_t at = c + s * 32;
      const bool in = !check || at + grp * 8 < end;          // whole granules: C and chunks are multiples of 8
#pragma unroll
      for (int m = 0; m < RM; ++m) to.x[m][s] = in ? *reinterpret_cast<const u32x4v*>(x[m] + at) : u32x4v{};
#pragma unroll
      for (int n = 0; n < NT; ++n) to.w[n][s] = in ? *reinterpret_cast<const u32x4v*>(w[n] + at) : u32x4v{};
    }
  };
  f32x4v acc[RM][NT] = {};
  auto multiply = [&](const Step& v) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < RM; ++m) acc[m][n] = mfma16(v.w[n][s], v.x[m][s], acc[m][n]);
  };
  const int64_t c0 = (int64_t)split * a.chunk, c1 = min(a.C, c0 + a.chunk);
  int64_t c = c0 + wave * WIDE;
  if constexpr (shrink_registers(NT, RM, STEPS) <= 216) {
    Step p, q;
    if (c + WIDE <= c1) load(p, c, c1, false);
    while (c + WIDE <= c1) {
      if (c + 5 * WIDE <= c1) load(q, c + 4 * WIDE, c1, false);
      multiply(p);
      c += 4 * WIDE;
      if (c + WIDE > c1) break;
      if (c + 5 * WIDE <= c1) load(p, c + 4 * WIDE, c1, false);
      multiply(q);
      c += 4 * WIDE;
    }
  }
  for (; c < c1; c += 4 * WIDE) {
    Step p;
    load(p, c, c1, true);
    multiply(p);
  }
  // the waves' sums: a wave's share of the tiles each
  __shared__ f32x4v s_acc[kWaves][RM * NT > 8 ? 8 : RM * NT][64];
  constexpr int JOIN = RM * NT > 8 ? 8 : RM * NT;
#pragma unroll
  for (int k0 = 0; k0 < RM * NT; k0 += JOIN) {
    if (k0) __syncthreads();
#pragma unroll
    for (int k = 0; k < JOIN; ++k)
      if (k0 + k < RM * NT) s_acc[wave][k][lane] = acc[(k0 + k) / NT][(k0 + k) % NT];
    __syncthreads();
    for (int k = wave; k < JOIN && k0 + k < RM * NT; k += kWaves) {
      const f32x4v v = s_acc[0][k][lane] + s_acc[1][k][lane] + s_acc[2][k][lane] + s_acc[3][k][lane];
      const int m = (k0 + k) / NT * 16 + col, n = (k0 + k) % NT, j = n % RT * 16 + grp * 4;
      if (m < t.rows && j < a.r)
        *reinterpret_cast<f32x4v*>(a.part + ((int64_t)split * a.M + t.first + m) * (N * a.r) + n / RT * a.r + j) = v;
    }
  }
}

// ---- y + s B t -----------------------------------------------------------
// t enters as three bf16 numbers that add up to its 24 bits, so that the
// second product loses nothing against f32: the contraction is (part, rank),
// in units of eight ranks, four units a matrix instruction, and an operand of
// B serves all parts.  MFMA row 4 g + e of instruction q is output 8 g + 4 q +
// e, so two instructions leave eight neighbouring outputs of a row in a lane.
template <int NB>
struct Units {
  static constexpr int MFMAS = (3 * NB + 3) / 4, OPERANDS = NB < 4 ? 1 : NB / 4;
  static __device__ __forceinline__ int block(int q, int grp) { return NB < 4 ? grp % NB : q % OPERANDS * 4 + grp; }
  static __device__ __forceinline__ int part(int q, int grp) { return (4 * q + grp) / NB; }
};

__device__ __forceinline__ float silu_times(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// Eight outputs of a row as they lie in memory: loaded ahead where rows are 16-byte aligned.
template <typename Y>
struct Eight {
  u32x4v w[sizeof(Y) / 2];
  __device__ __forceinline__ void load(const Y* p) {
#pragma unroll
    for (int k = 0; k < (int)sizeof(Y) / 2; ++k) w[k] = *reinterpret_cast<const u32x4v*>(p + k * 4);
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(Y) == 4) return __builtin_bit_cast(float, (uint32_t)w[e >> 2][e & 3]);
    else return Bf16::to_f32((uint16_t)(w[0][e >> 1] >> (16 * (e & 1))));
  }
};

__device__ __forceinline__ float get_one(const float* p) { return *p; }
__device__ __forceinline__ float get_one(const uint16_t* p) { return Bf16::to_f32(*p); }
__device__ __forceinline__ void put_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void put_one(uint16_t* p, float v) { *p = (uint16_t)Bf16::pack(v, 0.0f); }
__device__ __forceinline__ void put_eight(float* p, const float (&v)[8]) {
  *reinterpret_cast<f32x4v*>(p) = f32x4v{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4v*>(p + 4) = f32x4v{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void put_eight(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<u32x4v*>(p) =
      u32x4v{Bf16::pack(v[0], v[1]), Bf16::pack(v[2], v[3]), Bf16::pack(v[4], v[5]), Bf16::pack(v[6], v[7])};
}

// MT tiles of 16 rows, SUB blocks of 32 columns a wave at a time: their rows of
// B and of y are asked for together, the first ones before t is put together.
// SWIGLU: targets 0 and 1 are gate and up, outputs go to target 0's out.
template <typename Y, int NB, int MT, int SUB, bool SWIGLU>
__global__ __launch_bounds__(kThreads, 2) void lora_expand_kernel(LoraArgs a) {
  typedef Units<NB> U;
  typedef typename std::conditional<SWIGLU, uint16_t, Y>::type Out;
  constexpr int R = NB * 8, ROWS = MT * 16, G = SWIGLU ? 2 : 1, PAD = 8;      // PAD: rows of t on different LDS banks
  __shared__ __align__(16) uint16_t s_t[G][3][ROWS][R + PAD];
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int k = 0, block = blockIdx.x % a.blocks;                  // target and its column block
  const int slot = blockIdx.x / a.blocks;
  if (!SWIGLU)
    while (block >= a.target[k].blocks) block -= a.target[k++].blocks;
  const Tile t = find_tile(a, slot, ROWS, a.bare);
  if (!t.live) return;
  const LoraTarget* const target = a.target + k;
  const bool on = t.adapter >= 0;
  if (!on && !SWIGLU && target->in_place) return;
  const int64_t out_n = target->R, end = min(out_n, (int64_t)(block + 1) * a.cols);

  u32x4v keep[U::OPERANDS];                                  // bits of the ranks that the adapter has
#pragma unroll
  for (int q = 0; q < U::OPERANDS; ++q) {
    const int have = t.rank - U::block(q, grp) * 8;
#pragma unroll
    for (int w = 0; w < 4; ++w) keep[q][w] = (have > 2 * w ? 0xFFFFu : 0u) | (have > 2 * w + 1 ? 0xFFFF0000u : 0u);
  }
  u32x4v b[G][SUB][U::OPERANDS][2];
  Eight<Y> y[G][SUB][MT];
  auto load = [&](int64_t c) __attribute__((always_inline)) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        const int64_t i0 = c + u * 32 * kWaves;
        if (on) {
#pragma unroll
          for (int q = 0; q < U::OPERANDS; ++q)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              // what B holds past the adapter's rank is cut below; the address stays inside the matrix
              const int64_t i = min(i0 + (col >> 2) * 8 + z * 4 + (col & 3), out_n - 1);
              b[g][u][q][z] = *reinterpret_cast<const u32x4v*>(target[g].b + ((int64_t)t.adapter * out_n + i) * R +
                                                               U::block(q, grp) * 8);
            }
        }
        if (a.aligned) {
          const int64_t i = min(i0 + grp * 8, (out_n - 8) & ~(int64_t)7);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            if (i >= 0)
              y[g][u][m].load(reinterpret_cast<const Y*>(target[g].y) +
                              (int64_t)(t.first + min(m * 16 + col, t.rows - 1)) * target[g].y_stride + i);
        }
      }
  };
  int64_t c = (int64_t)block * a.cols + wave * 32;
  load(c);

  if (on) {
    // the column chunks' sums, four ranks at a time: short entries may have many
    // chunks, and 16 lanes share them; long ones have few
    constexpr int SHARE = MT == 1 ? 16 : 1, ITEMS = G * ROWS * R / 4;
    const float scale = a.scales[t.adapter];
    const int lead = tid % SHARE;
    for (int x = tid / SHARE; x < ITEMS; x += kThreads / SHARE) {
      const int g = x / (ROWS * R / 4), m = x / (R / 4) % ROWS, j = x % (R / 4) * 4;
      if (MT == 1 && m >= t.rows) continue;                  // those columns of the product are not looked at
      f32x4v v = {};
      if (m < t.rows) {
        const float* part = a.part + (int64_t)(t.first + m) * (a.n * R) + (k + g) * R + j;
        const int64_t step = a.M * (a.n * R);
#pragma unroll 4
        for (int s = lead; s < a.splits; s += SHARE) v += *reinterpret_cast<const f32x4v*>(part + s * step);
      }
#pragma unroll
      for (int d = SHARE / 2; d; d >>= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += __shfl_xor(v[e], d);
      if (lead) continue;
      float hi[4], mid[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = j + e < t.rank ? v[e] * scale : 0.0f;
        hi[e] = Bf16::to_f32((uint16_t)Bf16::pack(f, 0.0f));
        const float rest = fabsf(f - hi[e]) < INFINITY ? f - hi[e] : 0.0f;   // an infinity or NaN stands in the first part alone
        mid[e] = Bf16::to_f32((uint16_t)Bf16::pack(rest, 0.0f));
        lo[e] = rest - mid[e];
      }
      *reinterpret_cast<u32x2v*>(&s_t[g][0][m][j]) = u32x2v{Bf16::pack(hi[0], hi[1]), Bf16::pack(hi[2], hi[3])};
      *reinterpret_cast<u32x2v*>(&s_t[g][1][m][j]) = u32x2v{Bf16::pack(mid[0], mid[1]), Bf16::pack(mid[2], mid[3])};
      *reinterpret_cast<u32x2v*>(&s_t[g][2][m][j]) = u32x2v{Bf16::pack(lo[0], lo[1]), Bf16::pack(lo[2], lo[3])};
    }
  }
  __syncthreads();

  while (c < end) {
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      const int64_t i0 = c + u * 32 * kWaves;
      if (i0 >= end) continue;
      f32x4v acc[G][MT][2] = {};
      if (on) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int q = 0; q < U::MFMAS; ++q) {
            const int part = U::part(q, grp), o = q % U::OPERANDS;
            const u32x4v lhs[2] = {b[g][u][o][0] & keep[o], b[g][u][o][1] & keep[o]};
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              u32x4v v = *reinterpret_cast<const u32x4v*>(&s_t[g][part < 3 ? part : 0][m * 16 + col][U::block(q, grp) * 8]);
              if (part == 3) v = u32x4v{};                   // the fourth quarter of a unit that three parts fill
#pragma unroll
              for (int z = 0; z < 2; ++z) acc[g][m][z] = mfma16(lhs[z], v, acc[g][m][z]);
            }
          }
      }
      const int64_t i = i0 + grp * 8;
      const int in = (int)min((int64_t)8, out_n - i);
      if (in <= 0) continue;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int64_t row = t.first + m * 16 + col;
        if (m * 16 + col >= t.rows) continue;
        Out* out = reinterpret_cast<Out*>(target->out) + row * target->out_stride + i;
        float v[8];
        if (a.aligned && in == 8) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[e] = y[0][u][m].get(e) + acc[0][m][e >> 2][e & 3];
            if constexpr (SWIGLU) v[e] = silu_times(v[e], y[1][u][m].get(e) + acc[1][m][e >> 2][e & 3]);
          }
          put_eight(out, v);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (e >= in) continue;
            v[e] = get_one(reinterpret_cast<const Y*>(target->y) + row * target->y_stride + i + e) + acc[0][m][e >> 2][e & 3];
            if constexpr (SWIGLU)
              v[e] = silu_times(v[e], get_one(reinterpret_cast<const Y*>(target[1].y) + row * target[1].y_stride + i + e) +
                                          acc[1][m][e >> 2][e & 3]);
            put_one(out + e, v[e]);
          }
        }
      }
    }
    c += SUB * 32 * kWaves;
    if (c < end) load(c);
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
  p.few = M <= (int64_t)kShort * entries;
  p.shrink_slots = slots_of(M, entries, p.few ? kShort : kLongShrink);
  p.expand_slots = slots_of(M, entries, p.few ? kShort : kLongExpand);
  // column chunks until the compute units have two workgroups, none shorter
  // than two steps of every wave.  Long entries: at most four, which every
  // workgroup of the second product adds up again.
  const int64_t want = 2 * (int64_t)device_cus() / (p.shrink_slots ? p.shrink_slots : 1), most = p.few ? 32 : 4;
  int64_t splits = (C + 255) / 256;
  if (splits > want) splits = want;
  if (splits > most) splits = most;
  if (splits < 1) splits = 1;
  p.chunk = ((C + splits - 1) / splits + 63) / 64 * 64;
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
void shrink_n(const LoraArgs& a, const LoraPlan& p, hipStream_t stream) {
  switch (a.n) {
    case 1: return shrink<1, RT>(a, p, stream);
    case 2: return shrink<2, RT>(a, p, stream);
    case 3: return shrink<3, RT>(a, p, stream);
    default: return shrink<4, RT>(a, p, stream);
  }
}

template <typename Y, int NB, bool SWIGLU>
void expand(const LoraArgs& a, const LoraPlan& p, hipStream_t stream) {
  const unsigned grid = (unsigned)(p.expand_slots * a.blocks);
  if (!p.few)
    lora_expand_kernel<Y, NB, kLongExpand / 16, 1, SWIGLU><<<grid, kThreads, 0, stream>>>(a);
  else if (a.cols == kCols)
    lora_expand_kernel<Y, NB, kShort / 16, 1, SWIGLU><<<grid, kThreads, 0, stream>>>(a);
  else
    lora_expand_kernel<Y, NB, kShort / 16, 4, SWIGLU><<<grid, kThreads, 0, stream>>>(a);
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
  switch (a.r) {
    case 8:
    case 16: shrink_n<1>(a, p, stream); break;
    case 32: shrink_n<2>(a, p, stream); break;
    default: shrink_n<4>(a, p, stream); break;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // columns of a workgroup: as many as leave the compute units four workgroups
  int64_t all = 0;
  for (int k = 0; k < (swiglu ? 1 : a.n); ++k) all += a.target[k].R;
  int64_t cols = p.expand_slots * all / (4 * (int64_t)device_cus());
  a.cols = (int)((cols < kCols ? kCols : cols > 4096 ? 4096 : cols) + kCols - 1) / kCols * kCols;
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
