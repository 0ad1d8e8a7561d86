// lora.hip -- low-rank adapters of many requests beside shared projections.
//
// Row m of entry e with adapter a:  t = A_a x_m,  y'_m = y_m + s_a B_a t.
// The first product reads x and A once and leaves f32 partial sums of its
// column chunks in the workspace; the second one adds them up, reads B and y
// and writes y'.  Two launches: every output needs the whole of t.
#include "internal.hpp"
#include "kv_common.hpp"

namespace trellis {
namespace {

constexpr int kThreads = 256, kWaves = 4;

// Rows of one entry that a workgroup takes: one MFMA tile where entries are
// short (its waves then share the columns), four where they are long.
constexpr int kFewRows = 16, kManyRows = 64;

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
// N matrices over one x, RT tiles of 16 ranks each, a chunk of columns a
// workgroup.  Both operands contract along their rows in memory: a lane's 16
// bytes are eight columns of one row, nothing goes through LDS.  The result has
// the row of x in the lane and four ranks in its registers.
template <int N, int RT, bool FEW>
__global__ __launch_bounds__(kThreads) void lora_shrink_kernel(LoraArgs a) {
  constexpr int NT = N * RT, STEPS = NT <= 2 ? 4 : NT <= 8 ? 2 : 1, JOIN = NT < 8 ? NT : 8;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.x / a.splits, split = blockIdx.x - slot * a.splits;
  const Tile t = find_tile(a, slot, FEW ? kFewRows : kManyRows, false);
  if (!t.live) return;
  const int r0 = FEW ? 0 : wave * 16;
  if (!FEW && r0 >= t.rows) return;
  const int64_t row = t.first + min(r0 + col, t.rows - 1);
  const uint16_t* x = a.x + row * a.x_stride + grp * 8;
  const uint16_t* w[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    // ranks past the adapter's are read as its last: nothing reads their sums
    const int j = min(n % RT * 16 + col, t.rank - 1);
    w[n] = a.target[n / RT].a + ((int64_t)t.adapter * a.r + j) * a.C + grp * 8;
  }
  f32x4v acc[NT] = {};
  const int64_t c0 = (int64_t)split * a.chunk, c1 = min(a.C, c0 + a.chunk);
  for (int64_t c = c0 + (FEW ? wave * 32 * STEPS : 0); c < c1; c += 32 * STEPS * (FEW ? kWaves : 1)) {
    u32x4v xv[STEPS], wv[NT][STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int64_t at = c + s * 32;
      const bool in = at + grp * 8 < c1;                     // whole granules: C and chunks are multiples of 8
      xv[s] = in ? *reinterpret_cast<const u32x4v*>(x + at) : u32x4v{};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        wv[n][s] = u32x4v{};
        if (n % RT * 16 < t.rank && in) wv[n][s] = *reinterpret_cast<const u32x4v*>(w[n] + at);
      }
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[n] = mfma16(wv[n][s], xv[s], acc[n]);
  }
  float* part = a.part + ((int64_t)split * a.M + t.first + r0 + col) * (N * a.r);
  auto put = [&](int n, f32x4v v) {
    const int j = n % RT * 16 + grp * 4;
    if (r0 + col < t.rows && j < a.r) *reinterpret_cast<f32x4v*>(part + n / RT * a.r + j) = v;
  };
  if constexpr (FEW) {
    __shared__ f32x4v s_acc[kWaves - 1][JOIN][64];
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += JOIN) {
      if (n0) __syncthreads();
      if (wave)
#pragma unroll
        for (int n = 0; n < JOIN; ++n)
          if (n0 + n < NT) s_acc[wave - 1][n][lane] = acc[n0 + n];
      __syncthreads();
      if (wave == 0)
#pragma unroll
        for (int n = 0; n < JOIN; ++n)
          if (n0 + n < NT) put(n0 + n, acc[n0 + n] + s_acc[0][n][lane] + s_acc[1][n][lane] + s_acc[2][n][lane]);
    }
  } else {
#pragma unroll
    for (int n = 0; n < NT; ++n) put(n, acc[n]);
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

// eight outputs of a row: from v, or into it; in == how many there are
template <typename Y>
__device__ __forceinline__ void load8(const Y* p, bool whole, int in, float (&v)[8]) {
  if (whole) {
    if constexpr (sizeof(Y) == 4) {
      const f32x4v lo = *reinterpret_cast<const f32x4v*>(p), hi = *reinterpret_cast<const f32x4v*>(p + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = lo[e], v[4 + e] = hi[e];
    } else {
      const u32x4v w = *reinterpret_cast<const u32x4v*>(p);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = Bf16::to_f32((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = 0.0f;
      if (e < in) {
        if constexpr (sizeof(Y) == 4) v[e] = p[e];
        else v[e] = Bf16::to_f32(p[e]);
      }
    }
  }
}

template <typename Y>
__device__ __forceinline__ void store8(Y* p, bool whole, int in, const float (&v)[8]) {
  if (whole) {
    if constexpr (sizeof(Y) == 4) {
      *reinterpret_cast<f32x4v*>(p) = f32x4v{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4v*>(p + 4) = f32x4v{v[4], v[5], v[6], v[7]};
    } else {
      *reinterpret_cast<u32x4v*>(p) = u32x4v{Bf16::pack(v[0], v[1]), Bf16::pack(v[2], v[3]), Bf16::pack(v[4], v[5]),
                                             Bf16::pack(v[6], v[7])};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < in) {
        if constexpr (sizeof(Y) == 4) p[e] = v[e];
        else p[e] = (uint16_t)Bf16::pack(v[e], 0.0f);
      }
  }
}

// MT tiles of 16 rows.  SWIGLU: targets 0 and 1 are gate and up, outputs go to
// target 0's out.
template <typename Y, int NB, int MT, bool SWIGLU>
__global__ __launch_bounds__(kThreads) void lora_expand_kernel(LoraArgs a) {
  typedef Units<NB> U;
  constexpr int R = NB * 8, ROWS = MT * 16, G = SWIGLU ? 2 : 1;
  __shared__ __align__(16) uint16_t s_t[G][3][ROWS][R];
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int k = 0, block = blockIdx.x % a.blocks;                  // target and its column block
  const int slot = blockIdx.x / a.blocks;
  if (!SWIGLU)
    while (block >= a.target[k].blocks) block -= a.target[k++].blocks;
  const Tile t = find_tile(a, slot, MT == 1 ? kFewRows : kManyRows, a.bare);
  if (!t.live) return;
  const LoraTarget* const target = a.target + k;
  const bool on = t.adapter >= 0;
  if (!on && !SWIGLU && target->in_place) return;
  if (on) {
    const float scale = a.scales[t.adapter];
    for (int x = tid; x < G * ROWS * R; x += kThreads) {
      const int g = x / (ROWS * R), m = x / R % ROWS, j = x % R;
      float v = 0.0f;
      if (m < t.rows && j < t.rank) {
        const float* part = a.part + (int64_t)(t.first + m) * (a.n * R) + (k + g) * R + j;
        for (int s = 0; s < a.splits; ++s) v += part[(int64_t)s * a.M * (a.n * R)];
        v *= scale;
      }
      const uint32_t hi = Bf16::pack(v, 0.0f);
      const float rest = v - Bf16::to_f32((uint16_t)hi);
      const bool fine = fabsf(rest) < INFINITY;              // an infinity or NaN stands in the first part alone
      const uint32_t mid = fine ? Bf16::pack(rest, 0.0f) : 0u;
      s_t[g][0][m][j] = (uint16_t)hi;
      s_t[g][1][m][j] = (uint16_t)mid;
      s_t[g][2][m][j] = (uint16_t)(fine ? Bf16::pack(rest - Bf16::to_f32((uint16_t)mid), 0.0f) : 0u);
    }
  }
  __syncthreads();
  u32x4v keep[U::OPERANDS];                                  // bits of the ranks that the adapter has
#pragma unroll
  for (int q = 0; q < U::OPERANDS; ++q) {
    const int have = t.rank - U::block(q, grp) * 8;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      keep[q][w] = (have > 2 * w ? 0xFFFFu : 0u) | (have > 2 * w + 1 ? 0xFFFF0000u : 0u);
  }
  const int64_t out_n = target->R, end = min(out_n, (int64_t)(block + 1) * a.cols);
  for (int64_t i0 = (int64_t)block * a.cols + wave * 32; i0 < end; i0 += 32 * kWaves) {
    f32x4v acc[G][MT][2] = {};
    if (on) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        u32x4v b[U::OPERANDS][2];
#pragma unroll
        for (int q = 0; q < U::OPERANDS; ++q)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int64_t i = min(i0 + (col >> 2) * 8 + y * 4 + (col & 3), out_n - 1);
            b[q][y] = u32x4v{};
            if (keep[q][0])
              b[q][y] = *reinterpret_cast<const u32x4v*>(target[g].b + ((int64_t)t.adapter * out_n + i) * R +
                                                         U::block(q, grp) * 8) & keep[q];
          }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if (MT > 1 && m * 16 >= t.rows) break;
#pragma unroll
          for (int q = 0; q < U::MFMAS; ++q) {
            const int part = U::part(q, grp);
            u32x4v v = {};
            if (part < 3) v = *reinterpret_cast<const u32x4v*>(&s_t[g][part][m * 16 + col][U::block(q, grp) * 8]);
#pragma unroll
            for (int y = 0; y < 2; ++y) acc[g][m][y] = mfma16(b[q % U::OPERANDS][y], v, acc[g][m][y]);
          }
        }
      }
    }
    const int64_t i = i0 + grp * 8;
    const int in = (int)min((int64_t)8, out_n - i);
    const bool whole = a.aligned && in == 8;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t row = t.first + m * 16 + col;
      if (m * 16 + col >= t.rows || in <= 0) continue;
      float v[8];
      load8(reinterpret_cast<const Y*>(target->y) + row * target->y_stride + i, whole, in, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += acc[0][m][e >> 2][e & 3];
      if constexpr (SWIGLU) {
        float u[8];
        load8(reinterpret_cast<const Y*>(target[1].y) + row * target[1].y_stride + i, whole, in, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = silu_times(v[e], u[e] + acc[1][m][e >> 2][e & 3]);
        store8(reinterpret_cast<uint16_t*>(target->out) + row * target->out_stride + i, whole, in, v);
      } else {
        store8(reinterpret_cast<Y*>(target->out) + row * target->out_stride + i, whole, in, v);
      }
    }
  }
}

// ---- launch --------------------------------------------------------------
// Short entries: 16 rows a tile; else 64 (32 at rank 128, whose parts of t
// would not fit).
bool few_rows(int64_t M, int entries) { return M <= (int64_t)kFewRows * entries; }

int64_t slots_of(int64_t M, int entries, int rows) {
  const int64_t most = (M + rows - 1) / rows + entries;      // every entry's last tile may be a short one
  return M < most ? M : most;
}

}  // namespace

LoraPlan lora_plan(int64_t M, int entries, int64_t C, int n, int r) {
  LoraPlan p;
  p.few = few_rows(M, entries);
  p.rows = p.few ? kFewRows : kManyRows;
  p.slots = slots_of(M, entries, p.rows);
  // column chunks until the compute units have two workgroups, none shorter
  // than two steps of every wave
  const int64_t least = p.few ? 256 : 128, want = 2 * (int64_t)device_cus() / (p.slots ? p.slots : 1);
  int64_t splits = (C + least - 1) / least;
  if (splits > want) splits = want;
  if (splits > 32) splits = 32;
  if (splits < 1) splits = 1;
  p.chunk = ((C + splits - 1) / splits + 63) / 64 * 64;
  p.splits = (int)((C + p.chunk - 1) / p.chunk);
  p.bytes = ((size_t)p.splits * (size_t)M * n * r * 4 + 255) / 256 * 256;
  return p;
}

namespace {

template <int N, int RT>
void shrink(const LoraArgs& a, const LoraPlan& p, hipStream_t stream) {
  const unsigned grid = (unsigned)(p.slots * p.splits);
  if (p.few)
    lora_shrink_kernel<N, RT, true><<<grid, kThreads, 0, stream>>>(a);
  else
    lora_shrink_kernel<N, RT, false><<<grid, kThreads, 0, stream>>>(a);
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
  const unsigned grid = (unsigned)(p.slots * a.blocks);
  if (p.few)
    lora_expand_kernel<Y, NB, 1, SWIGLU><<<grid, kThreads, 0, stream>>>(a);
  else
    lora_expand_kernel<Y, NB, 4, SWIGLU><<<grid, kThreads, 0, stream>>>(a);
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
  int64_t cols = p.slots * all / (4 * (int64_t)device_cus());
  a.cols = (int)((cols < 128 ? 128 : cols > 4096 ? 4096 : cols) + 127) / 128 * 128;
  a.bare = swiglu;
  for (;; a.cols *= 2) {                                     // a grid holds fewer than 2^32 threads
    a.blocks = 0;
    for (int k = 0; k < (swiglu ? 1 : a.n); ++k) {
      a.target[k].blocks = (int)((a.target[k].R + a.cols - 1) / a.cols);
      a.blocks += a.target[k].blocks;
      if (!a.target[k].in_place) a.bare = true;
    }
    if (p.slots * a.blocks < (1 << 23)) break;
  }
  if (swiglu)
    a.f32 ? expand_r<float, true>(a, p, stream) : expand_r<uint16_t, true>(a, p, stream);
  else
    a.f32 ? expand_r<float, false>(a, p, stream) : expand_r<uint16_t, false>(a, p, stream);
  return hipGetLastError();
}

}  // namespace trellis
