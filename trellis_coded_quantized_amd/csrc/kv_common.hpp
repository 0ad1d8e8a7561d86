// kv_common.hpp -- what the attention and cache kernels share: the element
// types, the paged key/value cache with its addressing, and wave-wide sums.
//
// The cache stores both operands of the attention in the order in which the
// matrix units take them.  An MFMA operand lane holds eight consecutive
// elements of the contraction (16 bytes).  Keys contract over the head
// dimension, values over the tokens, so a 16-byte granule holds
//   keys    8 dimensions of one token:  [page, head, D/8, P, 8]
//   values  8 tokens of one dimension:  [page, head, P/8, D, 8]
// and neighbouring granules belong to neighbouring tokens (keys) or
// dimensions (values), which are neighbouring lanes: every operand load is a
// contiguous 16 bytes a lane, and nothing is transposed when it is read.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace trellis {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef float f32x2p __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Element types: conversions (nearest even), the 32x32x16 MFMA, and the bits
// that tell infinities and NaN (an exponent of all ones).
struct Bf16 {
  static constexpr uint32_t kExp = 0x7F80u, kOne = 0x3F80u;
  static __device__ __forceinline__ float to_f32(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2p{a, b}, bf16x2));
  }
  static __device__ __forceinline__ f32x16 mfma(u32x4v a, u32x4v b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
  }
};

struct F16 {
  static constexpr uint32_t kExp = 0x7C00u, kOne = 0x3C00u;
  static __device__ __forceinline__ float to_f32(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2p{a, b}, f16x2));
  }
  static __device__ __forceinline__ f32x16 mfma(u32x4v a, u32x4v b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  }
};

// A page number from a table, kept inside the pool: entries that hold no
// page (-1) or a wrong one are read as page 0.  What is read there is another
// sequence's: readers cut it by page_ok, writers leave such slots alone.
__device__ __forceinline__ uint32_t page_in_pool(int32_t page, uint32_t pages) {
  return (uint32_t)page < pages ? (uint32_t)page : 0u;
}
__device__ __forceinline__ bool page_ok(int32_t page, uint32_t pages) { return (uint32_t)page < pages; }

// Inclusive sum over the 64 lanes of a wave.
__device__ __forceinline__ int wave_scan_add(int v) {
  const int lane = (int)__lane_id();
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

}  // namespace trellis
