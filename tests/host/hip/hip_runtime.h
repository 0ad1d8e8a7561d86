// What the library's headers take from HIP, for the CPU: device code one lane
// at a time (only code that exchanges nothing between lanes is run this way),
// and the host calls that a test stands in for.
#pragma once
#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <algorithm>

#define __device__
#define __forceinline__ inline
using std::max;
using std::min;
typedef int hipError_t;
typedef void* hipStream_t;
constexpr hipError_t hipSuccess = 0, hipErrorInvalidDevice = 101;
constexpr int hipFuncAttributeMaxDynamicSharedMemorySize = 8;
hipError_t hipGetDevice(int*);
hipError_t hipFuncSetAttribute(const void*, int, int);

extern unsigned host_lane;
inline unsigned __lane_id() { return host_lane; }
template <typename V> V __shfl_xor(V, int);
template <typename V> V __shfl_up(V, int);
template <typename V> int __any(V);
struct HostPair {
  uint32_t operator[](int) const;
};
HostPair host_swap(uint32_t, uint32_t);
#define __builtin_amdgcn_readfirstlane(x) (x)
#define __builtin_amdgcn_permlane32_swap(a, b, c, d) host_swap(a, b)
#define __builtin_amdgcn_exp2f(x) exp2f(x)
#define __builtin_amdgcn_sched_barrier(x)
#define __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, d, e, f) (c)
#define __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, d, e, f) (c)
