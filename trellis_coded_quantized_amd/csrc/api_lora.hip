// api_lora.hip -- the C ABI of the low-rank adapters (include/trellis.h):
// host-side validation and dispatch.  Nothing is launched or written unless
// every check passes.
#include "trellis.h"
#include "internal.hpp"

namespace {

using trellis::api_fail;

#define TRY(expr)                      \
  do {                                 \
    int _rc = (expr);                  \
    if (_rc != TRELLIS_OK) return _rc; \
  } while (0)

constexpr int64_t kMaxIndex = (int64_t)1 << 31;
static_assert(TRELLIS_LORA_MAX == sizeof(trellis::LoraArgs::target) / sizeof(trellis::LoraTarget), "targets of a call");

int need_ptr(const char* fn, const char* name, const void* p, size_t align) {
  if (!p) return api_fail(TRELLIS_EINVAL, "%s: %s is NULL", fn, name);
  if (reinterpret_cast<uintptr_t>(p) % align != 0)
    return api_fail(TRELLIS_EINVAL, "%s: %s not %zu-byte aligned", fn, name, align);
  return TRELLIS_OK;
}

int check_sizes(const char* fn, int64_t M, int64_t C, int n, int n_targets, int rank) {
  if (n_targets < 1 || n_targets > TRELLIS_LORA_MAX)
    return api_fail(TRELLIS_EINVAL, "%s: n_targets=%d outside 1..%d", fn, n_targets, TRELLIS_LORA_MAX);
  if (rank != 8 && rank != 16 && rank != 32 && rank != 64)
    return api_fail(TRELLIS_EUNSUPPORTED, "%s: rank=%d not in {8, 16, 32, 64}", fn, rank);
  if (C < 1 || C >= kMaxIndex) return api_fail(TRELLIS_EINVAL, "%s: C=%lld outside 1..2^31-1", fn, (long long)C);
  if (C % 8 != 0) return api_fail(TRELLIS_EUNSUPPORTED, "%s: C=%lld not a multiple of 8", fn, (long long)C);
  if (n < 1 || n > 65535) return api_fail(TRELLIS_EINVAL, "%s: n=%d entries outside 1..65535", fn, n);
  if (M < 0 || M > TRELLIS_LORA_MAX_ROWS)
    return api_fail(TRELLIS_EINVAL, "%s: M=%lld outside 0..%d", fn, (long long)M, TRELLIS_LORA_MAX_ROWS);
  return TRELLIS_OK;
}

int check_matrix(const char* fn, const trellis_lora_target& t, int y_dtype) {
  const size_t size = y_dtype == TRELLIS_OUT_F32 ? 4 : 2;
  if (t.R < 1 || t.R > TRELLIS_LORA_MAX_OUTPUTS)
    return api_fail(TRELLIS_EINVAL, "%s: R=%lld outside 1..%d", fn, (long long)t.R, TRELLIS_LORA_MAX_OUTPUTS);
  if (t.y_stride < t.R) return api_fail(TRELLIS_EINVAL, "%s: y_stride=%lld below R", fn, (long long)t.y_stride);
  TRY(need_ptr(fn, "a", t.a, 16));
  TRY(need_ptr(fn, "b", t.b, 16));
  return need_ptr(fn, "y", t.y, size);
}

// whether rows of R elements can be read and written 16 bytes at a time
bool aligned_rows(const void* p, int64_t stride, size_t size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * (int64_t)size % 16 == 0;
}

int run(const char* fn, bool swiglu, const uint16_t* x, int64_t x_stride, const trellis_lora_target* targets,
        int n_targets, int y_dtype, const int32_t* starts, const int32_t* adapters, int n, const float* scales,
        const int32_t* ranks, int64_t pool, int rank, int64_t M, int64_t C, void* workspace, size_t workspace_bytes,
        void* stream) {
  TRY(check_sizes(fn, M, C, n, n_targets, rank));
  if (y_dtype != TRELLIS_OUT_BF16 && y_dtype != TRELLIS_OUT_F32)
    return api_fail(TRELLIS_EINVAL, "%s: y_dtype=%d unknown", fn, y_dtype);
  if (pool < 1 || pool >= kMaxIndex)
    return api_fail(TRELLIS_EINVAL, "%s: pool=%lld adapters outside 1..2^31-1", fn, (long long)pool);
  if (x_stride < C || x_stride % 8 != 0)
    return api_fail(TRELLIS_EINVAL, "%s: x_stride=%lld not a multiple of 8 of at least %lld", fn, (long long)x_stride,
                    (long long)C);
  if (M == 0) return trellis::api_ok();
  const size_t size = y_dtype == TRELLIS_OUT_F32 ? 4 : 2, out_size = swiglu ? 2 : size;
  trellis::LoraArgs a{};
  a.whole = 1;
  for (int k = 0; k < n_targets; ++k) {
    const trellis_lora_target& t = targets[k];
    TRY(check_matrix(fn, t, y_dtype));
    a.target[k] = trellis::LoraTarget{t.a, t.b, t.y, t.out, t.R, t.y_stride, t.out_stride, 0, 0};
    a.whole &= t.R % 8 == 0 && aligned_rows(t.y, t.y_stride, size);
    if (swiglu && k) continue;                               // target 0's out is the call's
    TRY(need_ptr(fn, "out", t.out, out_size));
    if (t.out_stride < t.R) return api_fail(TRELLIS_EINVAL, "%s: out_stride=%lld below R", fn, (long long)t.out_stride);
    if (!swiglu && t.out == t.y && t.out_stride != t.y_stride)
      return api_fail(TRELLIS_EINVAL, "%s: out is y with another stride", fn);
    a.target[k].in_place = !swiglu && t.out == t.y;
    a.whole &= aligned_rows(t.out, t.out_stride, out_size);
  }
  TRY(need_ptr(fn, "x", x, 16));
  TRY(need_ptr(fn, "starts", starts, 4));
  TRY(need_ptr(fn, "adapters", adapters, 4));
  TRY(need_ptr(fn, "scales", scales, 4));
  if (ranks) TRY(need_ptr(fn, "ranks", ranks, 4));
  const size_t need = trellis::lora_plan(M, n, C, n_targets, rank).bytes;
  if (workspace_bytes < need)
    return api_fail(TRELLIS_EWORKSPACE, "%s: workspace %zu bytes < required %zu", fn, workspace_bytes, need);
  TRY(need_ptr(fn, "workspace", workspace, 256));
  a.x = x;
  a.starts = starts;
  a.adapters = adapters;
  a.ranks = ranks;
  a.scales = scales;
  a.part = reinterpret_cast<float*>(workspace);
  a.x_stride = x_stride;
  a.M = M;
  a.C = C;
  a.n = n_targets;
  a.r = rank;
  a.entries = n;
  a.pool = (int)pool;
  a.f32 = y_dtype == TRELLIS_OUT_F32;
  return trellis::api_hip(fn, trellis::launch_lora(a, swiglu, (hipStream_t)stream));
}

}  // namespace

extern "C" {

size_t trellis_lora_workspace_bytes(int64_t M, int64_t C, int n, int n_targets, int rank) {
  if (check_sizes("trellis_lora_workspace_bytes", M, C, n, n_targets, rank) != TRELLIS_OK || M == 0) return 0;
  return trellis::lora_plan(M, n, C, n_targets, rank).bytes;
}

int trellis_lora_add(const uint16_t* x, int64_t x_stride, const trellis_lora_target* targets, int n_targets,
                     int y_dtype, const int32_t* starts, const int32_t* adapters, int n, const float* scales,
                     const int32_t* ranks, int64_t pool, int rank, int64_t M, int64_t C, void* workspace,
                     size_t workspace_bytes, void* stream) {
  const char* fn = "trellis_lora_add";
  if (!targets) return api_fail(TRELLIS_EINVAL, "%s: targets is NULL", fn);
  return run(fn, false, x, x_stride, targets, n_targets, y_dtype, starts, adapters, n, scales, ranks, pool, rank, M, C,
             workspace, workspace_bytes, stream);
}

int trellis_lora_swiglu(const uint16_t* x, int64_t x_stride, const trellis_lora_target* gate,
                        const trellis_lora_target* up, uint16_t* out, int64_t out_stride, int y_dtype,
                        const int32_t* starts, const int32_t* adapters, int n, const float* scales,
                        const int32_t* ranks, int64_t pool, int rank, int64_t M, int64_t C, void* workspace,
                        size_t workspace_bytes, void* stream) {
  const char* fn = "trellis_lora_swiglu";
  if (!gate || !up) return api_fail(TRELLIS_EINVAL, "%s: %s is NULL", fn, gate ? "up" : "gate");
  if (gate->R != up->R)
    return api_fail(TRELLIS_EINVAL, "%s: gate has %lld outputs, up %lld", fn, (long long)gate->R, (long long)up->R);
  trellis_lora_target both[2] = {*gate, *up};
  both[0].out = out;
  both[0].out_stride = out_stride;
  for (int k = 0; k < 2 && y_dtype == TRELLIS_OUT_BF16; ++k)
    if (both[k].y == out && both[k].y_stride != out_stride)
      return api_fail(TRELLIS_EINVAL, "%s: out is %s with another stride", fn, k ? "up" : "gate");
  if (y_dtype == TRELLIS_OUT_F32 && (gate->y == out || up->y == out))
    return api_fail(TRELLIS_EINVAL, "%s: out is an f32 input", fn);
  return run(fn, true, x, x_stride, both, 2, y_dtype, starts, adapters, n, scales, ranks, pool, rank, M, C, workspace,
             workspace_bytes, stream);
}

}  // extern "C"
