// internal.hpp -- host-side launchers shared between the C-ABI layer
// (api.hip) and the kernel translation units.  Every launcher assumes the
// caller already validated geometry, pointers and workspace size.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

namespace trellis {

// Raises one kernel's limit of dynamic LDS, once for each device.  Calls may
// come from several threads at a time: two that are both the first raise it
// twice, which does no harm.
class LdsLimit {
  std::atomic<uint64_t> raised_{0};

 public:
  hipError_t raise(const void* kernel, size_t bytes) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return hipErrorInvalidDevice;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (raised_.load(std::memory_order_acquire) & bit) return hipSuccess;
    const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == hipSuccess) raised_.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

// axis 1 (gate/up when codes1 != nullptr).  The persistent kernel keeps a
// ring of 16-row code tiles in LDS and x in registers; axis1_supported says
// whether a shape fits (LDS and register budget), checked on the host.
// Rows wider than 5120 columns run as column chunks into f32 partials in the
// workspace (axis1_workspace_bytes), folded by a second kernel.
constexpr size_t kAxis1MaxLdsBytes = 160 * 1024;
bool axis1_supported(int64_t R, int64_t C, int M, int k, bool gateup);
// grouped plain axis-1 call: n <= axis1_max_group() matrices of the same C
// and k over the same x, one launch (the row groups of all of them)
int axis1_max_group();
bool axis1_group_supported(const int64_t* R, int n, int64_t C, int M, int k);
hipError_t launch_axis1_group(const uint32_t* const* codes, const uint16_t* const* scales, void* const* outs,
                              const int64_t* R, int n, const uint16_t* x, int out_f32, int64_t C, int M, int k,
                              hipStream_t stream);
size_t axis1_workspace_bytes(int64_t R, int64_t C, int M, int k, bool gateup);
hipError_t launch_axis1(const uint32_t* codes0, const uint16_t* scales0, const uint32_t* codes1,
                        const uint16_t* scales1, const uint16_t* x, void* out, int out_f32,
                        float* gate_f32, float* up_f32, int64_t R, int64_t C, int M, int k,
                        void* workspace, hipStream_t stream);

// measurement probes: the gate/up kernel without the decode (timing floor,
// one launch, C <= 5120), and the register-only decode of `iters` runs per
// thread (the instruction mix of the matvec loop without memory)
hipError_t launch_gateup_decode_free(const uint32_t* c0, const uint16_t* s0, const uint32_t* c1, const uint16_t* s1,
                                     const uint16_t* x, uint16_t* out, int64_t R, int64_t C, int M, int k,
                                     hipStream_t stream);
constexpr int kProbeThreads = 512;
hipError_t launch_decode_only(const uint32_t* runs, float* wave_sums, int blocks, int iters, int k,
                              hipStream_t stream);

// axis 0 (split-K over stored rows, MFMA on 32-row blocks, then a fold)
bool axis0_supported(int64_t R, int64_t C, int M, int k);
size_t axis0_workspace_bytes(int64_t R, int64_t C, int M, int k);
// The static device scratch that stands in for the axis-0 workspace in the
// allocation-free call: kAxis0ScratchBytes per device, its address resolved
// once per device (the current one) and cached.
constexpr size_t kAxis0ScratchBytes = (size_t)4 << 20;
constexpr int kMaxDevices = 64;
hipError_t axis0_scratch(void** ptr);
// interleave: codes in the block-interleaved k = 3 layout [C/512, R, 48]
hipError_t launch_axis0(const uint32_t* codes, const uint16_t* scales, const uint16_t* x,
                        void* out, int out_f32, int64_t R, int64_t C, int M, int k,
                        void* workspace, hipStream_t stream, int interleave = 0);

// expansion and decode export
hipError_t launch_expand(const uint32_t* codes, const uint16_t* scales, uint16_t* out, int64_t R,
                         int64_t C, int k, hipStream_t stream, int interleave = 0);
hipError_t launch_decode_states(const uint32_t* codes, int64_t R, int64_t C, int k,
                                uint16_t* states, int16_t* y, float* value, hipStream_t stream);

// compute units of the current device (cached per device)
int device_cus();

// fused prefill (32-bit buffer offsets: x and the codes each below 2 GiB);
// the workspace holds x in operand order and the f32 partial tiles of the
// tiles split along the contraction.  R is the output count, C the
// contraction length: axis 1 codes [R, C k / 32]; axis0 != 0: codes
// [C, R k / 32] (the stored transpose), scales [C].
bool prefill_fused_supported(int64_t R, int64_t C, int64_t M, int k);
size_t prefill_fused_workspace_bytes(int64_t R, int64_t C, int64_t M, int axis0 = 0);
// interleave (axis 0, k = 3, R % 512 == 0): codes in the block-interleaved
// layout [R/512, C, 48].
hipError_t launch_prefill_fused(const uint32_t* codes, const uint16_t* scales, const uint16_t* x,
                                uint16_t* out, int64_t R, int64_t C, int64_t M, int k,
                                void* workspace, hipStream_t stream, int axis0 = 0, int interleave = 0);

// ---- low-rank adapters ----------------------------------------------------

struct LoraTarget {
  const uint16_t *a, *b;      // [pool, r, C], [pool, R, r]
  const void* y;
  void* out;
  int64_t R, y_stride, out_stride;
  int in_place;               // out is y: rows without an adapter need no copy
  int blocks;                 // column blocks of the second product
};

struct LoraArgs {
  const uint16_t* x;
  const int32_t *starts, *adapters, *ranks;   // ranks: NULL for r everywhere
  const float* scales;
  float* part;                // [splits, M, n * r]
  int64_t x_stride, M, C;
  LoraTarget target[4];
  int n, r, entries, pool, f32;
  int whole;                  // y and out: rows 16-byte aligned, whole granules of eight
  // filled by launch_lora
  int64_t chunk;
  int first_target, splits, cols, blocks, slots, bare;
};

// How a call is cut: row tiles, column chunks, bytes of the workspace.
struct LoraPlan {
  bool few;                   // short entries
  int splits;
  int64_t shrink_slots, expand_slots, chunk;
  size_t bytes;
};
LoraPlan lora_plan(int64_t M, int entries, int64_t C, int n, int r);
// swiglu: targets 0 and 1 are gate and up, target 0's out receives the result
hipError_t launch_lora(LoraArgs a, bool swiglu, hipStream_t stream);

// ---- attention over the paged cache and its page operations --------------

// Errors of the C entry points, wherever they are defined: set the thread's
// message and return the status.
int api_fail(int code, const char* fmt, ...);
int api_ok();
int api_hip(const char* fn, hipError_t e);

// What the fold of split keys has to know of a unit.
struct PartNote {
  int parts;                  // 0: nothing to fold here
  int first, rows;            // the entry's first row of q, its rows per key head
  int place;                  // few rows: slot of the first part; trees: row tile; else row tile << 1 | place
  int step;                   // trees: slots from part to part
};

// One attention call.  tree: `ancestors` is set, window and sinks are 0.
struct AttnArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* table;       // [seqs, width] pages
  const int32_t* lengths;     // [seqs]
  const int32_t* seq_ids;     // [entries] or NULL: entry e is sequence e
  const int32_t* q_start;     // [entries + 1]
  const int64_t* ancestors;   // [tokens], tree only
  uint16_t* out;
  float* part_o;              // partial outputs of split entries
  float* part_ml;             // their (bound, sum) pairs
  PartNote* part_note;
  int64_t tokens, q_stride, width, seqs;
  uint32_t pages;
  int entries, max_q, heads_q, heads_kv, head_dim, page_log2;
  int window, sinks, fp16;
  int tree;
  int target;                 // workgroups per key head that the keys are cut for
  int rounds;                 // slots a workgroup where units are many
  float scale;
};

// The same over a cache held in 8 bits: k and v are bytes.
struct Attn8Args : AttnArgs {
  const uint8_t* k_scale;     // [pages, heads, P/16] exponents
  const uint8_t* v_scale;
};

// Workspace of a call: filled into the args' part_* by launch_attention.
size_t attention_workspace_bytes(const AttnArgs& a);
hipError_t launch_attention(AttnArgs a, void* workspace, hipStream_t stream);
hipError_t launch_attention_kv8(Attn8Args a, void* workspace, hipStream_t stream);

struct QkNormRopeArgs {
  const uint16_t *q, *k, *v, *q_weight, *k_weight;
  const int32_t *positions, *slots;
  const float* inv_freq;
  uint16_t *out, *k_cache, *v_cache;
  int64_t q_stride, k_stride, v_stride, tokens;
  uint32_t pages;
  int heads_q, heads_kv, head_dim, rotary, page_log2, interleaved, fp16;
  float eps;
};
hipError_t launch_qk_norm_rope(const QkNormRopeArgs& a, hipStream_t stream);

// k_cache and v_cache of the base are not used.
struct QkNormRope8Args : QkNormRopeArgs {
  uint8_t *k8, *v8, *k_scale, *v_scale;
};
hipError_t launch_qk_norm_rope_kv8(const QkNormRope8Args& a, hipStream_t stream);

// Page operations.  table / lengths / refs are the cache's device state.
struct CacheArgs {
  uint16_t *k, *v;            // [layers, pages, heads, ...]
  int32_t *table, *lengths, *refs;
  int64_t seqs, width;
  uint32_t pages;
  int layers, heads, head_dim, page_log2;
};
constexpr int kCacheMaxEntries = 1024;    // sequences in one page operation
constexpr int kCacheMaxPath = 64;         // drafted rows kept by one accept
hipError_t launch_cache_reserve(const CacheArgs& c, const int32_t* seq_ids, int n, const int32_t* q_start,
                                int64_t tokens, int32_t* slots, int32_t* granted, void* workspace, hipStream_t stream);
size_t cache_reserve_workspace_bytes(const CacheArgs& c, int n);
hipError_t launch_cache_fork(const CacheArgs& c, const int32_t* parents, const int32_t* children, int n,
                             int32_t* granted, void* workspace, hipStream_t stream);
size_t cache_fork_workspace_bytes(const CacheArgs& c, int n);
hipError_t launch_cache_accept(const CacheArgs& c, const int32_t* seq_ids, int n, const int32_t* path, int max_path,
                               const int32_t* counts, int32_t* new_lengths, hipStream_t stream);
hipError_t launch_cache_free(const CacheArgs& c, const int32_t* seq_ids, int n, hipStream_t stream);

// The cache held in 8 bits: k and v of the CacheArgs are bytes.
struct Scales {
  uint8_t *k, *v;             // [layers, pages, heads, P/16]
};
hipError_t launch_cache_fork_kv8(const CacheArgs& c, const Scales& s, const int32_t* parents, const int32_t* children,
                                 int n, int32_t* granted, void* workspace, hipStream_t stream);
hipError_t launch_cache_accept_kv8(const CacheArgs& c, const Scales& s, const int32_t* seq_ids, int n,
                                   const int32_t* path, int max_path, const int32_t* counts, int32_t* new_lengths,
                                   hipStream_t stream);

}  // namespace trellis
