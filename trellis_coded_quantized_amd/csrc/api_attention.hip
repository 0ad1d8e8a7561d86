// api_attention.hip -- the C ABI of the attention operators and the cache's
// page operations (include/trellis.h): host-side validation and dispatch.
// Nothing is launched or written unless every check passes.
#include <cmath>

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

int need_ptr(const char* fn, const char* name, const void* p, size_t align) {
  if (!p) return api_fail(TRELLIS_EINVAL, "%s: %s is NULL", fn, name);
  if (reinterpret_cast<uintptr_t>(p) % align != 0)
    return api_fail(TRELLIS_EINVAL, "%s: %s not %zu-byte aligned", fn, name, align);
  return TRELLIS_OK;
}

int need_workspace(const char* fn, const void* ws, size_t have, size_t need) {
  if (need == 0) return TRELLIS_OK;
  if (have < need) return api_fail(TRELLIS_EWORKSPACE, "%s: workspace %zu bytes < required %zu", fn, have, need);
  return need_ptr(fn, "workspace", ws, 256);
}

// sizes and types of the cache; pointers are checked apart (size queries have none)
int check_cache(const char* fn, const trellis_kv_cache* c) {
  if (!c) return api_fail(TRELLIS_EINVAL, "%s: cache is NULL", fn);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return api_fail(TRELLIS_EUNSUPPORTED, "%s: head_dim=%d not in {64, 128, 256}", fn, c->head_dim);
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    return api_fail(TRELLIS_EUNSUPPORTED, "%s: page_size=%d not a power of two in 16..256", fn, c->page_size);
  if (c->dtype != TRELLIS_KV_BF16 && c->dtype != TRELLIS_KV_F16)
    return api_fail(TRELLIS_EINVAL, "%s: dtype=%d unknown", fn, c->dtype);
  if (c->heads < 1 || c->heads > 1024) return api_fail(TRELLIS_EINVAL, "%s: heads=%d outside 1..1024", fn, c->heads);
  if (c->layers < 1 || c->layers > 65535)
    return api_fail(TRELLIS_EINVAL, "%s: layers=%d outside 1..65535", fn, c->layers);
  if (c->pages < 1 || c->pages >= kMaxIndex || c->pages * c->page_size >= kMaxIndex)
    return api_fail(TRELLIS_EINVAL, "%s: pages=%lld (slots must number 1..2^31-1)", fn, (long long)c->pages);
  return TRELLIS_OK;
}

int check_cache_data(const char* fn, const trellis_kv_cache* c) {
  TRY(need_ptr(fn, "cache k", c->k, 16));
  return need_ptr(fn, "cache v", c->v, 16);
}

int check_one_layer(const char* fn, const trellis_kv_cache* c) {
  if (c->layers != 1)
    return api_fail(TRELLIS_EINVAL, "%s: layers=%d, this call works on one layer", fn, c->layers);
  return TRELLIS_OK;
}

int check_state(const char* fn, const trellis_kv_cache* c, const trellis_kv_state* s) {
  if (!s) return api_fail(TRELLIS_EINVAL, "%s: state is NULL", fn);
  if (s->seqs < 1 || s->seqs >= kMaxIndex || s->width < 1 || s->width >= kMaxIndex ||
      s->width * c->page_size >= kMaxIndex)
    return api_fail(TRELLIS_EINVAL, "%s: table of %lld x %lld (width * page_size must stay below 2^31)", fn,
                    (long long)s->seqs, (long long)s->width);
  return TRELLIS_OK;
}

int check_state_data(const char* fn, const trellis_kv_state* s, bool refs) {
  TRY(need_ptr(fn, "table", s->table, 16));
  TRY(need_ptr(fn, "lengths", s->lengths, 16));
  return refs ? need_ptr(fn, "refs", s->refs, 16) : TRELLIS_OK;
}

int check_heads(const char* fn, int heads_q, const trellis_kv_cache* c) {
  if (heads_q < 1 || heads_q % c->heads != 0 || heads_q > 65535)
    return api_fail(TRELLIS_EINVAL, "%s: heads_q=%d not a multiple of the cache's %d heads", fn, heads_q, c->heads);
  return TRELLIS_OK;
}

int check_stride(const char* fn, const char* name, int64_t stride, int64_t row) {
  if (stride % 8 != 0 || stride < row)
    return api_fail(TRELLIS_EINVAL, "%s: %s=%lld not a multiple of 8 of at least %lld", fn, name, (long long)stride,
                    (long long)row);
  return TRELLIS_OK;
}

int check_tokens(const char* fn, int64_t tokens) {
  if (tokens < 0 || tokens >= kMaxIndex)
    return api_fail(TRELLIS_EINVAL, "%s: tokens=%lld outside 0..2^31-1", fn, (long long)tokens);
  return TRELLIS_OK;
}

int log2_of(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

// sizes of an attention call, without its pointers
int attention_sizes(const char* fn, const trellis_kv_cache* cache, const trellis_kv_state* state, int n,
                    int64_t tokens, int heads_q, int max_q, bool tree, int window, int sinks, trellis::AttnArgs* a) {
  TRY(check_cache(fn, cache));
  TRY(check_one_layer(fn, cache));
  TRY(check_state(fn, cache, state));
  TRY(check_heads(fn, heads_q, cache));
  TRY(check_tokens(fn, tokens));
  if (n < 1 || n > 65535) return api_fail(TRELLIS_EINVAL, "%s: n=%d entries outside 1..65535", fn, n);
  if (max_q < 1 || (tree && max_q > TRELLIS_TREE_MAX))
    return api_fail(TRELLIS_EINVAL, "%s: max_q=%d outside 1..%d", fn, max_q, tree ? TRELLIS_TREE_MAX : 2147483647);
  if (window < 0 || sinks < 0)
    return api_fail(TRELLIS_EINVAL, "%s: window=%d, sinks=%d must not be negative", fn, window, sinks);
  *a = trellis::AttnArgs{};
  a->tokens = tokens;
  a->width = state->width;
  a->seqs = state->seqs;
  a->pages = (uint32_t)cache->pages;
  a->entries = n;
  a->max_q = (int64_t)max_q < tokens ? max_q : tokens > 0 ? (int)tokens : 1;
  a->heads_q = heads_q;
  a->heads_kv = cache->heads;
  a->head_dim = cache->head_dim;
  a->page_log2 = log2_of(cache->page_size);
  a->tree = tree;
  a->window = window;
  const int64_t room = state->width * cache->page_size;
  a->sinks = (int64_t)sinks < room ? sinks : (int)room;
  a->fp16 = cache->dtype == TRELLIS_KV_F16;
  return TRELLIS_OK;
}

int attention(const char* fn, const uint16_t* q, int64_t q_stride, const trellis_kv_cache* cache,
              const trellis_kv_state* state, const int32_t* seq_ids, int n, const int32_t* q_start,
              const int64_t* ancestors, int64_t tokens, int heads_q, int max_q, bool tree, int window, int sinks,
              float scale, uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  trellis::AttnArgs a;
  TRY(attention_sizes(fn, cache, state, n, tokens, heads_q, max_q, tree, window, sinks, &a));
  TRY(check_stride(fn, "q_stride", q_stride, (int64_t)heads_q * cache->head_dim));
  if (!(scale > 0.0f) || std::isinf(scale)) return api_fail(TRELLIS_EINVAL, "%s: scale=%g not finite and > 0", fn, scale);
  TRY(check_cache_data(fn, cache));
  TRY(check_state_data(fn, state, false));
  if (tokens == 0) return trellis::api_ok();
  TRY(need_ptr(fn, "q", q, 16));
  TRY(need_ptr(fn, "q_start", q_start, 4));
  if (tree) TRY(need_ptr(fn, "ancestors", ancestors, 8));
  if (seq_ids) TRY(need_ptr(fn, "seq_ids", seq_ids, 4));
  TRY(need_ptr(fn, "out", out, 16));
  TRY(need_workspace(fn, workspace, workspace_bytes, trellis::attention_workspace_bytes(a)));
  a.q = q;
  a.q_stride = q_stride;
  a.k = cache->k;
  a.v = cache->v;
  a.table = state->table;
  a.lengths = state->lengths;
  a.seq_ids = seq_ids;
  a.q_start = q_start;
  a.ancestors = ancestors;
  a.out = out;
  a.scale = scale;
  return trellis::api_hip(fn, trellis::launch_attention(a, workspace, (hipStream_t)stream));
}

// checks shared by the page operations
int cache_call(const char* fn, const trellis_kv_cache* cache, const trellis_kv_state* state, int n, bool data,
               trellis::CacheArgs* c) {
  TRY(check_cache(fn, cache));
  TRY(check_state(fn, cache, state));
  if (n < 1 || n > TRELLIS_CACHE_MAX_SEQS)
    return api_fail(TRELLIS_EINVAL, "%s: n=%d sequences outside 1..%d", fn, n, TRELLIS_CACHE_MAX_SEQS);
  if (state->width * n >= kMaxIndex)
    return api_fail(TRELLIS_EINVAL, "%s: %d rows of %lld pages are too many for one call", fn, n,
                    (long long)state->width);
  if (data) TRY(check_state_data(fn, state, true));
  *c = trellis::CacheArgs{cache->k,    cache->v,     state->table,           state->lengths, state->refs,
                          state->seqs, state->width, (uint32_t)cache->pages, cache->layers,  cache->heads,
                          cache->head_dim, log2_of(cache->page_size)};
  return TRELLIS_OK;
}

}  // namespace

extern "C" {

int trellis_qk_norm_rope(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                         int64_t v_stride, const uint16_t* q_weight, const uint16_t* k_weight,
                         const int32_t* positions, const float* inv_freq, int rotary_dim, int interleaved, float eps,
                         const int32_t* slots, uint16_t* out, const trellis_kv_cache* cache, int64_t tokens,
                         int heads_q, void* stream) {
  const char* fn = "trellis_qk_norm_rope";
  TRY(check_cache(fn, cache));
  TRY(check_one_layer(fn, cache));
  if (heads_q < 1 || heads_q > 65535) return api_fail(TRELLIS_EINVAL, "%s: heads_q=%d outside 1..65535", fn, heads_q);
  TRY(check_tokens(fn, tokens));
  const int64_t D = cache->head_dim;
  TRY(check_stride(fn, "q_stride", q_stride, heads_q * D));
  TRY(check_stride(fn, "k_stride", k_stride, cache->heads * D));
  TRY(check_stride(fn, "v_stride", v_stride, cache->heads * D));
  if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 16 != 0)
    return api_fail(TRELLIS_EINVAL, "%s: rotary_dim=%d not a multiple of 16 in 0..%d", fn, rotary_dim, (int)D);
  if (!(eps >= 0.0f) || std::isinf(eps)) return api_fail(TRELLIS_EINVAL, "%s: eps=%g not finite and >= 0", fn, eps);
  TRY(check_cache_data(fn, cache));
  if (tokens == 0) return trellis::api_ok();
  TRY(need_ptr(fn, "q", q, 16));
  TRY(need_ptr(fn, "k", k, 16));
  TRY(need_ptr(fn, "v", v, 16));
  TRY(need_ptr(fn, "q_weight", q_weight, 16));
  TRY(need_ptr(fn, "k_weight", k_weight, 16));
  TRY(need_ptr(fn, "positions", positions, 4));
  if (rotary_dim) TRY(need_ptr(fn, "inv_freq", inv_freq, 4));
  TRY(need_ptr(fn, "slots", slots, 4));
  TRY(need_ptr(fn, "out", out, 16));
  trellis::QkNormRopeArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.positions = positions;
  a.slots = slots;
  a.inv_freq = inv_freq;
  a.out = out;
  a.k_cache = cache->k;
  a.v_cache = cache->v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.tokens = tokens;
  a.pages = (uint32_t)cache->pages;
  a.heads_q = heads_q;
  a.heads_kv = cache->heads;
  a.head_dim = cache->head_dim;
  a.rotary = rotary_dim;
  a.page_log2 = log2_of(cache->page_size);
  a.interleaved = interleaved != 0;
  a.fp16 = cache->dtype == TRELLIS_KV_F16;
  a.eps = eps;
  return trellis::api_hip(fn, trellis::launch_qk_norm_rope(a, (hipStream_t)stream));
}

size_t trellis_tree_attention_workspace_bytes(const trellis_kv_cache* cache, const trellis_kv_state* state, int n,
                                              int64_t tokens, int heads_q, int max_q) {
  trellis::AttnArgs a;
  if (attention_sizes("trellis_tree_attention_workspace_bytes", cache, state, n, tokens, heads_q, max_q, true, 0, 0,
                      &a) != TRELLIS_OK)
    return 0;
  return tokens ? trellis::attention_workspace_bytes(a) : 0;
}

int trellis_tree_attention(const uint16_t* q, int64_t q_stride, const trellis_kv_cache* cache,
                           const trellis_kv_state* state, const int32_t* seq_ids, int n, const int32_t* q_start,
                           const int64_t* ancestors, int64_t tokens, int heads_q, int max_q, float scale,
                           uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  return attention("trellis_tree_attention", q, q_stride, cache, state, seq_ids, n, q_start, ancestors, tokens,
                   heads_q, max_q, true, 0, 0, scale, out, workspace, workspace_bytes, stream);
}

size_t trellis_window_attention_workspace_bytes(const trellis_kv_cache* cache, const trellis_kv_state* state, int n,
                                                int64_t tokens, int heads_q, int max_q, int window, int sinks) {
  trellis::AttnArgs a;
  if (attention_sizes("trellis_window_attention_workspace_bytes", cache, state, n, tokens, heads_q, max_q, false,
                      window, sinks, &a) != TRELLIS_OK)
    return 0;
  return tokens ? trellis::attention_workspace_bytes(a) : 0;
}

int trellis_window_attention(const uint16_t* q, int64_t q_stride, const trellis_kv_cache* cache,
                             const trellis_kv_state* state, const int32_t* seq_ids, int n, const int32_t* q_start,
                             int64_t tokens, int heads_q, int max_q, int window, int sinks, float scale,
                             uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  return attention("trellis_window_attention", q, q_stride, cache, state, seq_ids, n, q_start, nullptr, tokens,
                   heads_q, max_q, false, window, sinks, scale, out, workspace, workspace_bytes, stream);
}

size_t trellis_cache_reserve_workspace_bytes(const trellis_kv_cache* cache, const trellis_kv_state* state, int n) {
  trellis::CacheArgs c;
  if (cache_call("trellis_cache_reserve_workspace_bytes", cache, state, n, false, &c) != TRELLIS_OK) return 0;
  return trellis::cache_reserve_workspace_bytes(c, n);
}

int trellis_cache_reserve(const trellis_kv_cache* cache, const trellis_kv_state* state, const int32_t* seq_ids, int n,
                          const int32_t* q_start, int64_t tokens, int32_t* slots, int32_t* granted, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const char* fn = "trellis_cache_reserve";
  trellis::CacheArgs c;
  TRY(cache_call(fn, cache, state, n, true, &c));
  TRY(check_tokens(fn, tokens));
  TRY(need_ptr(fn, "seq_ids", seq_ids, 4));
  TRY(need_ptr(fn, "q_start", q_start, 4));
  if (tokens) TRY(need_ptr(fn, "slots", slots, 4));
  TRY(need_ptr(fn, "granted", granted, 4));
  TRY(need_workspace(fn, workspace, workspace_bytes, trellis::cache_reserve_workspace_bytes(c, n)));
  return trellis::api_hip(fn, trellis::launch_cache_reserve(c, seq_ids, n, q_start, tokens, slots, granted, workspace,
                                                            (hipStream_t)stream));
}

size_t trellis_cache_fork_workspace_bytes(const trellis_kv_cache* cache, const trellis_kv_state* state, int n) {
  trellis::CacheArgs c;
  if (cache_call("trellis_cache_fork_workspace_bytes", cache, state, n, false, &c) != TRELLIS_OK) return 0;
  return trellis::cache_fork_workspace_bytes(c, n);
}

int trellis_cache_fork(const trellis_kv_cache* cache, const trellis_kv_state* state, const int32_t* parents,
                       const int32_t* children, int n, int32_t* granted, void* workspace, size_t workspace_bytes,
                       void* stream) {
  const char* fn = "trellis_cache_fork";
  trellis::CacheArgs c;
  TRY(cache_call(fn, cache, state, n, true, &c));
  TRY(check_cache_data(fn, cache));
  TRY(need_ptr(fn, "parents", parents, 4));
  TRY(need_ptr(fn, "children", children, 4));
  TRY(need_ptr(fn, "granted", granted, 4));
  TRY(need_workspace(fn, workspace, workspace_bytes, trellis::cache_fork_workspace_bytes(c, n)));
  return trellis::api_hip(fn, trellis::launch_cache_fork(c, parents, children, n, granted, workspace,
                                                         (hipStream_t)stream));
}

int trellis_cache_accept(const trellis_kv_cache* cache, const trellis_kv_state* state, const int32_t* seq_ids, int n,
                         const int32_t* path, int max_path, const int32_t* counts, int32_t* new_lengths, void* stream) {
  const char* fn = "trellis_cache_accept";
  trellis::CacheArgs c;
  TRY(cache_call(fn, cache, state, n, false, &c));
  TRY(check_state_data(fn, state, false));
  TRY(check_cache_data(fn, cache));
  if (max_path < 1 || max_path > TRELLIS_ACCEPT_MAX)
    return api_fail(TRELLIS_EINVAL, "%s: max_path=%d outside 1..%d", fn, max_path, TRELLIS_ACCEPT_MAX);
  TRY(need_ptr(fn, "seq_ids", seq_ids, 4));
  TRY(need_ptr(fn, "path", path, 4));
  TRY(need_ptr(fn, "counts", counts, 4));
  TRY(need_ptr(fn, "new_lengths", new_lengths, 4));
  return trellis::api_hip(fn, trellis::launch_cache_accept(c, seq_ids, n, path, max_path, counts, new_lengths,
                                                           (hipStream_t)stream));
}

int trellis_cache_free(const trellis_kv_cache* cache, const trellis_kv_state* state, const int32_t* seq_ids, int n,
                       void* stream) {
  const char* fn = "trellis_cache_free";
  trellis::CacheArgs c;
  TRY(cache_call(fn, cache, state, n, true, &c));
  TRY(need_ptr(fn, "seq_ids", seq_ids, 4));
  return trellis::api_hip(fn, trellis::launch_cache_free(c, seq_ids, n, (hipStream_t)stream));
}

}  // extern "C"
