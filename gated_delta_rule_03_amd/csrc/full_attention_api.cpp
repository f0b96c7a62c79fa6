// Host side of the full-attention layers' operators: norm and rotation of the
// query and key heads with its backward, the paged cache and attention over
// it.  Validation and launches on the caller's stream; no allocation, no
// synchronisation, no host reads of device memory.
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "api_util.h"
#include "kda_internal.h"

namespace {

using kda::align_up;
using kda::stage;

constexpr int32_t kMaxHeads = 65535;
constexpr int32_t kMaxSequences = 1 << 24;            // kda_append_kv, kda_read_kv
constexpr int32_t kMaxAttentionSequences = 4096;      // their block counts sit in shared memory
constexpr int64_t kMaxAttentionRows = 1 << 30;        // n_tokens * num_heads

bool known_dtype(int32_t t) { return t == KDA_BF16 || t == KDA_FP32; }

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// What every one of these operators refuses of a geometry.
kda_status_t check_shape(const kda_config_t* cfg, int64_t n_tokens, int64_t kv_heads, int64_t least_kv) {
  if (!cfg) return KDA_ERR_INVALID_ARGUMENT;
  if (cfg->num_heads < 1 || cfg->head_k_dim < 1 || n_tokens < 0 || kv_heads < least_kv) return KDA_ERR_INVALID_ARGUMENT;
  const int d = cfg->head_k_dim;
  if ((d != 64 && d != 128 && d != 256) || cfg->head_v_dim != d) return KDA_ERR_UNSUPPORTED;
  if (cfg->num_heads > kMaxHeads || kv_heads > kMaxHeads) return KDA_ERR_UNSUPPORTED;
  if (!known_dtype(cfg->io_dtype) || !known_dtype(cfg->out_dtype)) return KDA_ERR_UNSUPPORTED;
  if (n_tokens > INT64_MAX / (8ll * (cfg->num_heads + kv_heads) * d)) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

kda_status_t check_rope(const kda_config_t* cfg, const kda_rope_t* rope) {
  if (!rope) return KDA_OK;
  if (rope->rotary_dim < 0 || rope->num_axes < 1 || (rope->interleaved != 0 && rope->interleaved != 1))
    return KDA_ERR_INVALID_ARGUMENT;
  if (rope->rotary_dim % 16 || rope->rotary_dim > cfg->head_k_dim || rope->num_axes > 4) return KDA_ERR_UNSUPPORTED;
  if (rope->rotary_dim > 0 && !rope->inv_freq) return KDA_ERR_INVALID_ARGUMENT;
  if (!aligned(rope->inv_freq, 4) || !aligned(rope->axis, 4)) return KDA_ERR_INVALID_ARGUMENT;
  return KDA_OK;
}

kda::RopeArgs rope_args(const kda_rope_t* rope, const int32_t* positions, int64_t n_tokens) {
  kda::RopeArgs r = {0, 0, 1, nullptr, nullptr, positions, n_tokens};
  if (rope && rope->rotary_dim > 0) {
    r.rotary_dim = rope->rotary_dim;
    r.interleaved = rope->interleaved;
    r.num_axes = rope->num_axes;
    r.inv_freq = rope->inv_freq;
    r.axis = rope->axis;
  }
  return r;
}

// A row stride of `heads` heads: whole 16-byte steps, no overlap.
bool bad_stride(int64_t stride, int64_t heads, int d) { return stride % 8 || stride < heads * d; }

bool far_stride(int64_t stride, int64_t n_tokens) { return n_tokens > 0 && stride > INT64_MAX / 4 / n_tokens; }

kda_status_t check_heads(const kda_config_t* cfg, const kda_rope_t* rope, int64_t n_tokens, int32_t kv_heads,
                         int64_t q_stride, int64_t k_stride, float eps) {
  kda_status_t s = check_shape(cfg, n_tokens, kv_heads, 0);
  if (s == KDA_OK) s = check_rope(cfg, rope);
  if (s != KDA_OK) return s;
  if (std::isnan(eps) || eps < 0.f) return KDA_ERR_INVALID_ARGUMENT;
  if (bad_stride(q_stride, cfg->num_heads, cfg->head_k_dim) ||
      (kv_heads > 0 && bad_stride(k_stride, kv_heads, cfg->head_k_dim)))
    return KDA_ERR_INVALID_ARGUMENT;
  if (far_stride(q_stride, n_tokens) || (kv_heads > 0 && far_stride(k_stride, n_tokens))) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

// What the operators on a cache refuse of it; N and n_tokens are positive.
kda_status_t check_cache(const kda_kv_cache_t* c) {
  if (c->num_pages < 0 || c->max_pages < 0 || c->page_size < 1) return KDA_ERR_INVALID_ARGUMENT;
  if (c->page_size != 32 && c->page_size != 64 && c->page_size != 128 && c->page_size != 256) return KDA_ERR_UNSUPPORTED;
  if (!c->lengths || (c->max_pages > 0 && !c->page_table)) return KDA_ERR_INVALID_ARGUMENT;
  if (c->num_pages > 0 && (!c->k || !c->k_scale || !c->v || !c->v_scale)) return KDA_ERR_INVALID_ARGUMENT;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 8) || !aligned(c->v_scale, 8) ||
      !aligned(c->page_table, 4) || !aligned(c->lengths, 4) || !aligned(c->cu_seqlens, 4))
    return KDA_ERR_INVALID_ARGUMENT;
  return KDA_OK;
}

kda::CacheArgs cache_args(const kda_kv_cache_t* c, int32_t N, int64_t n_tokens) {
  int shift = 0;
  while ((1 << shift) < c->page_size) ++shift;
  return {static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->k_scale), static_cast<uint8_t*>(c->v),
          static_cast<uint8_t*>(c->v_scale), c->num_pages, shift, c->num_kv_heads, c->max_pages, c->page_table,
          c->lengths, c->cu_seqlens, N, n_tokens};
}

kda_status_t check_attention(const kda_config_t* cfg, int32_t kv_heads, int32_t N, int64_t n_tokens, int32_t max_q) {
  const kda_status_t s = check_shape(cfg, n_tokens, kv_heads, 1);
  if (s != KDA_OK) return s;
  if (N < 0 || max_q < 0 || cfg->num_heads % kv_heads) return KDA_ERR_INVALID_ARGUMENT;
  if (N > kMaxAttentionSequences || n_tokens > kMaxAttentionRows / cfg->num_heads) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

}  // namespace

extern "C" {

kda_status_t kda_qk_norm_rope(const kda_config_t* cfg, const kda_rope_t* rope, int64_t n_tokens, int32_t num_kv_heads,
                              const void* q, int64_t q_stride, const void* k, int64_t k_stride, const float* q_weight,
                              const float* k_weight, float eps, const int32_t* positions, void* q_out, void* k_out,
                              void* stream) {
  const kda_status_t s = check_heads(cfg, rope, n_tokens, num_kv_heads, q_stride, k_stride, eps);
  if (s != KDA_OK) return s;
  if (n_tokens == 0) return KDA_OK;
  if (!q || !q_out || (num_kv_heads > 0 && (!k || !k_out))) return KDA_ERR_INVALID_ARGUMENT;
  if (rope && rope->rotary_dim > 0 && !positions) return KDA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(q_out, 16) ||
      !aligned(k_out, 16) || !aligned(positions, 4))
    return KDA_ERR_INVALID_ARGUMENT;
  const kda::QkArgs x = {{cfg->num_heads, num_kv_heads}, {q, k},         {q_stride, k_stride},
                         {q_weight, k_weight},           {nullptr, nullptr}, {q_out, k_out}};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return stage(cfg, KDA_STAGE_ROPE, st, [&] {
    return kda::launch_qk_norm_rope(cfg->head_k_dim, rope_args(rope, positions, n_tokens), x, eps,
                                    cfg->io_dtype == KDA_BF16, cfg->out_dtype == KDA_BF16, st);
  });
}

size_t kda_qk_norm_rope_backward_workspace_bytes(const kda_config_t* cfg, int64_t n_tokens, int32_t num_kv_heads) {
  if (check_shape(cfg, n_tokens, num_kv_heads, 0) != KDA_OK) return 0;
  const int d = cfg->head_k_dim;
  const size_t parts = static_cast<size_t>(kda::qk_norm_rope_bwd_parts(d, n_tokens, cfg->num_heads + num_kv_heads));
  return align_up((parts ? parts : 1) * 2 * d * 4);
}

kda_status_t kda_qk_norm_rope_backward(const kda_config_t* cfg, const kda_rope_t* rope, int64_t n_tokens,
                                       int32_t num_kv_heads, const void* q, int64_t q_stride, const void* k,
                                       int64_t k_stride, const float* q_weight, const float* k_weight, float eps,
                                       const int32_t* positions, const void* dq_out, const void* dk_out, float* dq,
                                       float* dk, float* d_weight, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  const kda_status_t s = check_heads(cfg, rope, n_tokens, num_kv_heads, q_stride, k_stride, eps);
  if (s != KDA_OK) return s;
  if (!d_weight || !workspace) return KDA_ERR_INVALID_ARGUMENT;
  if (n_tokens > 0) {
    if (!q || !dq_out || !dq || (num_kv_heads > 0 && (!k || !dk_out || !dk))) return KDA_ERR_INVALID_ARGUMENT;
    if (rope && rope->rotary_dim > 0 && !positions) return KDA_ERR_INVALID_ARGUMENT;
  }
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(dq_out, 16) ||
      !aligned(dk_out, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(d_weight, 16) ||
      !aligned(workspace, 16) || !aligned(positions, 4))
    return KDA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < kda_qk_norm_rope_backward_workspace_bytes(cfg, n_tokens, num_kv_heads))
    return KDA_ERR_WORKSPACE_TOO_SMALL;
  const kda::QkArgs x = {{cfg->num_heads, num_kv_heads}, {q, k},           {q_stride, k_stride},
                         {q_weight, k_weight},           {dq_out, dk_out}, {dq, dk}};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return stage(cfg, KDA_STAGE_BACKWARD, st, [&] {
    return kda::launch_qk_norm_rope_bwd(cfg->head_k_dim, rope_args(rope, positions, n_tokens), x, eps, d_weight,
                                        static_cast<float*>(workspace), cfg->io_dtype == KDA_BF16,
                                        cfg->out_dtype == KDA_BF16, st);
  });
}

kda_status_t kda_append_kv(const kda_config_t* cfg, const kda_rope_t* rope, const kda_kv_cache_t* cache, int32_t N,
                           int64_t n_tokens, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           const float* k_weight, float eps, const int32_t* positions, void* stream) {
  if (!cache) return KDA_ERR_INVALID_ARGUMENT;
  kda_status_t s = check_shape(cfg, n_tokens, cache->num_kv_heads, 1);
  if (s == KDA_OK) s = check_rope(cfg, rope);
  if (s != KDA_OK) return s;
  if (N < 0 || std::isnan(eps) || eps < 0.f) return KDA_ERR_INVALID_ARGUMENT;
  if (N > kMaxSequences) return KDA_ERR_UNSUPPORTED;
  if (bad_stride(k_stride, cache->num_kv_heads, cfg->head_k_dim) ||
      bad_stride(v_stride, cache->num_kv_heads, cfg->head_k_dim))
    return KDA_ERR_INVALID_ARGUMENT;
  if (far_stride(k_stride, n_tokens) || far_stride(v_stride, n_tokens)) return KDA_ERR_UNSUPPORTED;
  if (N == 0 || n_tokens == 0) return KDA_OK;
  s = check_cache(cache);
  if (s != KDA_OK) return s;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_weight, 16) || !aligned(positions, 4))
    return KDA_ERR_INVALID_ARGUMENT;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return stage(cfg, KDA_STAGE_CACHE, st, [&] {
    return kda::launch_append_kv(cfg->head_k_dim, rope_args(rope, positions, n_tokens), cache_args(cache, N, n_tokens),
                                 k, k_stride, v, v_stride, k_weight, eps, cfg->io_dtype == KDA_BF16, st);
  });
}

kda_status_t kda_read_kv(const kda_config_t* cfg, const kda_kv_cache_t* cache, int32_t N, int64_t n_tokens,
                         void* k_out, void* v_out, void* stream) {
  if (!cache) return KDA_ERR_INVALID_ARGUMENT;
  kda_status_t s = check_shape(cfg, n_tokens, cache->num_kv_heads, 1);
  if (s != KDA_OK) return s;
  if (N < 0) return KDA_ERR_INVALID_ARGUMENT;
  if (N > kMaxSequences) return KDA_ERR_UNSUPPORTED;
  if (N == 0 || n_tokens == 0 || (!k_out && !v_out)) return KDA_OK;
  s = check_cache(cache);
  if (s != KDA_OK) return s;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return KDA_ERR_INVALID_ARGUMENT;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return stage(cfg, KDA_STAGE_CACHE, st, [&] {
    return kda::launch_read_kv(cfg->head_k_dim, cache_args(cache, N, n_tokens), k_out, v_out,
                               cfg->out_dtype == KDA_BF16, st);
  });
}

size_t kda_paged_attention_workspace_bytes(const kda_config_t* cfg, int32_t num_kv_heads, int32_t N, int64_t n_tokens,
                                           int32_t max_q) {
  if (check_attention(cfg, num_kv_heads, N, n_tokens, max_q) != KDA_OK) return 0;
  return align_up(kda::paged_attention_ws(cfg->head_k_dim, N, num_kv_heads, cfg->num_heads / num_kv_heads, n_tokens, max_q,
                                          cfg->io_dtype == KDA_BF16, cfg->out_dtype == KDA_BF16));
}

kda_status_t kda_paged_attention(const kda_config_t* cfg, const kda_kv_cache_t* cache, int32_t N, int64_t n_tokens,
                                 int32_t max_q, const void* q, float scale, void* o, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (!cache) return KDA_ERR_INVALID_ARGUMENT;
  kda_status_t s = check_attention(cfg, cache->num_kv_heads, N, n_tokens, max_q);
  if (s != KDA_OK) return s;
  if (!std::isfinite(scale)) return KDA_ERR_INVALID_ARGUMENT;
  if (N == 0 || n_tokens == 0) return KDA_OK;
  s = check_cache(cache);
  if (s != KDA_OK) return s;
  if (!q || !o || !workspace || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 16))
    return KDA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < kda_paged_attention_workspace_bytes(cfg, cache->num_kv_heads, N, n_tokens, max_q))
    return KDA_ERR_WORKSPACE_TOO_SMALL;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return stage(cfg, KDA_STAGE_ATTENTION, st, [&] {
    return kda::launch_paged_attention(cfg->head_k_dim, cache_args(cache, N, n_tokens), q,
                                       cfg->num_heads / cache->num_kv_heads, scale, max_q, o, lse, workspace,
                                       cfg->io_dtype == KDA_BF16, cfg->out_dtype == KDA_BF16, st);
  });
}

}  // extern "C"
