// Host side of the operators around the core: the residual RMS norm, the
// output epilogue's 8-bit form, both backward passes and the block-scaled
// e4m3 product.  Validation and launches on the caller's stream; no
// allocation, no synchronisation, no host reads of device memory.
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "api_util.h"
#include "kda_internal.h"

namespace {

using kda::align_up;
using kda::stage;

bool known_dtype(int32_t t) { return t == KDA_BF16 || t == KDA_FP32; }

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

bool bad_eps(float eps) { return std::isnan(eps) || eps < 0.f; }

// What the norm and its backward refuse of a row length and a token count.
kda_status_t check_rows(const kda_config_t* cfg, int64_t n_tokens, int32_t hidden) {
  if (!cfg) return KDA_ERR_INVALID_ARGUMENT;
  if (!known_dtype(cfg->io_dtype) || !known_dtype(cfg->out_dtype)) return KDA_ERR_UNSUPPORTED;
  if (n_tokens < 0 || hidden < 1) return KDA_ERR_INVALID_ARGUMENT;
  if (hidden % 8 || hidden > kda::kMaxHidden) return KDA_ERR_UNSUPPORTED;
  if (n_tokens > INT64_MAX / (4 * static_cast<int64_t>(hidden))) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

// What the epilogue's 8-bit form and its backward refuse of a geometry.
kda_status_t check_heads(const kda_config_t* cfg, int64_t n_tokens) {
  if (!cfg) return KDA_ERR_INVALID_ARGUMENT;
  if (cfg->num_heads < 1 || cfg->head_v_dim < 1) return KDA_ERR_INVALID_ARGUMENT;
  if (cfg->num_heads > 65535) return KDA_ERR_UNSUPPORTED;
  const int dv = cfg->head_v_dim;
  if (dv != 16 && dv != 32 && dv != 64 && dv != 128) return KDA_ERR_UNSUPPORTED;
  if (!known_dtype(cfg->io_dtype) || !known_dtype(cfg->out_dtype)) return KDA_ERR_UNSUPPORTED;
  if (n_tokens < 0) return KDA_ERR_INVALID_ARGUMENT;
  if (n_tokens > INT64_MAX / (4 * static_cast<int64_t>(cfg->num_heads) * dv)) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

kda_status_t add_rmsnorm(const kda_config_t* cfg, int64_t n_tokens, int32_t hidden, const void* x,
                         const void* residual, const float* weight, float eps, void* h, void* y, float* y_scale,
                         bool fp8, void* stream) {
  const kda_status_t s = check_rows(cfg, n_tokens, hidden);
  if (s != KDA_OK) return s;
  if (bad_eps(eps)) return KDA_ERR_INVALID_ARGUMENT;
  if (n_tokens == 0) return KDA_OK;
  if (!x || !weight || !y || (fp8 && !y_scale)) return KDA_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(h, 16) ||
      !aligned(y, fp8 ? 8 : 16) || !aligned(y_scale, 4))
    return KDA_ERR_INVALID_ARGUMENT;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return stage(cfg, KDA_STAGE_NORM, st, [&] {
    return kda::launch_add_rmsnorm(n_tokens, hidden, x, residual, weight, eps, h, y, y_scale,
                                   cfg->io_dtype == KDA_BF16, cfg->out_dtype == KDA_BF16, st);
  });
}

}  // namespace

extern "C" {

kda_status_t kda_add_rmsnorm(const kda_config_t* cfg, int64_t n_tokens, int32_t hidden, const void* x,
                             const void* residual, const float* weight, float eps, void* h, void* y, void* stream) {
  return add_rmsnorm(cfg, n_tokens, hidden, x, residual, weight, eps, h, y, nullptr, false, stream);
}

kda_status_t kda_add_rmsnorm_fp8(const kda_config_t* cfg, int64_t n_tokens, int32_t hidden, const void* x,
                                 const void* residual, const float* weight, float eps, void* h, void* y,
                                 float* y_scale, void* stream) {
  return add_rmsnorm(cfg, n_tokens, hidden, x, residual, weight, eps, h, y, y_scale, true, stream);
}

size_t kda_add_rmsnorm_backward_workspace_bytes(const kda_config_t* cfg, int64_t n_tokens, int32_t hidden) {
  if (check_rows(cfg, n_tokens, hidden) != KDA_OK) return 0;
  const size_t parts = static_cast<size_t>(kda::add_rmsnorm_bwd_parts(n_tokens));
  return align_up((parts ? parts : 1) * static_cast<size_t>(hidden) * 4);
}

kda_status_t kda_add_rmsnorm_backward(const kda_config_t* cfg, int64_t n_tokens, int32_t hidden, const void* h,
                                      const float* weight, float eps, const void* dy, const float* d_h, float* dx,
                                      float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  const kda_status_t s = check_rows(cfg, n_tokens, hidden);
  if (s != KDA_OK) return s;
  if (bad_eps(eps) || !dweight || !workspace) return KDA_ERR_INVALID_ARGUMENT;
  if (n_tokens > 0 && (!h || !weight || !dy || !dx)) return KDA_ERR_INVALID_ARGUMENT;
  if (!aligned(h, 16) || !aligned(weight, 16) || !aligned(dy, 16) || !aligned(d_h, 16) || !aligned(dx, 16) ||
      !aligned(dweight, 16) || !aligned(workspace, 16))
    return KDA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < kda_add_rmsnorm_backward_workspace_bytes(cfg, n_tokens, hidden))
    return KDA_ERR_WORKSPACE_TOO_SMALL;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return stage(cfg, KDA_STAGE_BACKWARD, st, [&] {
    return kda::launch_add_rmsnorm_bwd(n_tokens, hidden, h, weight, eps, dy, d_h, dx, dweight,
                                       static_cast<float*>(workspace), cfg->io_dtype == KDA_BF16,
                                       cfg->out_dtype == KDA_BF16, st);
  });
}

kda_status_t kda_output_gate_fp8(const kda_config_t* cfg, int64_t n_tokens, const void* o, const void* gate,
                                 const float* o_norm_weight, float eps, void* y, float* y_scale, void* stream) {
  const kda_status_t s = check_heads(cfg, n_tokens);
  if (s != KDA_OK) return s;
  if (bad_eps(eps)) return KDA_ERR_INVALID_ARGUMENT;
  if (n_tokens == 0) return KDA_OK;
  if (!o || !gate || !o_norm_weight || !y || !y_scale) return KDA_ERR_INVALID_ARGUMENT;
  if (!aligned(o, 16) || !aligned(gate, 16) || !aligned(o_norm_weight, 16) || !aligned(y, 8) || !aligned(y_scale, 4))
    return KDA_ERR_INVALID_ARGUMENT;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return stage(cfg, KDA_STAGE_OUTPUT_GATE, st, [&] {
    return kda::launch_output_gate_fp8(cfg->head_v_dim, n_tokens, cfg->num_heads * cfg->head_v_dim, o, gate,
                                       o_norm_weight, eps, static_cast<uint8_t*>(y), y_scale,
                                       cfg->out_dtype == KDA_BF16, cfg->io_dtype == KDA_BF16, st);
  });
}

size_t kda_output_gate_backward_workspace_bytes(const kda_config_t* cfg, int64_t n_tokens) {
  if (check_heads(cfg, n_tokens) != KDA_OK) return 0;
  const int dv = cfg->head_v_dim;
  const size_t parts = static_cast<size_t>(kda::output_gate_bwd_parts(dv, n_tokens * cfg->num_heads));
  return align_up((parts ? parts : 1) * dv * 4);
}

kda_status_t kda_output_gate_backward(const kda_config_t* cfg, int64_t n_tokens, const void* o, const void* gate,
                                      const float* o_norm_weight, float eps, const void* dy, void* d_o, float* d_gate,
                                      float* d_weight, void* workspace, size_t workspace_bytes, void* stream) {
  const kda_status_t s = check_heads(cfg, n_tokens);
  if (s != KDA_OK) return s;
  if (bad_eps(eps) || !d_weight || !workspace) return KDA_ERR_INVALID_ARGUMENT;
  if (n_tokens > 0 && (!o || !gate || !o_norm_weight || !dy || !d_o || !d_gate)) return KDA_ERR_INVALID_ARGUMENT;
  if (!aligned(o, 16) || !aligned(gate, 16) || !aligned(o_norm_weight, 16) || !aligned(dy, 16) || !aligned(d_o, 16) ||
      !aligned(d_gate, 16) || !aligned(d_weight, 16) || !aligned(workspace, 16))
    return KDA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < kda_output_gate_backward_workspace_bytes(cfg, n_tokens)) return KDA_ERR_WORKSPACE_TOO_SMALL;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return stage(cfg, KDA_STAGE_BACKWARD, st, [&] {
    return kda::launch_output_gate_bwd(cfg->head_v_dim, n_tokens * cfg->num_heads, o, gate, o_norm_weight, eps, dy,
                                       d_o, d_gate, d_weight, static_cast<float*>(workspace),
                                       cfg->out_dtype == KDA_BF16, cfg->io_dtype == KDA_BF16, st);
  });
}

kda_status_t kda_fp8_matmul(const kda_config_t* cfg, int64_t M, int32_t N, int32_t K, const void* a,
                            const float* a_scale, const void* w, const float* w_scale, void* y, void* stream) {
  if (!cfg) return KDA_ERR_INVALID_ARGUMENT;
  if (!known_dtype(cfg->out_dtype)) return KDA_ERR_UNSUPPORTED;
  if (M < 0 || N < 1 || K < 1) return KDA_ERR_INVALID_ARGUMENT;
  if (K % 16 || K > (1 << 20) || N > (1 << 20) || M > INT32_MAX) return KDA_ERR_UNSUPPORTED;
  if (M == 0) return KDA_OK;
  if (!a || !a_scale || !w || !w_scale || !y) return KDA_ERR_INVALID_ARGUMENT;
  if (!aligned(a, 16) || !aligned(a_scale, 4) || !aligned(w, 16) || !aligned(w_scale, 4) || !aligned(y, 16))
    return KDA_ERR_INVALID_ARGUMENT;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return stage(cfg, KDA_STAGE_MATMUL, st, [&] {
    return kda::launch_fp8_matmul(M, N, K, static_cast<const uint8_t*>(a), a_scale, static_cast<const uint8_t*>(w),
                                  w_scale, y, cfg->out_dtype == KDA_BF16, st);
  });
}

}  // extern "C"
