// Entry point of prompt attention in include/memra.h: argument validation and launch; its test hook.
#include "host_checks.cuh"
#include "memra_testing.h"
#include "prompt.cuh"

using namespace memra;

namespace {

int prompt_attn(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                const int32_t *cu_seqlens, int32_t batch, int32_t total_tokens, int32_t n_heads, int32_t n_kv_heads,
                int32_t head_dim, float sm_scale, int32_t window, void *out, int32_t *status, void *stream,
                int test_extra_tx = 0) {
  if (batch < 0 || total_tokens < 0 || n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || window < 0)
    return MEMRA_ERR_INVALID_ARG;
  if (head_dim != 128 && head_dim != 256) return MEMRA_ERR_UNSUPPORTED;
  if (n_heads / n_kv_heads > MEMRA_MAX_GROUP || n_kv_heads > 65535 || batch > 65535) return MEMRA_ERR_UNSUPPORTED;
  if (!std::isfinite(sm_scale) || !(sm_scale > 0.f)) return MEMRA_ERR_INVALID_ARG;
  const int64_t qw = static_cast<int64_t>(n_heads) * head_dim, kw = static_cast<int64_t>(n_kv_heads) * head_dim;
  // a token's heads lie side by side; 16-byte steps and 40-bit strides are what the tensor copies take
  if (q_stride < qw || k_stride < kw || v_stride < kw || ((q_stride | k_stride | v_stride) & 7))
    return MEMRA_ERR_INVALID_ARG;
  if (q_stride >= (1ll << 38) || k_stride >= (1ll << 38) || v_stride >= (1ll << 38)) return MEMRA_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(status) & 3u) return MEMRA_ERR_INVALID_ARG;
  if (batch == 0 || total_tokens == 0) return MEMRA_OK;
  if (!q || !k || !v || !cu_seqlens || !out || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u))
    return MEMRA_ERR_INVALID_ARG;
  PromptParams p;
  p.q = static_cast<const __half *>(q);
  p.k = static_cast<const __half *>(k);
  p.v = static_cast<const __half *>(v);
  p.cu_seqlens = cu_seqlens;
  p.out = static_cast<__half *>(out);
  p.status = status;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.batch = batch;
  p.total = total_tokens;
  p.n_heads = n_heads;
  p.n_kv_heads = n_kv_heads;
  p.group = n_heads / n_kv_heads;
  p.window = window;
  p.tpt = 128 / p.group;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.test_extra_tx = test_extra_tx;
  return cuda_status(launch_prompt(head_dim, p, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" int memra_prompt_attn(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                 int64_t v_stride, const int32_t *cu_seqlens, int32_t batch, int32_t total_tokens,
                                 int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, float sm_scale, int32_t window,
                                 void *out, int32_t *status, void *stream) {
  return prompt_attn(q, q_stride, k, k_stride, v, v_stride, cu_seqlens, batch, total_tokens, n_heads, n_kv_heads,
                     head_dim, sm_scale, window, out, status, stream);
}

// memra_testing.h: the same call with a first copy whose wait cannot complete.
extern "C" int memra_testing_prompt_attn_short_copy(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                                    const void *v, int64_t v_stride, const int32_t *cu_seqlens,
                                                    int32_t batch, int32_t total_tokens, int32_t n_heads,
                                                    int32_t n_kv_heads, int32_t head_dim, float sm_scale,
                                                    int32_t window, void *out, int32_t *status, void *stream) {
  return prompt_attn(q, q_stride, k, k_stride, v, v_stride, cu_seqlens, batch, total_tokens, n_heads, n_kv_heads,
                     head_dim, sm_scale, window, out, status, stream, 16);
}
