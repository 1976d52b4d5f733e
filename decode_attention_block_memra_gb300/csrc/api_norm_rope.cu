// Entry point of the norm, rotation and append of rows in include/memra.h: argument validation and the launch.
#include "host_checks.cuh"
#include "norm_rope.cuh"

using namespace memra;

namespace {

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A token's heads lie side by side and every row starts on a 16-byte boundary.
bool rows_ok(const void *p, int64_t stride, int32_t heads, int32_t head_dim) {
  return p && aligned16(p) && stride >= static_cast<int64_t>(heads) * head_dim && stride % 8 == 0;
}

}  // namespace

extern "C" int memra_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                  int64_t v_stride, const float *q_weight, const float *k_weight, float eps,
                                  const int32_t *positions, const float *inv_freq, int32_t rotary_dim,
                                  int32_t interleaved, int32_t n_tok, int32_t n_heads, int32_t n_kv_heads,
                                  int32_t head_dim, void *q_out, int64_t q_out_stride, void *k_out,
                                  int64_t k_out_stride, const memra_kv_cache *cache, const int32_t *slot_mapping,
                                  void *stream) {
  if (n_tok < 0 || n_heads < 1 || n_kv_heads < 1 || rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 16)
    return MEMRA_ERR_INVALID_ARG;
  if (head_dim != 128 && head_dim != 256) return MEMRA_ERR_UNSUPPORTED;
  if (n_heads > 65535 || n_kv_heads > 65535) return MEMRA_ERR_UNSUPPORTED;
  if (!std::isfinite(eps) || eps < 0.f) return MEMRA_ERR_INVALID_ARG;
  if (cache) {
    const int st = check_cache(cache);
    if (st) return st;
    if (cache->head_dim != head_dim || cache->n_kv_heads != n_kv_heads) return MEMRA_ERR_INVALID_ARG;
  }
  if (n_tok == 0) return MEMRA_OK;
  if (!rows_ok(q, q_stride, n_heads, head_dim) || !rows_ok(q_out, q_out_stride, n_heads, head_dim))
    return MEMRA_ERR_INVALID_ARG;
  // keys come in exactly when they go somewhere, values and slots exactly when there is a cache
  if ((k != nullptr) != (k_out != nullptr || cache != nullptr) || (v != nullptr) != (cache != nullptr) ||
      (slot_mapping != nullptr) != (cache != nullptr) || !aligned4(slot_mapping))
    return MEMRA_ERR_INVALID_ARG;
  if ((k && !rows_ok(k, k_stride, n_kv_heads, head_dim)) || (v && !rows_ok(v, v_stride, n_kv_heads, head_dim)) ||
      (k_out && !rows_ok(k_out, k_out_stride, n_kv_heads, head_dim)))
    return MEMRA_ERR_INVALID_ARG;
  if (!aligned4(q_weight) || !aligned4(k_weight)) return MEMRA_ERR_INVALID_ARG;
  if (rotary_dim > 0 && (!positions || !inv_freq || !aligned4(positions) || !aligned4(inv_freq)))
    return MEMRA_ERR_INVALID_ARG;
  NormRopeParams p{};
  p.q = static_cast<const __half *>(q);
  p.k = static_cast<const __half *>(k);
  p.v = static_cast<const __half *>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.q_out = static_cast<__half *>(q_out);
  p.k_out = static_cast<__half *>(k_out);
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  p.slots = slot_mapping;
  if (cache) {
    p.cache = QuantTarget{static_cast<uint8_t *>(cache->k_pool), static_cast<uint8_t *>(cache->v_pool), n_kv_heads,
                          cache->k_fmt, cache->v_fmt, cache->k_scale, cache->v_scale};
    p.status = cache->status;
    p.num_pages = cache->num_pages;
  }
  p.eps = eps;
  p.tokens = n_tok;
  p.n_heads = n_heads;
  p.n_kv_heads = n_kv_heads;
  p.half = rotary_dim / 2;
  p.interleaved = interleaved != 0;
  return cuda_status(launch_norm_rope(head_dim, p, device_sms(), static_cast<cudaStream_t>(stream)));
}
