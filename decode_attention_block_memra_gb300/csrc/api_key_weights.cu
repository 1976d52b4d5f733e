// Entry point of the key weights in include/memra.h: argument validation and the launch; the test hook.
#include <algorithm>

#include "host_checks.cuh"
#include "key_weights.cuh"
#include "memra_testing.h"

using namespace memra;

namespace {

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int key_weights(const memra_kv_cache *cache, const void *q, int64_t q_stride, const float *lse,
                const int32_t *cu_seqlens, const int32_t *page_table, int32_t max_pages_per_seq,
                const int32_t *seq_lens, int32_t max_seq_len, int32_t batch, int32_t total_tokens, int32_t n_heads,
                int32_t n_kv_heads, int32_t head_dim, float sm_scale, float keep, float *weights,
                int64_t weight_stride, void *stream, int test_extra_tx = 0) {
  const int st = check_cache(cache);
  if (st) return st;
  if (batch < 0 || total_tokens < 0 || n_heads < 1 || max_seq_len < 0 || max_pages_per_seq < 1 ||
      weight_stride < max_seq_len)
    return MEMRA_ERR_INVALID_ARG;
  if (n_kv_heads != cache->n_kv_heads || head_dim != cache->head_dim || n_heads % n_kv_heads)
    return MEMRA_ERR_INVALID_ARG;
  if (n_heads / n_kv_heads > MEMRA_MAX_GROUP || n_kv_heads > 65535 || batch > 65535) return MEMRA_ERR_UNSUPPORTED;
  if (!std::isfinite(sm_scale) || !(sm_scale > 0.f) || !std::isfinite(keep)) return MEMRA_ERR_INVALID_ARG;
  if (q_stride < static_cast<int64_t>(n_heads) * head_dim || q_stride % 8) return MEMRA_ERR_INVALID_ARG;
  if (q_stride >= (1ll << 38)) return MEMRA_ERR_UNSUPPORTED;       // what the tensor copies take
  if (batch == 0 || total_tokens == 0) return MEMRA_OK;
  // (without a key there is no weight: null will do)
  if (!q || !lse || !cu_seqlens || !page_table || !seq_lens || (!weights && max_seq_len > 0) || !aligned16(q) || !aligned4(lse) ||
      !aligned4(cu_seqlens) || !aligned4(page_table) || !aligned4(seq_lens) || !aligned4(weights))
    return MEMRA_ERR_INVALID_ARG;
  WeightParams p;
  p.k_pool = static_cast<const uint8_t *>(cache->k_pool);
  p.q = static_cast<const __half *>(q);
  p.q_stride = q_stride;
  p.lse = lse;
  p.cu_seqlens = cu_seqlens;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.weights = weights;
  p.weight_stride = weight_stride;
  p.status = cache->status;
  p.keep = keep;
  // staged values: q8_0 at half size, fp8 / NVFP4 without their tensor scale
  p.scale_log2 = sm_scale * (cache->k_fmt == MEMRA_KV_Q8_0 ? 2.f : cache->k_scale) * 1.4426950408889634f;
  p.batch = batch;
  p.total = total_tokens;
  p.n_heads = n_heads;
  p.group = n_heads / n_kv_heads;
  p.n_kv_heads = n_kv_heads;
  p.num_pages = cache->num_pages;
  p.max_pages = max_pages_per_seq;
  // (positions up to a tile past the end stay below 2^31)
  p.len_limit = static_cast<int32_t>(std::min<int64_t>(std::min<int64_t>(max_seq_len, INT32_MAX - 4 * kWeightKeys),
                                                       static_cast<int64_t>(max_pages_per_seq) * kPage));
  const int64_t all_rows = static_cast<int64_t>(total_tokens) * p.group;
  // (small row tiles by the rows of a sequence on average: what that costs and gains stands in key_weights.cu)
  const int rows = all_rows <= static_cast<int64_t>(batch) * kWeightRowsFew ? kWeightRowsFew : weight_rows(head_dim);
  p.hpt = std::min(p.group, rows);
  p.subs = static_cast<int>(ceil_div(p.group, p.hpt));
  p.tpt = std::max(1, rows / p.group);
  p.ctas = device_sms();
  p.test_extra_tx = test_extra_tx;
  return cuda_status(launch_key_weights(head_dim, rows, cache->k_fmt, p, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int memra_key_weights(const memra_kv_cache *cache, const void *q, int64_t q_stride, const float *lse,
                      const int32_t *cu_seqlens, const int32_t *page_table, int32_t max_pages_per_seq,
                      const int32_t *seq_lens, int32_t max_seq_len, int32_t batch, int32_t total_tokens,
                      int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, float sm_scale, float keep,
                      float *weights, int64_t weight_stride, void *stream) {
  return key_weights(cache, q, q_stride, lse, cu_seqlens, page_table, max_pages_per_seq, seq_lens, max_seq_len, batch,
                     total_tokens, n_heads, n_kv_heads, head_dim, sm_scale, keep, weights, weight_stride, stream);
}

// memra_testing.h: the same call with a first raw chunk whose wait cannot complete.
int memra_testing_key_weights_short_page(const memra_kv_cache *cache, const void *q, int64_t q_stride,
                                         const float *lse, const int32_t *cu_seqlens, const int32_t *page_table,
                                         int32_t max_pages_per_seq, const int32_t *seq_lens, int32_t max_seq_len,
                                         int32_t batch, int32_t total_tokens, int32_t n_heads, int32_t n_kv_heads,
                                         int32_t head_dim, float sm_scale, float keep, float *weights,
                                         int64_t weight_stride, void *stream) {
  return key_weights(cache, q, q_stride, lse, cu_seqlens, page_table, max_pages_per_seq, seq_lens, max_seq_len, batch,
                     total_tokens, n_heads, n_kv_heads, head_dim, sm_scale, keep, weights, weight_stride, stream, 16);
}

}  // extern "C"
