// Entry point of the eviction in include/memra.h: argument validation and launches.
#include <algorithm>

#include "evict.cuh"
#include "host_checks.cuh"

using namespace memra;

namespace {
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
}  // namespace

extern "C" int memra_kv_evict(const memra_kv_cache *cache, const int32_t *page_table, int32_t max_pages_per_seq,
                              const int32_t *seq_lens, int32_t max_seq_len, const float *weights,
                              int64_t weight_stride, const int32_t *budgets, int32_t max_budget, int32_t sink,
                              int32_t recent, const int32_t *dst_table, int32_t dst_pages_per_seq, int32_t batch,
                              int32_t *kept, float *new_weights, int64_t new_weight_stride, int32_t *new_lens,
                              void *stream) {
  int st = check_cache(cache);
  if (st) return st;
  if (batch < 0 || max_pages_per_seq < 1 || max_seq_len < 0 || max_budget < 0 || sink < 0 || recent < 0 ||
      dst_pages_per_seq < 0 || weight_stride < max_seq_len ||
      static_cast<int64_t>(dst_pages_per_seq) * kPage < max_budget || (new_weights && new_weight_stride < max_budget))
    return MEMRA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(batch) * cache->n_kv_heads > 65535) return MEMRA_ERR_UNSUPPORTED;
  if (max_budget > INT32_MAX - 65536) return MEMRA_ERR_UNSUPPORTED;        // rows up to some pages behind the last stay below 2^31
  if (batch == 0 || max_budget == 0) return MEMRA_OK;
  // (without a token there is no weight: null will do)
  if (!page_table || !seq_lens || (!weights && max_seq_len > 0) || !budgets || !dst_table || !kept || !aligned4(page_table) ||
      !aligned4(seq_lens) || !aligned4(weights) || !aligned4(budgets) || !aligned4(dst_table) || !aligned4(kept) ||
      !aligned4(new_weights) || !aligned4(new_lens) || (weights && weights == new_weights))
    return MEMRA_ERR_INVALID_ARG;
  EvictParams p;
  p.k_pool = static_cast<uint8_t *>(cache->k_pool);
  p.v_pool = static_cast<uint8_t *>(cache->v_pool);
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.weights = weights;
  p.budgets = budgets;
  p.dst_table = dst_table;
  p.kept = kept;
  p.new_weights = new_weights;
  p.new_lens = new_lens;
  p.status = cache->status;
  p.weight_stride = weight_stride;
  p.new_stride = new_weight_stride;
  p.batch = batch;
  p.n_kv_heads = cache->n_kv_heads;
  p.num_pages = cache->num_pages;
  p.max_pages = max_pages_per_seq;
  p.max_seq_len = max_seq_len;
  p.dst_pages = dst_pages_per_seq;
  p.max_budget = max_budget;
  p.sink = sink;
  p.recent = recent;
  p.len_limit = static_cast<int32_t>(std::min<int64_t>(std::min<int64_t>(max_seq_len, INT32_MAX - 65536),
                                                       static_cast<int64_t>(max_pages_per_seq) * kPage));
  p.k_fmt = cache->k_fmt;
  p.v_fmt = cache->v_fmt;
  p.k_seg = k_seg_bytes(cache->k_fmt, cache->head_dim);
  p.v_seg = v_seg_bytes(cache->v_fmt, cache->head_dim);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = cuda_status(launch_evict_select(p, device_sms(), s));
  if (st) return st;
  return cuda_status(launch_evict_move(cache->head_dim, p, device_sms(), s));
}
