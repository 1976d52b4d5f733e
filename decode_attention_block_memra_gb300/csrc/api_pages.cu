// Entry points of the page upkeep in include/memra.h: argument validation and launches.
#include "host_checks.cuh"
#include "pages.cuh"

using namespace memra;

namespace {
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
}  // namespace

extern "C" {

int memra_kv_copy_pages(const memra_kv_cache *cache, const int32_t *src_pages, const int32_t *dst_pages, int32_t n,
                        void *stream) {
  const int st = check_cache(cache);
  if (st) return st;
  if (n < 0) return MEMRA_ERR_INVALID_ARG;
  if (n == 0) return MEMRA_OK;
  if (!src_pages || !dst_pages || !aligned4(src_pages) || !aligned4(dst_pages)) return MEMRA_ERR_INVALID_ARG;
  CopyPagesParams p;
  p.k_pool = static_cast<uint4 *>(cache->k_pool);
  p.v_pool = static_cast<uint4 *>(cache->v_pool);
  p.src = src_pages;
  p.dst = dst_pages;
  p.status = cache->status;
  p.n = n;
  p.num_pages = cache->num_pages;
  const int64_t ku = static_cast<int64_t>(k_seg_bytes(cache->k_fmt, cache->head_dim)) / 16 * cache->n_kv_heads;
  const int64_t vu = static_cast<int64_t>(v_seg_bytes(cache->v_fmt, cache->head_dim)) / 16 * cache->n_kv_heads;
  if (ku + vu > INT32_MAX / 2) return MEMRA_ERR_UNSUPPORTED;
  p.k_units = static_cast<uint32_t>(ku);
  p.v_units = static_cast<uint32_t>(vu);
  p.runs = 0;
  return cuda_status(launch_copy_pages(p, static_cast<cudaStream_t>(stream)));
}

int memra_kv_compact(const memra_kv_cache *cache, const int32_t *page_table, int32_t max_pages_per_seq,
                     const int32_t *seq_lens, int32_t max_seq_len, const int32_t *accepted, int32_t max_accepted,
                     const int32_t *n_accepted, int32_t batch, int32_t n_nodes, void *stream) {
  const int st = check_cache(cache);
  if (st) return st;
  if (batch < 0 || n_nodes < 1 || max_accepted < 0 || max_pages_per_seq < 1 || max_seq_len < 0)
    return MEMRA_ERR_INVALID_ARG;
  if (n_nodes > MEMRA_MAX_TREE_NODES || batch > 65535 || cache->n_kv_heads > 65535) return MEMRA_ERR_UNSUPPORTED;
  if (max_accepted > n_nodes) return MEMRA_ERR_INVALID_ARG;
  if (batch == 0 || max_accepted == 0) return MEMRA_OK;
  if (!page_table || !seq_lens || !accepted || !n_accepted || !aligned4(page_table) || !aligned4(seq_lens) ||
      !aligned4(accepted) || !aligned4(n_accepted))
    return MEMRA_ERR_INVALID_ARG;
  CompactParams p;
  p.k_pool = static_cast<uint8_t *>(cache->k_pool);
  p.v_pool = static_cast<uint8_t *>(cache->v_pool);
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.accepted = accepted;
  p.n_accepted = n_accepted;
  p.status = cache->status;
  p.n_kv_heads = cache->n_kv_heads;
  p.num_pages = cache->num_pages;
  p.max_pages = max_pages_per_seq;
  p.max_seq_len = max_seq_len;
  p.n_nodes = n_nodes;
  p.max_accepted = max_accepted;
  p.k_fmt = cache->k_fmt;
  p.v_fmt = cache->v_fmt;
  p.k_seg = k_seg_bytes(cache->k_fmt, cache->head_dim);
  p.v_seg = v_seg_bytes(cache->v_fmt, cache->head_dim);
  p.parts = 0;
  return cuda_status(launch_compact(cache->head_dim, p, batch, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
