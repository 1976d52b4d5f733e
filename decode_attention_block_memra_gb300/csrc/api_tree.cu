// Entry points of tree attention in include/memra.h: argument validation, the plan, the launches; the test hook.
#include <algorithm>

#include "host_checks.cuh"
#include "memra_testing.h"
#include "tree.cuh"

using namespace memra;

namespace {

// The plan word (16 bytes), the partial rows, their log-sum-exp.
size_t tree_workspace(int64_t rows, int32_t head_dim, int32_t max_seq_len, size_t *lse_offset) {
  const int splits = tree_max_splits(max_seq_len);
  const size_t parts = splits > 1 ? static_cast<size_t>(rows) * splits : 0;
  const size_t o_bytes = parts * head_dim * sizeof(float);
  if (lse_offset) *lse_offset = 16 + o_bytes;
  return 16 + o_bytes + parts * sizeof(float);
}

// Every sequence fits one split, whatever the plan: no partials, no merge.
bool one_split(int32_t max_seq_len) { return tree_max_splits(max_seq_len) <= 1; }

}  // namespace

extern "C" {

size_t memra_tree_attn_workspace_bytes(int32_t batch, int32_t n_nodes, int32_t n_heads, int32_t head_dim,
                                       int32_t max_seq_len) {
  if (batch < 0 || n_nodes < 1 || n_nodes > MEMRA_MAX_TREE_NODES || n_heads < 1 ||
      (head_dim != 128 && head_dim != 256) || max_seq_len < 0)
    return 0;
  return tree_workspace(static_cast<int64_t>(batch) * n_nodes * n_heads, head_dim, max_seq_len, nullptr);
}

}  // extern "C"

namespace {

int tree_attn(const memra_kv_cache *cache, const void *q, const int32_t *page_table, int32_t max_pages_per_seq,
              const int32_t *seq_lens, int32_t max_seq_len, const uint64_t *tree_mask, int32_t batch, int32_t n_nodes,
              int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, float sm_scale, void *workspace,
              size_t workspace_bytes, void *out, void *stream, int test_extra_tx = 0) {
  int st = check_cache(cache);
  if (st) return st;
  if (batch < 0 || n_nodes < 1 || n_heads < 1 || max_seq_len < 0 || max_pages_per_seq < 1)
    return MEMRA_ERR_INVALID_ARG;
  if (n_kv_heads != cache->n_kv_heads || head_dim != cache->head_dim || n_heads % n_kv_heads)
    return MEMRA_ERR_INVALID_ARG;
  if (n_nodes > MEMRA_MAX_TREE_NODES || n_heads / n_kv_heads > MEMRA_MAX_GROUP || n_kv_heads > 65535)
    return MEMRA_ERR_UNSUPPORTED;
  if (!std::isfinite(sm_scale)) return MEMRA_ERR_INVALID_ARG;
  const int group = n_heads / n_kv_heads, rows = n_nodes * group;
  const int tiles = tree_tiles(head_dim, rows);
  const int row_ctas = static_cast<int>(ceil_div(rows, 128 * tiles));
  const int64_t all_rows = static_cast<int64_t>(batch) * n_nodes * n_heads;
  if (static_cast<int64_t>(n_kv_heads) * row_ctas > 65535 || batch > 65535 || all_rows > INT32_MAX)
    return MEMRA_ERR_UNSUPPORTED;
  if (batch == 0) return MEMRA_OK;
  if (!q || !page_table || !seq_lens || !tree_mask || !out || !aligned16(q) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(page_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(tree_mask) & 7u))
    return MEMRA_ERR_INVALID_ARG;
  const size_t need = memra_tree_attn_workspace_bytes(batch, n_nodes, n_heads, head_dim, max_seq_len);
  if (workspace_bytes < need) return MEMRA_ERR_WORKSPACE;
  if (!workspace || !aligned16(workspace)) return MEMRA_ERR_INVALID_ARG;
  size_t lse = 0;
  tree_workspace(all_rows, head_dim, max_seq_len, &lse);
  TreeParams p;
  p.k_pool = static_cast<const uint8_t *>(cache->k_pool);
  p.v_pool = static_cast<const uint8_t *>(cache->v_pool);
  p.q = static_cast<const __half *>(q);
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.mask = tree_mask;
  p.out = static_cast<__half *>(out);
  p.plan = static_cast<int32_t *>(workspace);
  p.o_part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + 16);
  p.lse_part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + lse);
  p.status = cache->status;
  p.batch = batch;
  p.n_nodes = n_nodes;
  p.n_heads = n_heads;
  p.group = group;
  p.n_kv_heads = n_kv_heads;
  p.num_pages = cache->num_pages;
  p.max_pages = max_pages_per_seq;
  p.max_seq_len = max_seq_len;
  // (positions up to a chunk past the end stay below 2^31)
  p.len_limit = static_cast<int32_t>(std::min<int64_t>(
      std::min<int64_t>(max_seq_len, INT32_MAX - kTreeKeys), static_cast<int64_t>(max_pages_per_seq) * kPage));
  // Where the sequences alone fill the GPU four times over, none is cut for its sake (and no CTA adds
  // up the lengths of so many, nor of more chunks than 32 bits count).
  p.slots = std::max(1, device_sms() / (n_kv_heads * row_ctas));
  if (batch >= 4 * p.slots || one_split(max_seq_len) ||
      static_cast<int64_t>(batch) * tree_ceil(max_seq_len, kTreeKeys) > INT32_MAX)
    p.slots = 0;
  p.max_splits = tree_max_splits(max_seq_len);
  p.row_ctas = row_ctas;
  // staged values: q8_0 / q5_1 / q4_0 at half size, fp8 / NVFP4 without their tensor scale
  p.scale_log2 = std::fabs(sm_scale) * (cache->k_fmt == MEMRA_KV_Q8_0 ? 2.f : cache->k_scale) * 1.4426950408889634f;
  p.q_and = p.scale_log2 == 0.f ? 0u : 0xFFFFFFFFu;
  p.q_xor = sm_scale < 0.f ? 0x80008000u : 0u;
  if (p.scale_log2 == 0.f) p.scale_log2 = 1.f;
  p.v_post = scaled_format(cache->v_fmt) ? cache->v_scale : 2.f;
  p.test_extra_tx = test_extra_tx;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = cuda_status(launch_tree(head_dim, cache->k_fmt, cache->v_fmt, p, s));
  if (st || one_split(max_seq_len)) return st;
  return cuda_status(launch_tree_merge(head_dim, p, s));
}

}  // namespace

extern "C" int memra_tree_attn(const memra_kv_cache *cache, const void *q, const int32_t *page_table,
                               int32_t max_pages_per_seq, const int32_t *seq_lens, int32_t max_seq_len,
                               const uint64_t *tree_mask, int32_t batch, int32_t n_nodes, int32_t n_heads,
                               int32_t n_kv_heads, int32_t head_dim, float sm_scale, void *workspace,
                               size_t workspace_bytes, void *out, void *stream) {
  return tree_attn(cache, q, page_table, max_pages_per_seq, seq_lens, max_seq_len, tree_mask, batch, n_nodes, n_heads,
                   n_kv_heads, head_dim, sm_scale, workspace, workspace_bytes, out, stream);
}

// memra_testing.h: the same call with a first chunk whose wait cannot complete.
extern "C" int memra_testing_tree_attn_short_page(const memra_kv_cache *cache, const void *q, const int32_t *page_table,
                                                  int32_t max_pages_per_seq, const int32_t *seq_lens,
                                                  int32_t max_seq_len, const uint64_t *tree_mask, int32_t batch,
                                                  int32_t n_nodes, int32_t n_heads, int32_t n_kv_heads,
                                                  int32_t head_dim, float sm_scale, void *workspace,
                                                  size_t workspace_bytes, void *out, void *stream) {
  return tree_attn(cache, q, page_table, max_pages_per_seq, seq_lens, max_seq_len, tree_mask, batch, n_nodes, n_heads,
                   n_kv_heads, head_dim, sm_scale, workspace, workspace_bytes, out, stream, 16);
}
