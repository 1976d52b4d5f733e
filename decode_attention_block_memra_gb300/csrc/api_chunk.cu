// Entry points of chunk attention in include/memra.h: argument validation, the launches; the test hook.
#include <algorithm>

#include "chunk.cuh"
#include "host_checks.cuh"
#include "memra_testing.h"

using namespace memra;

namespace {

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int chunk_ctas() { return std::min(device_sms(), kChunkCtasMax); }

// Float32 rows: two partial blocks of each CTA and what earlier sums of its block came to; the partials' log-sum-exp;
// what the merge joins.
struct Workspace {
  size_t lse, far, merges, bytes;
  Workspace(int head_dim) {
    const size_t rows = static_cast<size_t>(kChunkCtasMax) * chunk_tiles(head_dim) * kChunkRows;
    lse = 2 * rows * head_dim * sizeof(float);
    far = lse + 2 * rows * sizeof(float);
    merges = far + rows * kChunkFarCols(head_dim) * sizeof(float);
    bytes = merges + kChunkCtasMax * sizeof(int4);
  }
};

int chunk_attn(const memra_kv_cache *cache, const void *q, int64_t q_stride, const int32_t *cu_seqlens,
               const int32_t *page_table, int32_t max_pages_per_seq, const int32_t *seq_lens, int32_t max_seq_len,
               int32_t batch, int32_t total_tokens, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
               float sm_scale, int32_t window, void *workspace, size_t workspace_bytes, void *out, float *lse,
               void *stream, int test_extra_tx = 0) {
  int st = check_cache(cache);
  if (st) return st;
  if (batch < 0 || total_tokens < 0 || n_heads < 1 || max_seq_len < 0 || max_pages_per_seq < 1 || window < 0)
    return MEMRA_ERR_INVALID_ARG;
  if (n_kv_heads != cache->n_kv_heads || head_dim != cache->head_dim || n_heads % n_kv_heads)
    return MEMRA_ERR_INVALID_ARG;
  if (n_heads / n_kv_heads > MEMRA_MAX_GROUP || n_kv_heads > 65535 || batch > 65535) return MEMRA_ERR_UNSUPPORTED;
  if (!std::isfinite(sm_scale) || !(sm_scale > 0.f)) return MEMRA_ERR_INVALID_ARG;
  if (q_stride < static_cast<int64_t>(n_heads) * head_dim || q_stride % 8) return MEMRA_ERR_INVALID_ARG;
  if (batch == 0 || total_tokens == 0) return MEMRA_OK;
  if (!q || !cu_seqlens || !page_table || !seq_lens || !out || !aligned16(q) || !aligned16(out) ||
      !aligned4(cu_seqlens) || !aligned4(page_table) || !aligned4(seq_lens) || !aligned4(lse))
    return MEMRA_ERR_INVALID_ARG;
  const Workspace ws(head_dim);
  if (workspace_bytes < ws.bytes) return MEMRA_ERR_WORKSPACE;
  if (!workspace || !aligned16(workspace)) return MEMRA_ERR_INVALID_ARG;
  ChunkParams p;
  p.k_pool = static_cast<const uint8_t *>(cache->k_pool);
  p.v_pool = static_cast<const uint8_t *>(cache->v_pool);
  p.q = static_cast<const __half *>(q);
  p.q_stride = q_stride;
  p.cu_seqlens = cu_seqlens;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.out = static_cast<__half *>(out);
  p.lse = lse;
  uint8_t *const w = static_cast<uint8_t *>(workspace);
  p.o_part = reinterpret_cast<float *>(w);
  p.lse_part = reinterpret_cast<float *>(w + ws.lse);
  p.far = reinterpret_cast<float *>(w + ws.far);
  p.merges = reinterpret_cast<int4 *>(w + ws.merges);
  p.status = cache->status;
  p.batch = batch;
  p.total = total_tokens;
  p.n_heads = n_heads;
  p.group = n_heads / n_kv_heads;
  p.n_kv_heads = n_kv_heads;
  p.num_pages = cache->num_pages;
  p.max_pages = max_pages_per_seq;
  p.window = window;
  // (positions up to a step past the end stay below 2^31)
  int64_t limit = std::min<int64_t>(max_seq_len, INT32_MAX - 4 * kChunkKeys);
  if (window == 0) limit = std::min(limit, static_cast<int64_t>(max_pages_per_seq) * kPage);
  p.len_limit = static_cast<int32_t>(limit);
  p.tpt = kChunkRows / p.group;
  p.ctas = chunk_ctas();
  // staged values: q8_0 / q5_1 / q4_0 at half size, fp8 / NVFP4 without their tensor scale
  p.scale_log2 = sm_scale * (cache->k_fmt == MEMRA_KV_Q8_0 ? 2.f : cache->k_scale) * 1.4426950408889634f;
  p.v_post = scaled_format(cache->v_fmt) ? cache->v_scale : 2.f;
  p.test_extra_tx = test_extra_tx;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = cuda_status(launch_chunk(head_dim, cache->k_fmt, cache->v_fmt, p, s));
  // Blocks of fewer steps than this are never cut: no merge.
  if (st || max_seq_len <= (2 * kChunkSnap - 1) * kChunkKeys) return st;
  return cuda_status(launch_chunk_merge(head_dim, p, s));
}

}  // namespace

extern "C" {

size_t memra_chunk_attn_workspace_bytes(int32_t head_dim) {
  return head_dim == 128 || head_dim == 256 ? Workspace(head_dim).bytes : 0;
}

int memra_chunk_attn(const memra_kv_cache *cache, const void *q, int64_t q_stride, const int32_t *cu_seqlens,
                     const int32_t *page_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
                     int32_t max_seq_len, int32_t batch, int32_t total_tokens, int32_t n_heads, int32_t n_kv_heads,
                     int32_t head_dim, float sm_scale, int32_t window, void *workspace, size_t workspace_bytes,
                     void *out, float *lse, void *stream) {
  return chunk_attn(cache, q, q_stride, cu_seqlens, page_table, max_pages_per_seq, seq_lens, max_seq_len, batch,
                    total_tokens, n_heads, n_kv_heads, head_dim, sm_scale, window, workspace, workspace_bytes, out, lse,
                    stream);
}

// memra_testing.h: the same call with a first chunk whose wait cannot complete.
int memra_testing_chunk_attn_short_page(const memra_kv_cache *cache, const void *q, int64_t q_stride,
                                        const int32_t *cu_seqlens, const int32_t *page_table,
                                        int32_t max_pages_per_seq, const int32_t *seq_lens, int32_t max_seq_len,
                                        int32_t batch, int32_t total_tokens, int32_t n_heads, int32_t n_kv_heads,
                                        int32_t head_dim, float sm_scale, int32_t window, void *workspace,
                                        size_t workspace_bytes, void *out, float *lse, void *stream) {
  return chunk_attn(cache, q, q_stride, cu_seqlens, page_table, max_pages_per_seq, seq_lens, max_seq_len, batch,
                    total_tokens, n_heads, n_kv_heads, head_dim, sm_scale, window, workspace, workspace_bytes, out, lse,
                    stream, 16);
}

}  // extern "C"
