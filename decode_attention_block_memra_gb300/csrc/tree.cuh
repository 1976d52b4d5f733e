// Tree attention over the paged cache: the split plan, the parameters of its
// two kernels (the split pass and the merge) and their launchers.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "memra_device.cuh"

namespace memra {

// Keys of one step of the split pass (the N of the score MMA).
constexpr int kTreeKeys = 64;

// Row tiles (128 rows: nodes x the group's heads) of a CTA, one CTA to an SM: two
// past 128 rows at head_dim 128, so that a page is dequantized once for both (64
// nodes x 8 heads over 262,144 keys: 363 us when it was built, 438 with two CTAs of
// one tile; 370 now).
__host__ __device__ constexpr int tree_tiles(int D, int rows) { return D == 128 && rows > 128 ? 2 : 1; }

// The split plan.  A call's keys, in chunks of kTreeKeys, are cut so that one
// wave of the GPU (or as few whole waves as kTreeMaxChunks allows) holds all
// CTAs: C = ceil(chunks of all sequences / places) chunks each, and more
// (kTreeTrials times at most) while the sequences' rounded-up splits are more than
// the places (8 sequences of 4,104 keys at head_dim 256: 50 us with 160 splits on
// 152 SMs, 40 us with 144).
// C is at least kTreeMinChunks (the workspace's size goes by it) and at most
// kTreeMaxChunks: the tensor cores cut the float32 sums at every step, and over
// 13,824 keys in one split what was lost came to a quarter of the output's own
// rounding.  A sequence's splits are made equal.
// It depends on the lengths of all sequences of the call: a row's partial sums
// are grouped differently in another batch, and its last bits may differ.
constexpr int kTreeMinChunks = 4;
constexpr int kTreeMaxChunks = 120;
constexpr int kTreeTrials = 4;
constexpr int kTreeSplitPages = kTreeMaxChunks * kTreeKeys / kPage;
// Most splits of a sequence, unless kTreeMaxChunks makes more.
constexpr int kTreeMaxSplits = 160;

__host__ __device__ __forceinline__ int tree_ceil(int n, int c) { return n > 0 ? (n - 1) / c + 1 : 0; }

// Chunks of a split of a sequence of `chunks` chunks, C chunks wanted.
__host__ __device__ __forceinline__ int tree_split_chunks(int chunks, int C) {
  int c = C < tree_ceil(chunks, kTreeMaxSplits) ? tree_ceil(chunks, kTreeMaxSplits) : C;
  if (c > kTreeMaxChunks) c = kTreeMaxChunks;
  const int ns = tree_ceil(chunks, c);
  return ns > 1 ? tree_ceil(chunks, ns) : c;
}

// Most splits of any sequence of up to max_seq_len tokens, whatever the device and the call.
__host__ __device__ __forceinline__ int tree_max_splits(int max_seq_len) {
  const int chunks = tree_ceil(max_seq_len, kTreeKeys);
  const int by_min = tree_ceil(chunks, kTreeMinChunks), by_max = tree_ceil(chunks, kTreeMaxChunks);
  const int cap = by_max > kTreeMaxSplits ? by_max : kTreeMaxSplits;
  return by_min < cap ? by_min : cap;
}

struct TreeParams {
  const uint8_t *k_pool;
  const uint8_t *v_pool;
  const __half *q;              // [batch][n_nodes][n_heads][D]
  const int32_t *page_table;
  const int32_t *seq_lens;
  const uint64_t *mask;         // [batch][n_nodes]
  __half *out;
  float *o_part;                // [batch * n_nodes * n_heads][max_splits][D]
  float *lse_part;              // [batch * n_nodes * n_heads][max_splits]
  int32_t *plan;                // C, from the split pass to the merge
  int32_t *status;
  int batch, n_nodes, n_heads, group, n_kv_heads, num_pages, max_pages, max_seq_len;
  int len_limit;                // min(max_seq_len, tokens of a page table's row): lengths are clamped to it
  int slots;                    // CTAs of a wave per (KV head, rows of a CTA); 0: sequences are cut at kTreeMaxChunks only
  int max_splits;               // partials per row in the workspace
  int row_ctas;                 // CTAs over the rows of one KV head
  float scale_log2;             // |sm_scale| * (post-scale of the staged K values) * log2(e); 1 for sm_scale 0
  uint32_t q_and, q_xor;        // applied to the query's fp16 pairs: the scale's sign, or zeros for sm_scale 0
  float v_post;                 // post-scale of the staged V values
  int test_extra_tx;            // the test hook's: bytes that CTA 0 expects beyond its first chunk's (0 elsewhere)
};

cudaError_t launch_tree(int D, int kf, int vf, const TreeParams &p, cudaStream_t st);
cudaError_t launch_tree_merge(int D, const TreeParams &p, cudaStream_t st);

}  // namespace memra
