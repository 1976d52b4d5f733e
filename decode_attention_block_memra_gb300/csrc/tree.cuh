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

// CTAs of the split pass that share an SM.
__host__ __device__ constexpr int tree_ctas_per_sm(int D) { return D == 128 ? 2 : 1; }

// Smallest split: it keeps a CTA's fixed costs (the query tile, the first
// pages' latency, the output rows) to a fraction of its time.
constexpr int kTreeSplitTokens = 768;
// Largest split (its page ids lie in shared memory).
constexpr int kTreeSplitMax = 15360;
constexpr int kTreeSplitPages = kTreeSplitMax / kPage;
// Most splits that a sequence is cut into to fill the GPU.
constexpr int kTreeMaxSplits = 160;

// Split size of a sequence of T tokens: about `target` splits, never fewer
// than kTreeSplitTokens or more than kTreeSplitMax tokens, a multiple of 64.
// It depends on T and `target` (the device, the KV heads and the rows of one
// sequence) only: a sequence's bytes are the same alone or in any batch.
__host__ __device__ __forceinline__ int tree_split_tokens(int T, int target) {
  const int c = ((T > 0 ? (T - 1) / target + 1 : 0) + 63) / 64 * 64;
  return c < kTreeSplitTokens ? kTreeSplitTokens : (c > kTreeSplitMax ? kTreeSplitMax : c);
}

__host__ __device__ __forceinline__ int tree_ceil(int T, int c) { return T > 0 ? (T - 1) / c + 1 : 0; }

// Most splits of any sequence of up to T tokens: those of the smallest size,
// capped by the target, or past target * kTreeSplitMax tokens by the largest size.
__host__ __device__ __forceinline__ int tree_most_splits(int T, int target) {
  const int cap = tree_ceil(T, kTreeSplitMax) > target ? tree_ceil(T, kTreeSplitMax) : target;
  return tree_ceil(T, kTreeSplitTokens) < cap ? tree_ceil(T, kTreeSplitTokens) : cap;
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
  int32_t *status;
  int batch, n_nodes, n_heads, group, n_kv_heads, num_pages, max_pages, max_seq_len;
  int target;                   // splits that fill the GPU
  int max_splits;               // partials per row in the workspace
  int row_ctas;                 // 128-row tiles of one KV head
  float scale_log2;             // |sm_scale| * (post-scale of the staged K values) * log2(e); 1 for sm_scale 0
  uint32_t q_and, q_xor;        // applied to the query's fp16 pairs: the scale's sign, or zeros for sm_scale 0
  float v_post;                 // post-scale of the staged V values
};

cudaError_t launch_tree(int D, int kf, int vf, const TreeParams &p, cudaStream_t st);
cudaError_t launch_tree_merge(int D, const TreeParams &p, cudaStream_t st);

}  // namespace memra
