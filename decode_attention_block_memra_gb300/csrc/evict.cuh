// Parameters and launchers of the eviction kernels (evict.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "memra_device.cuh"

namespace memra {

struct EvictParams {
  uint8_t *k_pool;
  uint8_t *v_pool;
  const int32_t *page_table;      // [batch][max_pages]
  const int32_t *seq_lens;
  const float *weights;           // [batch][n_kv_heads][weight_stride]
  const int32_t *budgets;
  const int32_t *dst_table;       // [batch][dst_pages]
  int32_t *kept;                  // [batch][n_kv_heads][max_budget]
  float *new_weights;             // [batch][n_kv_heads][new_stride], or null
  int32_t *new_lens;              // [batch], or null
  int32_t *status;
  int64_t weight_stride, new_stride;
  int batch, n_kv_heads, num_pages, max_pages, max_seq_len, dst_pages, max_budget, sink, recent;
  int len_limit;                  // min(max_seq_len, tokens of a page table's row): lengths are clamped to it
  int k_fmt, v_fmt, k_seg, v_seg;
};

cudaError_t launch_evict_select(const EvictParams &p, int sms, cudaStream_t st);
cudaError_t launch_evict_move(int D, const EvictParams &p, int sms, cudaStream_t st);

}  // namespace memra
