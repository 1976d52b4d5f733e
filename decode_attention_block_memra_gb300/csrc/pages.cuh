// Parameters and launchers of the page-upkeep kernels (pages.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "memra_device.cuh"

namespace memra {

struct CopyPagesParams {
  uint4 *k_pool;
  uint4 *v_pool;
  const int32_t *src;
  const int32_t *dst;
  int32_t *status;
  int n, num_pages;
  uint32_t k_units, v_units;      // 16-byte units of a page in each pool
  uint32_t runs;                  // CTAs' worth of units per page, set by the launcher
};

struct CompactParams {
  uint8_t *k_pool;
  uint8_t *v_pool;
  const int32_t *page_table;
  const int32_t *seq_lens;
  const int32_t *accepted;
  const int32_t *n_accepted;
  int32_t *status;
  int n_kv_heads, num_pages, max_pages, max_seq_len, n_nodes, max_accepted;
  int k_fmt, v_fmt, k_seg, v_seg;
  int parts;                      // CTAs over the bytes of a row, set by the launcher
};

cudaError_t launch_copy_pages(CopyPagesParams p, cudaStream_t st);
cudaError_t launch_compact(int D, CompactParams p, int batch, cudaStream_t st);

}  // namespace memra
