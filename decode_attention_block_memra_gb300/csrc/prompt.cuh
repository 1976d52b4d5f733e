// Parameters and launcher of the prompt-attention kernel (prompt.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "memra_device.cuh"

namespace memra {

struct PromptParams {
  const __half *q, *k, *v;
  const int32_t *cu_seqlens;      // [batch + 1]
  __half *out;                    // [total][n_heads][D]
  int32_t *status;
  int64_t q_stride, k_stride, v_stride;   // elements from one token to the next
  int batch, total, n_heads, n_kv_heads, group, window;
  int tpt;                        // tokens per 128-row tile: 128 / group
  float scale_log2;               // sm_scale * log2(e)
  int test_extra_tx;              // the test hook's: bytes that CTA 0 expects beyond its first copy of K (0 elsewhere)
};

cudaError_t launch_prompt(int D, const PromptParams &p, cudaStream_t st);

}  // namespace memra
