// Key weights: how the work is cut, the parameters of the kernel and its launcher.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "memra_device.cuh"

namespace memra {

constexpr int kWeightKeys = 128;           // keys of a tile (the M of the MMA)
// Query rows of a tile (its N): what shared memory holds of them; and where the sequences have few rows on
// average, so that more raw pages can be in flight instead.
__host__ __device__ constexpr int weight_rows(int D) { return D == 128 ? 128 : 64; }
constexpr int kWeightRowsFew = 32;

struct WeightParams {
  const uint8_t *k_pool;
  const __half *q;              // token t's heads at q + t * q_stride
  int64_t q_stride;
  const float *lse;             // [total][n_heads]
  const int32_t *cu_seqlens;    // [batch + 1]
  const int32_t *page_table;    // [batch][max_pages]
  const int32_t *seq_lens;
  float *weights;               // [batch][n_kv_heads][weight_stride]
  int64_t weight_stride;
  int32_t *status;
  float keep, scale_log2;       // sm_scale * (post-scale of the staged K values) * log2(e)
  int batch, total, n_heads, group, n_kv_heads, num_pages, max_pages;
  int len_limit;                // lengths are clamped to it
  int hpt, subs, tpt;           // heads of a row tile, row tiles that a token's heads take, tokens of a row tile
  int ctas;
  int test_extra_tx;            // the test hook's: bytes that CTA 0 expects beyond its first raw chunk's (0 elsewhere)
};

// `rows`: query rows of a tile, weight_rows(D) or kWeightRowsFew
cudaError_t launch_key_weights(int D, int rows, int kf, const WeightParams &p, cudaStream_t st);

}  // namespace memra
