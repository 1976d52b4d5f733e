// Parameters and launcher of the kernel that makes query and key rows ready (norm_rope.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv_quant.cuh"

namespace memra {

struct NormRopeParams {
  const __half *q, *k, *v;        // token t's heads at + t * stride; k and v null where the call has none
  int64_t q_stride, k_stride, v_stride;
  const float *q_weight, *k_weight;       // [D], null: no norm
  const int32_t *positions;       // [tokens]
  const float *inv_freq;          // [half]
  __half *q_out, *k_out;          // k_out null: keys go to the cache only
  int64_t q_out_stride, k_out_stride;
  const int32_t *slots;           // [tokens], null: nothing is stored
  QuantTarget cache;
  int32_t *status;
  float eps;
  int tokens, n_heads, n_kv_heads, num_pages;
  int half;                       // rotated pairs: rotary_dim / 2
  int interleaved;
  // set by the launcher: row groups of a token by kind; units of a token, and row groups of one of its queries' and of one of its keys' or values'; units in all
  int k_passes, v_passes, q_passes, parts, q_share, kv_share;
  int64_t units;
};

cudaError_t launch_norm_rope(int D, NormRopeParams p, int sms, cudaStream_t st);

}  // namespace memra
