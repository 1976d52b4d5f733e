// Host-side argument checks shared by the entry points.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "memra_device.cuh"

namespace memra {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool k_format_ok(int f) { return f == MEMRA_KV_Q8_0 || f == MEMRA_KV_FP8_E4M3 || f == MEMRA_KV_NVFP4; }
inline bool v_format_ok(int f) {
  return f == MEMRA_KV_Q5_1 || f == MEMRA_KV_Q4_0 || f == MEMRA_KV_FP8_E4M3 || f == MEMRA_KV_NVFP4;
}
// formats with a float32 per-tensor scale
inline bool scaled_format(int f) { return f == MEMRA_KV_FP8_E4M3 || f == MEMRA_KV_NVFP4; }

inline int check_cache(const memra_kv_cache *c) {
  if (!c) return MEMRA_ERR_INVALID_ARG;
  if (!k_format_ok(c->k_fmt) || !v_format_ok(c->v_fmt)) return MEMRA_ERR_UNSUPPORTED;
  if (c->page_size != MEMRA_PAGE_SIZE) return MEMRA_ERR_UNSUPPORTED;
  if (c->head_dim != 128 && c->head_dim != 256) return MEMRA_ERR_UNSUPPORTED;
  if (c->n_kv_heads < 1 || c->num_pages < 1) return MEMRA_ERR_INVALID_ARG;
  if (!c->k_pool || !c->v_pool || !aligned16(c->k_pool) || !aligned16(c->v_pool)) return MEMRA_ERR_INVALID_ARG;
  if (c->status && (reinterpret_cast<uintptr_t>(c->status) & 3u)) return MEMRA_ERR_INVALID_ARG;
  if (scaled_format(c->k_fmt) && !(std::isfinite(c->k_scale) && c->k_scale > 0.f)) return MEMRA_ERR_INVALID_ARG;
  if (scaled_format(c->v_fmt) && !(std::isfinite(c->v_scale) && c->v_scale > 0.f)) return MEMRA_ERR_INVALID_ARG;
  // pools larger than 2^31 segments per head are fine (size_t offsets)
  return MEMRA_OK;
}

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? MEMRA_OK : MEMRA_ERR_CUDA; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Streaming multiprocessors of the current device (queried once per device).
inline int device_sms() {
  static int cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  if (!cached[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 1;
    cached[dev] = n;
  }
  return cached[dev];
}

}  // namespace memra
