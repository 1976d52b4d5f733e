// Shared-memory accesses and fp16 pieces of the kernels that feed the
// fifth-generation tensor cores; and, for the prefix passes of cascade.cu, the
// staging of quantized pages: raw K and V words of a page segment in shared
// memory to fp16 operand values (hi, and for the block-scaled integer formats the
// low part of an exact pair).  The tree kernel stages whole runs of codes and has
// its own.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "memra_device.cuh"

namespace memra {

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// One thread: copy `bytes` (a multiple of 16, both addresses 16-byte aligned)
// from shared to global memory through the async proxy, as one bulk
// async-group of this thread.
__device__ __forceinline__ void bulk_store_s2g(void *dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// One thread: its bulk stores have completed, writes performed (before the
// CTA, and its shared memory, goes away).
__device__ __forceinline__ void bulk_store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

// fp16 of the low e4m3 byte of `byte`, broadcast to both halves.
__device__ __forceinline__ __half2 e4m3_scale_h2(uint32_t byte) {
  const uint32_t h = e4m3x2_to_half2(byte & 0xFFu) & 0xFFFFu;
  return bits_h2(h | (h << 16));
}

// Raw shared-memory words of one K staging item (token t of a staged page,
// dims 8u .. 8u + 7): the 8 code bytes (NVFP4: the 8-byte group holding the
// item's 16 nibbles) and the block-scale bits.  Layout formulas of memra.h.
struct KRaw {
  uint2 w;
  uint32_t s;
};

template <int D, int KF>
__device__ __forceinline__ KRaw load_k8(uint32_t seg, int t, int u) {
  constexpr int NB = D / 32;
  const int b = u >> 2, c = u & 3;
  const uint32_t lane = 4 * (t & 7) + c;
  KRaw r;
  if constexpr (KF == MEMRA_KV_NVFP4) {
    r.w = lds64(seg + ((b >> 1) * 32 + lane) * 16 + (b & 1) * 8);
    r.s = lds8(seg + 8 * D + t * (D / 16) + (u >> 1));
  } else {
    r.w = lds64(seg + (((t >> 3) * (NB / 2) + (b >> 1)) * 32 + lane) * 16 + (b & 1) * 8);
    r.s = KF == MEMRA_KV_Q8_0 ? lds16(seg + 16 * D + (t * NB + b) * 2) : 0u;
  }
  return r;
}

// The item's 8 values as fp16 (hi) plus, for q8_0, the low parts (lo).
template <int KF>
__device__ __forceinline__ void convert_k8(const KRaw &r, int t, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  if constexpr (KF == MEMRA_KV_Q8_0) {
    const __half2 d2 = bits_h2(r.s | (r.s << 16));
    const __half2 half = __float2half2_rn(0.5f), off = __float2half2_rn(-576.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // codes are stored as q + 128: splice under 1024 -> 1152 + q, then q / 2 exactly
      const uint32_t word = k < 2 ? r.w.x : r.w.y;
      const __half2 code = bits_h2(__byte_perm(word, 0x64646464u, k & 1 ? 0x4342 : 0x4140));
      const __half2 qh = __hfma2(code, half, off);
      const __half2 h = __hmul2(qh, d2);
      hi[k] = h2_bits(h);
      lo[k] = h2_bits(__hfma2(qh, d2, __hneg2(h)));
    }
  } else if constexpr (KF == MEMRA_KV_FP8_E4M3) {
    e4m3x4_to_half2x2(r.w.x, hi[0], hi[1]);
    e4m3x4_to_half2x2(r.w.y, hi[2], hi[3]);
  } else {   // NVFP4: bytes t/8 and t/8 + 2 of each word hold the (2k, 2k + 1) dim pairs
    const int sh = 8 * (t >> 3);
    const __half2 s2 = e4m3_scale_h2(r.s);
    hi[0] = h2_bits(__hmul2(bits_h2(e2m1x2_to_half2((r.w.x >> sh) & 0xFFu)), s2));
    hi[1] = h2_bits(__hmul2(bits_h2(e2m1x2_to_half2((r.w.x >> (sh + 16)) & 0xFFu)), s2));
    hi[2] = h2_bits(__hmul2(bits_h2(e2m1x2_to_half2((r.w.y >> sh) & 0xFFu)), s2));
    hi[3] = h2_bits(__hmul2(bits_h2(e2m1x2_to_half2((r.w.y >> (sh + 16)) & 0xFFu)), s2));
  }
}

// Raw words of one V staging task of the q5_1 / q4_0 / fp8 layouts: page half
// ph, block b, dim group vg and pair h (dims 32 b + 4 vg + 2 h, + 1), tokens
// 8 ph + 2 c + f.
struct VRaw {
  uint32_t lw[4];              // per c: the code word of pair h
  uint32_t hw[4], dw[4], mw[4];
};

template <int D, int VF>
__device__ __forceinline__ VRaw load_v_task(uint32_t seg, int ph, int b, int vg, int h) {
  constexpr int NB = D / 32;
  VRaw r;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t lane = 4 * vg + c;
    r.hw[c] = r.dw[c] = r.mw[c] = 0u;
    if constexpr (VF == MEMRA_KV_FP8_E4M3) {
      r.lw[c] = lds32(seg + (b * 32 + lane) * 16 + 8 * h + 4 * ph);
    } else {
      const uint32_t doff = ((c * NB + b) * 4 + 2 * ph) * 2;
      r.lw[c] = lds32(seg + ((b >> 1) * 32 + lane) * 16 + (b & 1) * 8 + 4 * h);
      if constexpr (VF == MEMRA_KV_Q5_1) {
        r.hw[c] = lds32(seg + 8 * D + (lane * (NB / 2) + (b >> 1)) * 4);
        r.dw[c] = lds32(seg + 10 * D + doff);
        r.mw[c] = lds32(seg + 11 * D + doff);
      } else {
        r.dw[c] = lds32(seg + 8 * D + doff);
      }
    }
  }
  return r;
}

// The task's values: for dim s of the pair, tokens 2c, 2c + 1 as one fp16
// pair hi[s][c] (and lo[s][c] for q5_1 / q4_0).
template <int VF>
__device__ __forceinline__ void convert_v_task(const VRaw &r, int ph, int b, int h, uint32_t (&hi)[2][4],
                                               uint32_t (&lo)[2][4]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if constexpr (VF == MEMRA_KV_FP8_E4M3) {
      // bytes 2 s + f of the word: (s = 0: f = 0, 1), (s = 1: f = 0, 1)
      e4m3x4_to_half2x2(r.lw[c], hi[0][c], hi[1][c]);
    } else {
      // Both tokens of the pair (f = 0, 1) at once: their codes sit 16 bits
      // apart in the words, and their scales are the two halves of dw, mw.
      // The value, halved, is d q/2 (+ m/2 for q5_1) as hi + lo fp16 parts:
      // the product rounded and its residual (one FMA), and for q5_1 the
      // rounded sum with m/2 and its error (TwoSum).  The _rn operations are
      // never contracted into FMAs.  The parts are exact while the residual
      // is representable in fp16 (d >= 2^-13); below that, the residual and
      // m/2 are rounded to fp16 subnormals (at most 2^-25 off each).
      const __half2 d2 = bits_h2(r.dw[c]);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int sh = 8 * ph + 4 * s;
        uint32_t codes = (r.lw[c] >> sh) & 0x000F000Fu;
        if constexpr (VF == MEMRA_KV_Q5_1) codes |= ((r.hw[c] >> (sh + 2 * (b & 1) + h)) & 0x00010001u) << 4;
        // 1024 + q as fp16, then q/2 (q5_1) or (q - 8)/2 (q4_0), exactly
        const __half2 q2 = __hfma2(bits_h2(codes | 0x64006400u), __float2half2_rn(0.5f),
                                   __float2half2_rn(VF == MEMRA_KV_Q5_1 ? -512.f : -516.f));
        const __half2 p_hi = __hmul2_rn(q2, d2);
        const __half2 p_lo = __hfma2(q2, d2, __hneg2(p_hi));
        if constexpr (VF == MEMRA_KV_Q5_1) {
          const __half2 m2 = __hmul2_rn(bits_h2(r.mw[c]), __float2half2_rn(0.5f));
          const __half2 s2 = __hadd2_rn(p_hi, m2);
          const __half2 bb = __hsub2_rn(s2, p_hi);
          const __half2 e2 = __hadd2_rn(__hsub2_rn(p_hi, __hsub2_rn(s2, bb)), __hsub2_rn(m2, bb));
          hi[s][c] = h2_bits(s2);
          lo[s][c] = h2_bits(__hadd2_rn(e2, p_lo));
        } else {
          hi[s][c] = h2_bits(p_hi);
          lo[s][c] = h2_bits(p_lo);
        }
      }
    }
  }
}

}  // namespace memra
