// Where the bytes of a token's row lie in a page segment, for the kernels that
// move rows as they are (compaction, eviction).
#pragma once

#include "memra_device.cuh"

namespace memra {

// Byte x (0 .. seg / 16 - 1) of a token's row in a page segment lies, by the
// layout of memra.h, at a part that depends on x plus a part that depends on
// the token t alone, one of a few kinds; x means the same part of the row for
// every t.
enum RowPart { kKCodes = 0, kKHalves, kKNvCodes, kKNvScales, kVBytes, kVFifths, kVHalves, kVFp8, kVNvBytes, kVNvScales };

template <int D>
__device__ __forceinline__ int token_offset(int part, int t) {
  constexpr int NB = D / 32;
  const int c = (t & 7) >> 1, f = t & 1, p = t >> 3;
  switch (part) {
    case kKCodes: return (p * (NB / 2) * 32 + 4 * (t & 7)) * 16;
    case kKHalves: return t * NB * 2;
    case kKNvCodes: return 4 * (t & 7) * 16 + p;
    case kKNvScales: return t * (D / 16);
    case kVBytes: return c * 16 + 2 * f + p;
    case kVFifths: return c * (NB / 2) * 4 + 2 * f + p;
    case kVHalves: return (c * NB * 4 + 2 * p + f) * 2;
    case kVFp8: return c * 16 + 4 * p + f;
    case kVNvBytes: return c * 16 + f + 2 * p;
    default: return c * (D / 16) * 4 + f + 2 * p;           // kVNvScales
  }
}

template <int D>
__device__ __forceinline__ int k_byte(int fmt, int x, int &part) {
  if (fmt == MEMRA_KV_NVFP4) {
    part = x < D / 2 ? kKNvCodes : kKNvScales;
    return x < D / 2 ? ((x >> 5) * 32 + ((x >> 3) & 3)) * 16 + ((x >> 1) & 3) * 4 + 2 * (x & 1) : 8 * D + x - D / 2;
  }
  part = x < D ? kKCodes : kKHalves;
  return x < D ? ((x >> 6) * 32 + ((x >> 3) & 3)) * 16 + ((x >> 5) & 1) * 8 + (x & 7) : 16 * D + x - D;
}

template <int D>
__device__ __forceinline__ int v_byte(int fmt, int x, int &part) {
  constexpr int NB = D / 32;
  const int lane = 4 * ((x >> 2) & 7);                       // the lane of the run (x >> 5), but for the token's share
  if (fmt == MEMRA_KV_FP8_E4M3) {
    part = kVFp8;
    return ((x >> 5) * 32 + lane) * 16 + 8 * ((x >> 1) & 1) + 2 * (x & 1);
  }
  if (x < D / 2) {
    part = fmt == MEMRA_KV_NVFP4 ? kVNvBytes : kVBytes;
    return ((x >> 5) * 32 + lane) * 16 + (fmt == MEMRA_KV_NVFP4 ? (x & 3) * 4 : ((x >> 1) & 1) * 8 + 4 * (x & 1));
  }
  x -= D / 2;
  if (fmt == MEMRA_KV_NVFP4) {
    part = kVNvScales;
    return 8 * D + x * 4;
  }
  if (fmt == MEMRA_KV_Q5_1) {
    if (x < D / 8) {
      part = kVFifths;
      return 8 * D + (4 * (x / (NB / 2)) * (NB / 2) + x % (NB / 2)) * 4;
    }
    x -= D / 8;
  }
  part = kVHalves;                                           // scales, and D bytes on the minima of q5_1
  const int m = x >= 2 * NB;
  x -= m ? 2 * NB : 0;
  return (fmt == MEMRA_KV_Q5_1 ? 10 : 8) * D + m * D + (x >> 1) * 8 + (x & 1);
}

}  // namespace memra
