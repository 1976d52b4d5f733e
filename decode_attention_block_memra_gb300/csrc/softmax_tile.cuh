// Pieces of the row softmax over a score tile in registers (thread = row).
#pragma once

#include <stdint.h>

#include "memra_device.cuh"

namespace memra {

// Two floats as an fp16 pair; what is past fp16's range is cut to its largest value (infinities too; NaN stays NaN).
__device__ __forceinline__ uint32_t pack_half2_sat(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two float32 products in one instruction.
__device__ __forceinline__ uint64_t mul_f2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// named_barrier_sync, and whether x holds in all of its threads.
__device__ __forceinline__ bool named_barrier_and(int id, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\t"
      "bar.red.and.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}

// Two fp16 NaN; as one float32, NaN too: what rows hold whose kernel gave up a wait.
constexpr uint32_t kNanPair = 0x7FFF7FFFu;

// Largest of N scores (float bits).
template <int N>
__device__ __forceinline__ float row_max(const uint32_t (&s)[N]) {
  static_assert(N % 8 == 0, "four chains of pairs");
  float m[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) m[e] = fmaxf(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
#pragma unroll
  for (int c = 8; c < N; c += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = max3(m[e], __uint_as_float(s[c + 2 * e]), __uint_as_float(s[c + 2 * e + 1]));
  return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}

// p = 2^(s * scale - m) of 2 N scores from s, as fp16 pairs into w; adds them to the pair of sums.
template <int N>
__device__ __forceinline__ void row_weights(const uint32_t *s, float scale, float m, uint32_t *w, uint64_t &sum) {
  const uint64_t scale2 = pack_f2(scale, scale), minus_m = pack_f2(-m, -m);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    float x0, x1;
    unpack_f2(fma_f2(pack_f2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), scale2, minus_m), x0, x1);
    const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
    sum = add_f2(sum, pack_f2(p0, p1));
    w[e] = pack_half2(p0, p1);
  }
}

}  // namespace memra
