// Query and key rows made ready for attention in one pass: each head's row is
// normalized, its first dims are turned by the token's position, and the keys
// (with the values) are stored in the paged cache where the call has one.
//
//   y = x / sqrt(mean(x^2) + eps) * w
//   (a, b) -> (a cos - b sin, b cos + a sin),  angle = position * inv_freq[j],
//   (a, b) = (y_j, y_{j + R/2})  or, interleaved,  (y_{2j}, y_{2j+1})
//
// Everything is float32 until the one rounding to fp16; the stored bytes are those
// that kv_append makes of the rounded row.  A key next to a border of its 8-bit code
// falls to one side or the other by its last bits: in float32 some five codes of 8
// million differ from exact arithmetic's, so keys, a small part of the rows, are carried
// as unevaluated sums of two floats from the sum of squares to the rounding.  What is left
// is the angles' 2^-33: of 2 to 4 million turned keys a few at most are not the fp16 value next to
// the exact one, and those lie within 2^-32 of the middle of two (16,384 tokens of 16 and 2 heads, D 256,
// fp8 cache: 88 us, 77 with keys in float32).
//
// Angles.  position * inv_freq reaches 10^5 and more radians, where float32 has no
// digits left behind the point.  So a frequency is kept in turns (inv_freq / 2 pi)
// as a 64-bit binary fraction, rounded once, and the position multiplies it modulo
// 2^64: whole turns fall away exactly.  What is left within an eighth of a turn goes
// through the Taylor series of sine and cosine, their first three terms as two floats.
//
// A row is D / 8 lanes of 8 consecutive dims (one 16-byte load); a warp takes 32 / (D / 8)
// heads of one token at a time, of one kind (K, V or Q), so that it never diverges
// in the quantizer.  With many tokens a warp's unit is all rows of a token: every unit
// costs the same, the angles are taken once, and no warp waits for another.  With few, a
// token is cut into as many units as give every warp one.  The next rows' loads are in
// flight throughout.
//
// Bound by bytes with many tokens, and by the arithmetic of the keys and of the quantizers
// beside them: those 16,384 tokens move 319 MB in 88 us, 3.6 TB/s (queries alone: 268 MB in
// 54 us, 5.0 TB/s; 130 us into q8_0/q5_1, all dims turned, where fp8 takes 106).  2,048 tokens of 32 and 4 heads,
// D 128, no cache: 38 MB in 14.6 us, 12.2 where they are in L2; a warp walks a token's 20 row groups.  With few, by
// the chain of one row: a launch of 8 tokens takes 4.9 us.
#include <algorithm>

#include "kv_stage.cuh"
#include "norm_rope.cuh"

namespace memra {
namespace {

constexpr int kWarps = 8;

// An unevaluated sum, |lo| <= half an ulp of hi.
struct Two {
  float hi, lo;
};

// a * b exactly (Dekker, with a fused product); a + b exactly (Knuth), and for |a| >= |b|.
__device__ __forceinline__ Two two_prod(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ Two fast_two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
// Sums and products but for 2^-45 of them (of the operands, for a sum that cancels).
__device__ __forceinline__ Two add(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi);
  return {s.hi, s.lo + (a.lo + b.lo)};
}
__device__ __forceinline__ Two mul(Two a, Two b) {
  const Two p = two_prod(a.hi, b.hi);
  return {p.hi, fmaf(a.hi, b.lo, fmaf(a.lo, b.hi, p.lo))};
}

// The sum as a float32 that fp16 rounding takes to where it takes the sum itself: to nearest, but for a float that may be the
// middle of two fp16 values (12 bits of zeros at its end).  There what float32 has cut decides, and the float moves a
// step that way (without that, one key in 16,000 became such a middle, and then the neighbour of what it should be).
// Where a part is infinite or NaN, what float32 alone gives; -0 stays -0.
__device__ __forceinline__ float rounded(Two a) {
  const float y = a.hi + a.lo, rest = two_sum(a.hi, a.lo).lo;      // (NaN where the sum is infinite)
  if (y != y || (y == a.hi && rest == 0.f)) return a.hi;
  const uint32_t bits = __float_as_uint(y);
  if ((bits & 0xFFFu) || !(rest < 0.f || rest > 0.f)) return y;
  return __uint_as_float((rest > 0.f) == (y > 0.f) ? bits + 1u : bits - 1u);
}

// Eight sums; all but a few sets of them, without a border or a NaN (whose bits are all ones), need no closer look (16,384 tokens
// of 2 KV heads, D 256: 88 us, 85 rounded to nearest, 102 with the closer look at every sum).
__device__ __forceinline__ void rounded(const Two (&v)[8], float (&x)[8]) {
  uint32_t least = ~0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = v[i].hi + v[i].lo;
    least = min(least, (__float_as_uint(x[i]) + 1u) << 20);
  }
  if (least > 1u << 20) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = rounded(v[i]);
}

// Times a float.
__device__ __forceinline__ Two times(Two a, float b) {
  const Two p = two_prod(a.hi, b);
  return {p.hi, fmaf(a.lo, b, p.lo)};
}
// a b + c d.
__device__ __forceinline__ Two dot(Two a, Two b, Two c, Two d) {
  const Two p = two_prod(a.hi, b.hi), q = two_prod(c.hi, d.hi), s = two_sum(p.hi, q.hi);
  const float lo = fmaf(a.hi, b.lo, fmaf(a.lo, b.hi, p.lo)), lo1 = fmaf(c.hi, d.lo, fmaf(c.lo, d.hi, q.lo));
  return {s.hi, s.lo + (lo + lo1)};
}

// 1 / sqrt(a): an approximation y and one Newton step, y + y (1 - a y^2) / 2, whose correction is the low part.
__device__ __forceinline__ Two rsqrt_two(Two a) {
  const float y = rsqrtf(a.hi);
  const Two p = mul(a, two_prod(y, y));
  return {y, 0.5f * y * (__fsub_rn(1.f, p.hi) - p.lo)};
}

__device__ __forceinline__ void unpack(const uint4 &y, float (&x)[8]) {
  const uint32_t in[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(bits_h2(in[i]));
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
  return make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
}

// Sine and cosine of `rest` 2^-64 turns, an eighth of a turn at most, by their Taylor series, the first three terms as sums of two floats: off
// by less than 2^-33 (with the third in float32, and the square of the angle as the product leaves it, the cosine was off by 2^-26.8).
__device__ __forceinline__ void sin_cos(long long rest, Two &sine, Two &cosine) {
  // 2 pi / 2^64, 1 / 6, 1 / 24, 1 / 120
  constexpr float kHi = 0x1.921fb6p-62f, kLo = -0x1.777a5cp-87f;
  constexpr float k6 = 1.f / 6.f, k6Lo = static_cast<float>(1.0 / 6.0 - static_cast<double>(k6));
  constexpr float k24 = 1.f / 24.f, k24Lo = static_cast<float>(1.0 / 24.0 - static_cast<double>(k24));
  constexpr float k120 = 1.f / 120.f, k120Lo = static_cast<float>(1.0 / 120.0 - static_cast<double>(k120));
  const float r = __ll2float_rn(rest), r_lo = __ll2float_rn(rest - __float2ll_rn(r));
  const Two x = mul({r, r_lo}, {kHi, kLo}), square = mul(x, x), z = fast_two_sum(square.hi, square.lo);
  const float z3 = z.hi * z.hi * z.hi;
  // x - x z / 6 + x z^2 / 120 - x z^3 (1/5040 - ..)
  const Two xz = mul(x, z), cube = mul(xz, {-k6, -k6Lo}), fifth = mul(mul(xz, z), {k120, k120Lo});
  const float odd = fmaf(z.hi, fmaf(z.hi, -1.f / 39916800.f, 1.f / 362880.f), -1.f / 5040.f);
  const Two s0 = two_sum(x.hi, cube.hi), s = two_sum(s0.hi, fifth.hi);
  sine = fast_two_sum(s.hi, fmaf(x.hi * z3, odd, (s0.lo + s.lo) + (x.lo + cube.lo) + fifth.lo));
  // 1 - z / 2 + z^2 / 24 - z^3 (1/720 - ..)
  const Two fourth = mul(mul(z, z), {k24, k24Lo});
  const float even = fmaf(z.hi, fmaf(z.hi, fmaf(z.hi, 1.f / 479001600.f, -1.f / 3628800.f), 1.f / 40320.f), -1.f / 720.f);
  const Two c0 = fast_two_sum(1.f, -0.5f * z.hi), c = two_sum(c0.hi, fourth.hi);
  cosine = fast_two_sum(c.hi, fmaf(z3, even, (c0.lo + c.lo) + fmaf(-0.5f, z.lo, fourth.lo)));
}

// e4m3 codes of the lane's eight values over the scale, the first in the lowest byte.
__device__ __forceinline__ uint2 fp8_codes(const uint4 &y, float scale) {
  const float r = __frcp_rn(scale);
  const uint32_t in[4] = {y.x, y.y, y.z, y.w};
  uint32_t two[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(bits_h2(in[i]));
    two[i] = __nv_cvt_float2_to_fp8x2(make_float2(div_by_scale(f.x, scale, r), div_by_scale(f.y, scale, r)),
                                      __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
}

// The V rows of an even slot and the one behind it, whose bytes lie side by side: words
// (a row alone takes a store for each byte: 16,384 tokens, 2 heads, D 256, fp8/fp8 137 us).
template <int D>
__device__ __forceinline__ void store_v_fp8_pair(const QuantTarget &dst, int page, int t, int head, int l, uint4 even,
                                                 uint4 odd) {
  uint8_t *to = dst.v_pool + (static_cast<size_t>(page) * dst.n_kv_heads + head) * v_seg_bytes(MEMRA_KV_FP8_E4M3, D) +
                (l / 4 * 32 + 8 * (l % 4) + (t % 8) / 2) * 16 + 4 * (t / 8);
  const uint2 a = fp8_codes(even, dst.v_scale), b = fp8_codes(odd, dst.v_scale);
#pragma unroll
  for (int u = 0; u < 2; ++u) {            // element 4 u + 2 h + s lies 64 u + 8 h + 2 s further on
    *reinterpret_cast<uint32_t *>(to + 64 * u) = __byte_perm(u ? a.y : a.x, u ? b.y : b.x, 0x5140);
    *reinterpret_cast<uint32_t *>(to + 64 * u + 8) = __byte_perm(u ? a.y : a.x, u ? b.y : b.x, 0x7362);
  }
}

// CTAS: to an SM.  Two, with all their registers, as long as their warps have a token each at most, so that the chain of one
// is what counts; else three (32 and 4 heads, D 128, fp8 cache: 2,048 tokens 15 us with two, 21 with three, 16,384 99 and 92).
template <int D, int CTAS>
__global__ void __launch_bounds__(32 * kWarps, CTAS) norm_rope_kernel(const NormRopeParams p) {
  constexpr int L = D / 8, ROWS = 32 / L;  // lanes of a row, rows of a warp
  __shared__ unsigned long long s_turns[D / 2];
  __shared__ __align__(16) float s_angles[kWarps][4][D / 2];    // sines, cosines and their low parts of each warp's token
  const int tid = threadIdx.x, lane = tid & 31, l = lane % L, sub = lane / L;
  float(&table)[4][D / 2] = s_angles[tid >> 5];
  grid_dependency_wait();
  allow_dependent_launch();
  if (p.half) {
    for (int j = tid; j < p.half; j += 32 * kWarps) {
      const double turns = static_cast<double>(p.inv_freq[j]) * 0.15915494309189533577;      // 1 / (2 pi)
      s_turns[j] = __double2ull_rz((turns - floor(turns)) * 18446744073709551616.0);
    }
    __syncthreads();
  }
  // Dims of this lane in the rotation: pairs j0 + i (half-split), or the lane's own four pairs.
  const bool turned = 8 * l < 2 * p.half, second = 8 * l >= p.half;
  const int j0 = !turned ? 0 : p.interleaved ? 4 * l : second ? 8 * l - p.half : 8 * l;
  const int partner = turned && !p.interleaved ? (second ? l - p.half / 8 : l + p.half / 8) : l;
  const float sign = second ? 1.f : -1.f;  // of the sine, for the lane's dims (half-split)
  float sn[8], cs[8];                      // this lane's
  // Whole warp: the angles of a position.
  auto angles = [&](int position) {
    __syncwarp();                          // (the ones before have been read)
    for (int j = lane; j < p.half; j += 32) {
      const unsigned long long turn = s_turns[j] * static_cast<unsigned long long>(static_cast<long long>(position));
      // the nearest quarter turn, and what is left (modulo a quarter)
      const unsigned quarter = static_cast<unsigned>((turn + (1ull << 61)) >> 62);
      Two s, c;
      sin_cos(static_cast<long long>(turn << 2) >> 2, s, c);
      const float as = quarter & 2 ? -1.f : 1.f, bs = (quarter + 1) & 2 ? -1.f : 1.f;
      table[0][j] = as * (quarter & 1 ? c.hi : s.hi), table[2][j] = as * (quarter & 1 ? c.lo : s.lo);
      table[1][j] = bs * (quarter & 1 ? s.hi : c.hi), table[3][j] = bs * (quarter & 1 ? s.lo : c.lo);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      if (i > 0 && p.interleaved) continue;
      const float4 s = *reinterpret_cast<const float4 *>(&table[0][j0 + i]);
      const float4 c = *reinterpret_cast<const float4 *>(&table[1][j0 + i]);
      sn[i] = s.x, sn[i + 1] = s.y, sn[i + 2] = s.z, sn[i + 3] = s.w;
      cs[i] = c.x, cs[i + 1] = c.y, cs[i + 2] = c.z, cs[i + 3] = c.w;
    }
    if (!p.interleaved)
#pragma unroll
      for (int i = 0; i < 8; ++i) sn[i] *= sign;
  };
  // Two rows of queries, normalized and turned.
  auto finish = [&](const float(&w)[8], float(&x)[2][8]) {
    if (p.q_weight) {
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[e] = fmaf(x[e][i], x[e][i], sum[e]);
#pragma unroll
      for (int d = 1; d < L; d <<= 1)
#pragma unroll
        for (int e = 0; e < 2; ++e) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], d);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float scale = rsqrtf(fmaf(sum[e], 1.f / D, p.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[e][i] *= scale * w[i];
      }
    }
    if (!p.half) return;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (p.interleaved) {
        if (turned) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = x[e][2 * i], b = x[e][2 * i + 1];
            x[e][2 * i] = fmaf(a, cs[i], -b * sn[i]);
            x[e][2 * i + 1] = fmaf(b, cs[i], a * sn[i]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float b = __shfl_sync(0xffffffffu, x[e][i], partner, L);
          if (turned) x[e][i] = fmaf(x[e][i], cs[i], b * sn[i]);
        }
      }
    }
  };
  // A row of keys, the same in sums of two floats.
  auto finish_key = [&](float(&x)[8]) {
    Two v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = {x[i], 0.f};
    if (p.k_weight) {
      Two sum{x[0] * x[0], 0.f};           // (the square of an fp16 value is exact)
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        const Two s = two_sum(sum.hi, x[i] * x[i]);
        sum = {s.hi, sum.lo + s.lo};
      }
#pragma unroll
      for (int d = 1; d < L; d <<= 1)
        sum = add(sum, {__shfl_xor_sync(0xffffffffu, sum.hi, d), __shfl_xor_sync(0xffffffffu, sum.lo, d)});
      const Two scale = rsqrt_two(add({sum.hi * (1.f / D), sum.lo * (1.f / D)}, {p.eps, 0.f}));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = times(times(scale, p.k_weight[8 * l + i]), x[i]);
    }
    // a cosine + b sine
    auto turn = [&](Two a, Two b, int j, float s) {
      return dot(a, {table[1][j], table[3][j]}, b, {s * table[0][j], s * table[2][j]});
    };
    if (p.half && p.interleaved) {
      if (turned) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Two a = v[2 * i], b = v[2 * i + 1];
          v[2 * i] = turn(a, b, j0 + i, -1.f);
          v[2 * i + 1] = turn(b, a, j0 + i, 1.f);
        }
      }
    } else if (p.half) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const Two b{__shfl_sync(0xffffffffu, v[i].hi, partner, L), __shfl_sync(0xffffffffu, v[i].lo, partner, L)};
        if (turned) v[i] = turn(v[i], b, j0 + i, sign);
      }
    }
    rounded(v, x);
  };
  auto weights = [&](const float *weight, float(&w)[8]) {       // the norm's, of this lane's dims
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = weight ? weight[8 * l + i] : 1.f;
  };
  float qw[8];
  weights(p.q_weight, qw);

  // Consecutive units go to different CTAs, so that the last ones spread over the GPU.
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
#pragma unroll 1
  for (int64_t unit = static_cast<int64_t>(tid >> 5) * gridDim.x + blockIdx.x; unit < p.units; unit += warps) {
    const int token = static_cast<int>(unit / p.parts), part = static_cast<int>(unit % p.parts);
    // Row groups of the unit by kind: all of the token's, or one share.
    int v0 = 0, v1 = p.v_passes, k0 = 0, k1 = p.k_passes, q0 = 0, q1 = p.q_passes;
    if (p.parts > 1) {
      const int vs = (p.v_passes + p.kv_share - 1) / p.kv_share, ks = (p.k_passes + p.kv_share - 1) / p.kv_share;
      auto cut = [](int i, int share, int passes) { return min(max(i, 0) * share, passes); };
      v0 = cut(part, p.kv_share, p.v_passes), v1 = cut(part + 1, p.kv_share, p.v_passes);
      k0 = cut(part - vs, p.kv_share, p.k_passes), k1 = cut(part + 1 - vs, p.kv_share, p.k_passes);
      q0 = cut(part - vs - ks, p.q_share, p.q_passes), q1 = cut(part + 1 - vs - ks, p.q_share, p.q_passes);
    }
    auto load = [&](const __half *base, int64_t stride, int pass, int end, int heads) {
      const int head = pass * ROWS + sub;
      return pass < end && head < heads ? *reinterpret_cast<const uint4 *>(base + token * stride + (head * D + 8 * l))
                                        : make_uint4(0, 0, 0, 0);
    };
    // the first rows of each kind
    uint4 yv = load(p.v, p.v_stride, v0, v1, p.n_kv_heads), yk = load(p.k, p.k_stride, k0, k1, p.n_kv_heads);
    uint4 yq[2] = {load(p.q, p.q_stride, q0, q1, p.n_heads), load(p.q, p.q_stride, q0 + 1, q1, p.n_heads)};
    int slot = p.slots && (v0 < v1 || k0 < k1) ? p.slots[token] : -1;
    const bool fp8 = v0 < v1 && p.cache.v_fmt == MEMRA_KV_FP8_E4M3;
    const int slot_after = fp8 && token + 1 < p.tokens ? p.slots[token + 1] : -1;
    const int slot_before = fp8 && token > 0 ? p.slots[token - 1] : -1;
    const bool turning = p.half && (k0 < k1 || q0 < q1);
    const int position = turning ? p.positions[token] : 0;
    if (slot >= 0 && slot / kPage >= p.num_pages) {
      if (k0 < k1 && lane == 0) flag_error(p.status, MEMRA_DEVERR_BAD_SLOT);
      slot = -1;
    }
    const int page = slot >= 0 ? slot / kPage : 0, place = slot >= 0 ? slot % kPage : 0;
    if (turning) angles(position);
    // fp8 values of an even slot and of the next token's are stored together, by the first of the two.
    const bool pair = fp8 && slot >= 0 && slot % 2 == 0 && slot_after == slot + 1;
    if (fp8 && slot >= 0 && slot % 2 == 1 && slot_before == slot - 1) v0 = v1;
#pragma unroll 1
    for (int pass = v0; pass < v1; ++pass) {
      const uint4 y = yv;
      yv = load(p.v, p.v_stride, pass + 1, v1, p.n_kv_heads);
      const int head = pass * ROWS + sub;
      if (pair) {
        const uint4 odd = load(p.v + p.v_stride, p.v_stride, pass, v1, p.n_kv_heads);
        if (head < p.n_kv_heads) store_v_fp8_pair<D>(p.cache, page, place, head, l, y, odd);
        continue;
      }
      quantize_store_row<D>(p.cache, slot >= 0 && head < p.n_kv_heads, page, place, head, l, y, y, false, true);
    }
#pragma unroll 1
    for (int pass = k0; pass < k1; ++pass) {
      float x[8];
      unpack(yk, x);
      yk = load(p.k, p.k_stride, pass + 1, k1, p.n_kv_heads);
      finish_key(x);
      const uint4 y = pack(x);
      const int head = pass * ROWS + sub;
      if (p.k_out && head < p.n_kv_heads)
        *reinterpret_cast<uint4 *>(p.k_out + token * p.k_out_stride + (head * D + 8 * l)) = y;
      if (p.slots)
        quantize_store_row<D>(p.cache, slot >= 0 && head < p.n_kv_heads, page, place, head, l, y, y, true, false);
    }
    // two query row groups at a time
    __half *dst = p.q_out + token * p.q_out_stride + 8 * l;
#pragma unroll 1
    for (int pass = q0; pass < q1; pass += 2) {
      float x[2][8];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        unpack(yq[e], x[e]);
        yq[e] = load(p.q, p.q_stride, pass + 2 + e, q1, p.n_heads);
      }
      finish(qw, x);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int head = (pass + e) * ROWS + sub;
        if (pass + e < q1 && head < p.n_heads) *reinterpret_cast<uint4 *>(dst + head * D) = pack(x[e]);
      }
    }
  }
}

template <int D, int CTAS>
cudaError_t launch(NormRopeParams p, int sms, cudaStream_t st) {
  constexpr int kRows = 32 / (D / 8);
  auto groups = [](int64_t n, int64_t per) { return static_cast<int>((n + per - 1) / per); };
  p.k_passes = p.k ? groups(p.n_kv_heads, kRows) : 0;
  p.v_passes = p.slots ? groups(p.n_kv_heads, kRows) : 0;
  p.q_passes = groups(p.n_heads, kRows);
  // A unit to a warp: a token's row groups of K and of V in shares as small as leave the queries' a warp, these in as many
  // as there are then (a row of K or V takes some three times a query's).  From so many tokens on that three units a
  // token are too many, whole tokens (32 and 8 heads, D 128, fp8: 512 tokens 11 us so, 17 whole, 15 group by group; 4,096
  // tokens 43 us whole, 67 group by group).
  const int64_t warps = static_cast<int64_t>(CTAS) * sms * kWarps, tokens = p.tokens, room = tokens > 0 ? warps / tokens : 0;
  p.parts = 1;
  for (int share = 1; p.parts == 1 && share <= std::max({p.k_passes, p.v_passes, 1}); ++share) {
    const int kv = groups(p.k_passes, share) + groups(p.v_passes, share);
    if (room <= kv) continue;
    p.kv_share = share, p.q_share = groups(p.q_passes, room - kv);
    p.parts = kv + groups(p.q_passes, p.q_share);
  }
  p.units = tokens * p.parts;
  // (an odd number of CTAs: even and odd tokens to every SM)
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((p.units + kWarps - 1) / kWarps, (static_cast<int64_t>(CTAS) * sms - 1) | 1));
  return launch_pdl(norm_rope_kernel<D, CTAS>, dim3(grid), dim3(32 * kWarps), 0, st, p);
}

}  // namespace

cudaError_t launch_norm_rope(int D, NormRopeParams p, int sms, cudaStream_t st) {
  if (p.tokens <= 2 * sms * kWarps) return D == 128 ? launch<128, 2>(p, sms, st) : launch<256, 2>(p, sms, st);
  return D == 128 ? launch<128, 3>(p, sms, st) : launch<256, 3>(p, sms, st);
}

}  // namespace memra
