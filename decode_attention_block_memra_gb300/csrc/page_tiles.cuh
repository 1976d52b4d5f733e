// Chunks of raw pages in shared memory to fp16 operand tiles in shared memory, for
// the kernels that dequantize a page once for many query rows (tree and chunk
// attention).
#pragma once

#include "kv_stage.cuh"

namespace memra {

// ---- staging: a chunk's raw pages in shared memory to operand tiles -------------
// Every raw code byte is read by 16-byte loads in lane order (the order of the
// page layout: conflict-free), and each value goes to the tile from the thread
// that read it.  A warp task is one 512-byte run of codes.

// Eight q8_0 or fp8 codes of K as fp16: q8_0 q d / 2 in hi + lo parts (d2 the
// scale in both halves), fp8 the value in hi.
template <int KF>
__device__ __forceinline__ void convert_k16(uint2 w, uint32_t d2, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  if constexpr (KF == MEMRA_KV_Q8_0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // stored q + 128, spliced under 1024: 1152 + q, then q / 2 exactly
      const uint32_t code = __byte_perm(k < 2 ? w.x : w.y, 0x64646464u, k & 1 ? 0x4342 : 0x4140);
      const uint32_t qh = hfma2_u32(code, 0x38003800u, 0xE080E080u);          // 0.5, -576
      hi[k] = hmul2_u32(qh, d2);
      lo[k] = hfms2_u32(qh, d2, hi[k]);
    }
  } else {
    e4m3x4_to_half2x2(w.x, hi[0], hi[1]);
    e4m3x4_to_half2x2(w.y, hi[2], hi[3]);
  }
}

// K^: token rows of 128 bytes (64 dims, the K axis of the score MMA), 128-byte-
// swizzled (the 16-byte unit of a row is XORed with the row's index in its group
// of 8), one block of KEYS rows per 64 dims.  A lane holds the same 8 dims of
// two 32-dim blocks; lanes of odd tokens store the second block first, so that
// eight lanes' 16-byte stores always fall on different banks.
// Tokens that do not exist stage whatever the pages hold: their scores are masked.
// ROWS: of the tile that `buf` is a part of, KEYS of them from a multiple of 8 on.
template <int D, int KF, int KEYS, int WARPS, int ROWS = KEYS>
__device__ __forceinline__ void stage_k(uint32_t raw, uint32_t buf, int warp, int lane) {
  constexpr int NB = D / 32, SEG = k_seg_bytes(KF, D), B2 = D / 64;
  constexpr uint32_t LO = ROWS * D * 2;
  const int tg = lane >> 2, kc = lane & 3;
  if constexpr (KF == MEMRA_KV_NVFP4) {
    // run (page, 64-dim block): words (b % 2, e / 4), bytes tp + 2 (e % 4 / 2), nibbles e % 2
    constexpr int TASKS = KEYS / kPage * B2;
    static_assert(TASKS % WARPS == 0, "whole tasks");
#pragma unroll
    for (int it = 0; it < TASKS / WARPS; ++it) {
      const int task = warp + it * WARPS, pg = task / B2, b2 = task % B2;
      const uint32_t seg = raw + pg * SEG;
      const uint4 x = lds128(seg + (b2 * 32 + lane) * 16);
#pragma unroll
      for (int tp = 0; tp < 2; ++tp)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool bp = e ^ (tg & 1);
          const uint32_t w0 = (bp ? x.z : x.x) >> (8 * tp), w1 = (bp ? x.w : x.y) >> (8 * tp);
          const int t = 8 * tp + tg, u = 4 * bp + kc;
          const __half2 s2 = e4m3_scale_h2(lds8(seg + 8 * D + t * (D / 16) + 4 * b2 + (u >> 1)));
          uint4 h;
          h.x = h2_bits(__hmul2(bits_h2(e2m1x2_to_half2(w0 & 0xFFu)), s2));
          h.y = h2_bits(__hmul2(bits_h2(e2m1x2_to_half2((w0 >> 16) & 0xFFu)), s2));
          h.z = h2_bits(__hmul2(bits_h2(e2m1x2_to_half2(w1 & 0xFFu)), s2));
          h.w = h2_bits(__hmul2(bits_h2(e2m1x2_to_half2((w1 >> 16) & 0xFFu)), s2));
          sts128(buf + b2 * ROWS * 128 + (kPage * pg + t) * 128 + ((u ^ tg) << 4), h);
        }
    }
  } else {
    // run (page, token half, 64-dim block): 8 bytes for each of the two 32-dim blocks
    constexpr unsigned TASKS = KEYS / 8 * B2, STEP = WARPS / B2;     // a warp's token groups are STEP apart
    static_assert(TASKS % WARPS == 0 && WARPS % B2 == 0 && (STEP % 2 == 0 || STEP == 1), "whole tasks");
    const unsigned g0 = static_cast<unsigned>(warp) / B2, b2 = static_cast<unsigned>(warp) % B2;
    const bool odd = tg & 1;
    const uint32_t sel0 = odd ? 0x3232u : 0x1010u, sel1 = odd ? 0x1010u : 0x3232u;
    const uint32_t row = buf + b2 * (ROWS * 128) + (8 * g0 + tg) * 128;
    const uint32_t to0 = row + (((odd ? 4 : 0) + kc) ^ tg) * 16, to1 = row + (((odd ? 0 : 4) + kc) ^ tg) * 16;
    const uint32_t codes = raw + (g0 >> 1) * SEG + (((g0 & 1) * B2 + b2) * 32 + lane) * 16;
    const uint32_t scales = raw + (g0 >> 1) * SEG + 16 * D + ((8 * (g0 & 1) + tg) * NB + 2 * b2) * 2;
    // (STEP = 1: every warp starts at group 0, so the halves of a page alternate)
    auto code_off = [](unsigned it) { return it * STEP / 2 * SEG + (it * STEP) % 2 * (B2 * 512); };
    auto scale_off = [](unsigned it) { return it * STEP / 2 * SEG + (it * STEP) % 2 * (8 * NB * 2); };
    constexpr unsigned PER = TASKS / WARPS, BATCH = PER < 4 ? PER : 4;
    uint4 x[BATCH];
    uint32_t d[BATCH];
#pragma unroll
    for (unsigned it = 0; it < PER; ++it) {
      if (it % BATCH == 0) {
#pragma unroll
        for (unsigned e = 0; e < BATCH; ++e) {
          x[e] = lds128(codes + code_off(it + e));
          d[e] = KF == MEMRA_KV_Q8_0 ? lds32(scales + scale_off(it + e)) : 0u;
        }
      }
      const uint4 y = x[it % BATCH];
      const uint2 w0 = make_uint2(odd ? y.z : y.x, odd ? y.w : y.y), w1 = make_uint2(odd ? y.x : y.z, odd ? y.y : y.w);
      uint32_t hi[4], lo[4];
      convert_k16<KF>(w0, __byte_perm(d[it % BATCH], 0, sel0), hi, lo);
      sts128(to0 + it * STEP * 1024, make_uint4(hi[0], hi[1], hi[2], hi[3]));
      if constexpr (KF == MEMRA_KV_Q8_0) sts128(to0 + it * STEP * 1024 + LO, make_uint4(lo[0], lo[1], lo[2], lo[3]));
      convert_k16<KF>(w1, __byte_perm(d[it % BATCH], 0, sel1), hi, lo);
      sts128(to1 + it * STEP * 1024, make_uint4(hi[0], hi[1], hi[2], hi[3]));
      if constexpr (KF == MEMRA_KV_Q8_0) sts128(to1 + it * STEP * 1024 + LO, make_uint4(lo[0], lo[1], lo[2], lo[3]));
    }
  }
}

__device__ __forceinline__ void sts64(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}

// Eight tokens (pairs in words), those whose bit is set; the others become zeros.
__device__ __forceinline__ uint4 keep_tokens(const uint32_t (&x)[4], uint32_t bits) {
  uint32_t y[4];
#pragma unroll
  for (int c = 0; c < 4; ++c)
    y[c] = x[c] & (((bits >> (2 * c)) & 1u ? 0xFFFFu : 0u) | ((bits >> (2 * c + 1)) & 1u ? 0xFFFF0000u : 0u));
  return make_uint4(y[0], y[1], y[2], y[3]);
}

// The 16 bits of page pg in the chunk's.
__device__ __forceinline__ uint32_t page_bits(uint64_t keep, int pg) {
  return static_cast<uint32_t>(keep >> (kPage * pg)) & 0xFFFFu;
}

// V^ of q5_1, q4_0 and fp8: token rows of 128 bytes (64 dims), 128-byte-swizzled
// (the 16-byte unit of a row is XORed with the row's index in its group of 8),
// one block of KEYS rows per 64 dims: the MN-major B operand of O += P V.  A
// lane holds 4 consecutive dims of 4 tokens, so nothing is transposed, and a
// warp's 8-byte stores fill all banks.  Tokens without a bit in `keep` become zeros:
// 0 * (what their bytes stand for) need not be 0.  q5_1 stages d (q - 16) where
// the blocks' centres have columns of their own (M_COLS), else d q + m by a TwoSum.
template <int D, int VF, int KEYS, int WARPS, bool M_COLS, uint32_t LO>
__device__ __forceinline__ void stage_v(uint32_t raw, uint32_t buf, uint64_t keep, int warp, int lane) {
  constexpr int NB = D / 32, SEG = v_seg_bytes(VF, D), B2 = D / 64;
  const int vg = lane >> 2, c = lane & 3;
  // token 8 p + 2 c + f of page pg, block b, dims 4 vg .. + 3
  auto at = [&](int pg, int p, int f, int b) {
    const int r8 = 2 * c + f, row = kPage * pg + 8 * p + r8;
    return buf + (b >> 1) * KEYS * 128 + row * 128 + ((((b & 1) * 64 + vg * 8)) ^ (r8 << 4));
  };
  if constexpr (VF == MEMRA_KV_FP8_E4M3) {
    // run (page, 32-dim block): words 2 h + p, bytes 2 s + f
    constexpr int TASKS = KEYS / kPage * NB;
    static_assert(TASKS % WARPS == 0, "whole tasks");
#pragma unroll
    for (int it = 0; it < TASKS / WARPS; ++it) {
      const int task = warp + it * WARPS, pg = task / NB, b = task % NB;
      const uint32_t bits = page_bits(keep, pg);
      const uint4 x = lds128(raw + pg * SEG + (b * 32 + lane) * 16);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        // bytes (s0 f0, s0 f1, s1 f0, s1 f1) to (s0 f0, s1 f0, s0 f1, s1 f1): one pair per token
        uint32_t h0[2], h1[2];
        e4m3x4_to_half2x2(__byte_perm(p ? x.y : x.x, 0, 0x3120), h0[0], h0[1]);
        e4m3x4_to_half2x2(__byte_perm(p ? x.w : x.z, 0, 0x3120), h1[0], h1[1]);
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const bool live = (bits >> (8 * p + 2 * c + f)) & 1u;
          sts64(at(pg, p, f, b), live ? h0[f] : 0u, live ? h1[f] : 0u);
        }
      }
    }
  } else {
    // run (page, 64-dim block): words 2 (b % 2) + h, bytes 2 f + p, nibbles s
    constexpr unsigned TASKS = KEYS / kPage * B2, STEP = WARPS / B2;       // a warp's pages are STEP apart
    static_assert(TASKS % WARPS == 0 && WARPS % B2 == 0, "whole tasks");
    const unsigned pg0 = static_cast<unsigned>(warp) / B2, b2 = static_cast<unsigned>(warp) % B2;
    uint32_t to[2][2];                   // [b % 2][f], the row of p = 0
#pragma unroll
    for (int e = 0; e < 4; ++e)
      to[e >> 1][e & 1] = buf + b2 * (KEYS * 128) + (kPage * pg0 + 2 * c + (e & 1)) * 128 +
                          (((e >> 1) * 64 + vg * 8) ^ ((2 * c + (e & 1)) << 4));
    const uint32_t seg0 = raw + pg0 * SEG;
    const uint32_t codes = seg0 + (b2 * 32 + lane) * 16, fifths = seg0 + 8 * D + (lane * (NB / 2) + b2) * 4;
    const uint32_t scales = seg0 + (VF == MEMRA_KV_Q5_1 ? 10 : 8) * D + (c * NB + 2 * b2) * 8;
#pragma unroll
    for (unsigned it = 0; it < TASKS / WARPS; ++it) {
      const uint32_t off = it * STEP * SEG, row = it * STEP * (kPage * 128);
      const uint4 x4 = lds128(codes + off);
      const uint32_t hw = VF == MEMRA_KV_Q5_1 ? lds32(fifths + off) : 0u;
      const uint4 d4 = lds128(scales + off);           // scales of the lane's tokens (halves 2 p + f), two blocks
      uint4 m4 = make_uint4(0, 0, 0, 0);
      if constexpr (VF == MEMRA_KV_Q5_1 && !M_COLS) m4 = lds128(scales + D + off);
      const uint32_t bits = page_bits(keep, pg0 + it * STEP);
#pragma unroll
      for (int bp = 0; bp < 2; ++bp) {
        uint32_t hi[4][2], lo[4][2];     // [byte 2 f + p][h]
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = bp ? (h ? x4.w : x4.z) : (h ? x4.y : x4.x);
          uint32_t l4 = x & 0x0F0F0F0Fu, h4 = (x >> 4) & 0x0F0F0F0Fu;
          if constexpr (VF == MEMRA_KV_Q5_1) {
            l4 |= (hw << (4 - 2 * bp - h)) & 0x10101010u;
            h4 |= (hw >> (2 * bp + h)) & 0x10101010u;
          }
          const uint32_t p01 = __byte_perm(l4, h4, 0x5140), p23 = __byte_perm(l4, h4, 0x7362);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // 1024 + q as fp16 for dims s = 0, 1; then q / 2 (q5_1), (q - 16) / 2 or (q - 8) / 2 (q4_0), exactly
            const uint32_t q2 = hfma2_u32(__byte_perm(k < 2 ? p01 : p23, 0x64646464u, k & 1 ? 0x4342 : 0x4140), 0x38003800u,
                                          VF == MEMRA_KV_Q4_0 ? 0xE008E008u : M_COLS ? 0xE010E010u : 0xE000E000u);   // 0.5; -516, -520, -512
            const int f = k >> 1, p = k & 1;
            const uint32_t sel = f ? 0x3232 : 0x1010;
            const uint32_t d2 = __byte_perm(bp ? (p ? d4.w : d4.z) : (p ? d4.y : d4.x), 0, sel);
            const uint32_t p_hi = h2_bits(__hmul2_rn(bits_h2(q2), bits_h2(d2)));
            const uint32_t p_lo = hfms2_u32(q2, d2, p_hi);
            if constexpr (VF == MEMRA_KV_Q5_1 && !M_COLS) {
              const __half2 m2 = __hmul2_rn(bits_h2(__byte_perm(bp ? (p ? m4.w : m4.z) : (p ? m4.y : m4.x), 0, sel)),
                                            __float2half2_rn(0.5f));
              const __half2 s2 = __hadd2_rn(bits_h2(p_hi), m2);
              const __half2 bb = __hsub2_rn(s2, bits_h2(p_hi));
              const __half2 e2 = __hadd2_rn(__hsub2_rn(bits_h2(p_hi), __hsub2_rn(s2, bb)), __hsub2_rn(m2, bb));
              hi[k][h] = h2_bits(s2);
              lo[k][h] = h2_bits(__hadd2_rn(e2, bits_h2(p_lo)));
            } else {
              hi[k][h] = p_hi;
              lo[k][h] = p_lo;
            }
          }
        }
        if (bits != 0xFFFFu) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (!((bits >> (8 * (k & 1) + 2 * c + (k >> 1))) & 1u)) hi[k][0] = hi[k][1] = lo[k][0] = lo[k][1] = 0u;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t at = to[bp][k >> 1] + row + (k & 1) * 1024;
          sts64(at, hi[k][0], hi[k][1]);
          sts64(at + LO, lo[k][0], lo[k][1]);
        }
      }
    }
  }
}

// V^T of NVFP4 (dim rows, tokens along K, core matrices): its lanes hold single
// dims, so a task gathers the 8 tokens of two dims and stores 16-byte rows.
template <int D, int KEYS, int WARPS>
__device__ __forceinline__ void stage_v_nvfp4(uint32_t raw, uint32_t buf, uint64_t keep, int st) {
  constexpr int SEG = v_seg_bytes(MEMRA_KV_NVFP4, D), TASKS = KEYS / kPage * 2 * (D / 16) * 8, IT = TASKS / (32 * WARPS);
  static_assert(IT * (32 * WARPS) == TASKS, "whole tasks");
#pragma unroll
  for (int it = 0; it < IT; ++it) {      // task (page, half page, 16-dim block b16, rr): dims 16 b16 + rr and + 8
    const int task = st + it * (32 * WARPS), rr = task & 7, b16 = (task >> 3) % (D / 16),
              ph = (task / (8 * (D / 16))) & 1, pg = task / (16 * (D / 16)), g = 2 * pg + ph;
    const uint32_t seg = raw + pg * SEG;
    uint32_t h0[4], h1[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t cw = lds32(seg + ((b16 >> 2) * 32 + 4 * rr + c) * 16 + (b16 & 3) * 4);
      const uint32_t sw = lds32(seg + 8 * D + (c * (D / 16) + b16) * 4);
      __half2 v[2];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int sh = 8 * (f + 2 * ph);
        v[f] = __hmul2(bits_h2(e2m1x2_to_half2((cw >> sh) & 0xFFu)), e4m3_scale_h2(sw >> sh));
      }
      h0[c] = h2_bits(__lows2half2(v[0], v[1]));
      h1[c] = h2_bits(__highs2half2(v[0], v[1]));
    }
    const uint32_t bits = page_bits(keep, pg) >> (8 * ph);
    const int d0 = 16 * b16 + rr;
    const uint32_t at = buf + ((d0 >> 3) * (KEYS / 8) + g) * 128 + (d0 & 7) * 16;
    sts128(at, keep_tokens(h0, bits));
    sts128(at + (KEYS / 8) * 128, keep_tokens(h1, bits));
  }
}

// The centres of q5_1's blocks, m / 2 + 8 d in hi + lo parts (a TwoSum; half the
// value, as everything is staged), as columns of V^: a further 64-column block of
// which the MMA takes 16, token n's hi and then lo parts of the four blocks in
// its first 16-byte unit.
template <int D, int KEYS>
__device__ __forceinline__ void stage_m(uint32_t raw, uint32_t buf, uint64_t keep, int n) {
  constexpr int NB = D / 32, SEG = v_seg_bytes(MEMRA_KV_Q5_1, D);
  static_assert(NB == 4, "8 bytes of each part");
  const int pg = n / kPage, t = n % kPage;
  const uint32_t at = raw + pg * SEG + 10 * D + (((t & 7) >> 1) * NB * 4 + 2 * (t >> 3) + (t & 1)) * 2;
  uint32_t hi[2], lo[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {            // two blocks at a time
    const __half2 d = bits_h2(lds16(at + 16 * e) | (lds16(at + 16 * e + 8) << 16));
    const __half2 m = bits_h2(lds16(at + D + 16 * e) | (lds16(at + D + 16 * e + 8) << 16));
    const __half2 a = __hmul2_rn(m, __float2half2_rn(0.5f)), b = __hmul2_rn(d, __float2half2_rn(8.f));
    const __half2 s = __hadd2_rn(a, b), bb = __hsub2_rn(s, a);
    hi[e] = h2_bits(s);
    lo[e] = h2_bits(__hadd2_rn(__hsub2_rn(a, __hsub2_rn(s, bb)), __hsub2_rn(b, bb)));
  }
  const bool live = (keep >> n) & 1u;
  const uint4 x = live ? make_uint4(hi[0], hi[1], lo[0], lo[1]) : make_uint4(0, 0, 0, 0);
  sts128(buf + n * 128 + ((n & 7) << 4), x);
}

}  // namespace memra
