// Tree attention: a tree of up to 64 drafted nodes per sequence against the
// block-quantized paged cache.  Node i sees every key before the tree's rows
// and, of the tree's own, those whose bit its mask word holds:
//
//   o_i = sum_u p_iu V^_u / sum_u p_iu,  p_iu = 2^(q_i . K^_u * scale * log2(e) - m_i)
//
// The rows of one KV head, nodes x the group's query heads, 128 to a tile, are
// the M side of tcgen05 MMAs, so a page is read and dequantized once for 128 of
// them (256 at head_dim 128).  CTA = (split of the keys, KV head, sequence, its rows):
//   * a copy warp brings raw pages into a ring of two to four chunks (64 keys);
//   * staging warps dequantize a chunk into fp16 operand tiles: exact hi + lo
//     pairs for q8_0, q5_1 and q4_0, single values for fp8 and NVFP4, so only P
//     is rounded (fp16, relative 2^-11 a weight);
//   * one MMA thread: S = Q K^T with Q in tensor memory, O += P V with P in
//     tensor memory over its scores; the A operands stay out of shared memory,
//     whose bandwidth the staged tiles need;
//   * groups of four softmax warps, thread = row.
// One CTA to an SM.  At head_dim 128 it has two softmax groups, each with an O of
// its own, and one's softmax fills the gaps of the other's MMAs: two row tiles
// past 128 rows; else one row tile whose chunks they take by turns, their O joined
// at the end (8 sequences x 8 nodes over 4,104 keys: 28.3 us, 31.2 as two CTAs on
// an SM, which also leave twice the partial rows to the merge).  Four of the eight
// staging warps take every other chunk (all eight on each: 44.8 for 39.8 us below).
// head_dim 256: one group, two score buffers, the scores a chunk ahead.
// What bounds it: no unit is saturated; the time is in chains of waits.  A chunk
// of q8_0/q5_1 is 28 KB in, 64 KB of tiles out and 66 KB read by the MMAs of each
// row tile through a shared memory of 128 bytes a clock, 1,060 clocks of MMAs and
// 4,900 warp instructions, and takes 1,810 clocks with one row tile: the one issuing
// thread finds its operands ready.  8 sequences x 16 nodes over 6,316 keys (32/4 heads,
// D 128, q8_0/q5_1): 40.2 us a call, 5.5 of them the merge, for 47 MB of pages (4
// splits a sequence on 128 of 152 SMs: 5 would not fit), tensor pipe 33%, shared memory
// 50 to 60%; 64 nodes over 262,144 keys: 370 us, both 69%; 31 nodes on 12 ragged
// sequences, D 256, fp8: 75.3 us, 38% and 68%.
// A sequence of one split writes its rows directly; the others leave (o, lse)
// partials that tree_merge_kernel joins.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "kv_stage.cuh"
#include "softmax_tile.cuh"
#include "tcgen05.cuh"
#include "tree.cuh"

namespace memra {
namespace {

constexpr int kTileRows = 128;
constexpr float kLazy = 8.f;               // log2 units: P stays <= 256 between rescales

template <int D, int KF, int VF, int MT>
struct TreeCfg {
  // Softmax groups of four warps, each with an O of its own: one per row tile; at head_dim 128 a single
  // row tile has two, which take the chunks by turns (kTurns) and are joined at the end.
  static constexpr int kGroups = D == 128 ? 2 : 1;
  static constexpr bool kTurns = kGroups > MT;
  static constexpr int kStep = kTurns ? 2 : 1;                  // chunks from one of a group's to its next
  static constexpr int kAhead = MT == 2 ? 1 : 2;                // chunks whose scores run ahead of the products
  static constexpr bool kKLo = KF == MEMRA_KV_Q8_0;
  static constexpr bool kVLo = VF == MEMRA_KV_Q5_1 || VF == MEMRA_KV_Q4_0;
  // Staging warps in two groups that take the chunks by turns, each with K^ and V^ tiles of its own;
  // at head_dim 256, where shared memory holds two pairs of single values only, with NVFP4 for K, V or both
  // beside fp8 (12 sequences x 31 nodes over 3,000 keys, one group / two: fp8/nvfp4 46.5 / 44.8, nvfp4/fp8
  // 41.2 / 38.6, nvfp4/nvfp4 49.0 / 46.1 us; 1 x 32 over 65,536: 63.8 / 59.1, 53.9 / 48.3, 69.4 / 64.0), but
  // not with fp8 alone, whose staging is short (38.3 / 39.6 and 48.7 / 50.9; 8 x 8 over 4,104: 23.2 / 22.6).
  static constexpr bool kNv = KF == MEMRA_KV_NVFP4 || VF == MEMRA_KV_NVFP4;
  static constexpr int kStageGroups = D == 128 || (kNv && !kKLo && !kVLo) ? 2 : 1, kStageWarps = 8 / kStageGroups;
  static constexpr int kStageWarp0 = 4 * kGroups, kMmaWarp = kStageWarp0 + 8, kCopyWarp = kMmaWarp + 1;
  static constexpr int kThreads = 32 * (kCopyWarp + 1);
  static constexpr int kPages = kTreeKeys / kPage;
  static constexpr int kKSeg = k_seg_bytes(KF, D), kVSeg = v_seg_bytes(VF, D);
  // q5_1's d q + m as d (q - 16) and, in 16 more columns of V^, the blocks' centres m + 16 d (hi and lo
  // parts; the others zero), joined to O at the end: an exact d q + m in two fp16 parts costs ten
  // operations a pair, d (q - 16) three.  (Centres and not minima: the sums of d q and of m over a long
  // context are large and nearly cancel, and the float32 accumulators lose what is left.)  The MMA is
  // at most 256 wide, so at head_dim 256 the pair it is.
  static constexpr bool kMCols = VF == MEMRA_KV_Q5_1 && D == 128;
  static constexpr int kOCols = D + (D == 128 ? 16 : 0);
  static constexpr bool kVRows = VF != MEMRA_KV_NVFP4;          // V staged as token rows (MN-major)
  static constexpr uint32_t kTile = kTreeKeys * D * 2;
  static constexpr uint32_t kLoOff = kTile + (kMCols ? kTreeKeys * 128 : 0);      // V: hi, centres, lo
  static constexpr uint32_t kKBuf = kTile * (kKLo ? 2 : 1), kVBuf = kVLo ? kLoOff + kTile : kTile;
  static constexpr uint32_t kRawBytes = kPages * (kKSeg + kVSeg);
  // Q in tensor memory.  Two row tiles fill its 512 columns with 48 of Q, 144 of O and 64 of scores each:
  // Q's last 32 dims lie in shared memory.
  static constexpr int kQTmem = MT == 2 ? 96 : D, kQSmem = D - kQTmem;
  // Operand tiles in turn, so that staging runs ahead of the MMAs, where they fit.
  static constexpr int kKBufs = kStageGroups, kVBufs = kStageGroups == 2 || !kVLo ? 2 : 1;
  // barriers and page ids, then K^ and V^ tiles, Q's last dims and the raw chunks; the output rows reuse
  // everything behind the page ids
  static constexpr uint32_t kOffBar = 0, kOffPid = 256, kOffK = 4096;
  static constexpr uint32_t kOffV = kOffK + kKBufs * kKBuf, kOffQ = kOffV + kVBufs * kVBuf;
  static constexpr uint32_t kOffRaw = kOffQ + MT * kTileRows * kQSmem * 2;
  // chunks of raw pages in flight: as many as fit, four at most
  static constexpr uint32_t kRoom = 227 * 1024;
  static constexpr int kRaw = (kRoom - kOffRaw) / kRawBytes < 4 ? (kRoom - kOffRaw) / kRawBytes : 4;
  static constexpr uint32_t kEnd = kOffRaw + kRaw * kRawBytes;
  static constexpr uint32_t kRowBytes = D * 4 + 16;             // padded output row
  static constexpr uint32_t kOffMl = kOffK + MT * kTileRows * kRowBytes;          // (m, l) of two groups, at the end
  static constexpr uint32_t kEndRows = kOffMl + (kTurns ? 2 * kTileRows * 8 : 0);
  // Tensor memory: a CTA that found its columns taken would wait in its
  // allocation, so shared memory is sized that no more CTAs of this or the
  // library's other tensor-memory kernels fit an SM than its 512 columns hold.
  static constexpr uint32_t kTCols = 512;
  static constexpr uint32_t kNeed = kEnd > kEndRows ? kEnd : kEndRows, kFloor = 150 * 1024;
  static constexpr uint32_t kSmem = kNeed < kFloor ? kFloor : kNeed;
  // tensor-memory columns: Q of each row tile, O of each group, two score buffers
  static constexpr uint32_t kQCol = 0, kOCol = MT * kQTmem / 2, kSCol = kOCol + kGroups * kOCols;
  static_assert(kOffPid + 4 * kTreeSplitPages <= kOffK && kRaw >= 2, "page ids; a chunk ahead");
  static_assert(kOffBar + 8 * (2 * kRaw + 17) + 4 <= kOffPid, "barriers and the tensor-memory address");
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kSCol + 2 * kTreeKeys <= kTCols, "tensor memory");
  static_assert(kRawBytes % 16 == 0 && kOffRaw % 16 == 0 && kOffK % 1024 == 0 && kTile % 1024 == 0, "alignment");
};

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
template <int D, int KF, int KEYS, int WARPS>
__device__ __forceinline__ void stage_k(uint32_t raw, uint32_t buf, int warp, int lane) {
  constexpr int NB = D / 32, SEG = k_seg_bytes(KF, D), B2 = D / 64;
  constexpr uint32_t LO = KEYS * D * 2;
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
          sts128(buf + b2 * KEYS * 128 + (kPage * pg + t) * 128 + ((u ^ tg) << 4), h);
        }
    }
  } else {
    // run (page, token half, 64-dim block): 8 bytes for each of the two 32-dim blocks
    constexpr unsigned TASKS = KEYS / 8 * B2, STEP = WARPS / B2;     // a warp's token groups are STEP apart
    static_assert(TASKS % WARPS == 0 && WARPS % B2 == 0 && (STEP % 2 == 0 || STEP == 1), "whole tasks");
    const unsigned g0 = static_cast<unsigned>(warp) / B2, b2 = static_cast<unsigned>(warp) % B2;
    const bool odd = tg & 1;
    const uint32_t sel0 = odd ? 0x3232u : 0x1010u, sel1 = odd ? 0x1010u : 0x3232u;
    const uint32_t row = buf + b2 * (KEYS * 128) + (8 * g0 + tg) * 128;
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

// Bit c: the row whose word is `word` sees key tok0 + c; `off` = tok0 - (position of the tree's first row).
__device__ __forceinline__ uint64_t seen_keys(uint64_t word, int off) {
  return off <= -kTreeKeys ? ~0ull : off < 0 ? word << -off | ((1ull << -off) - 1ull) : word >> off;
}

// The keys of the chunk's pages whose bit is set.
__device__ __forceinline__ uint64_t page_keys(uint32_t pmask) {
  uint64_t keys = 0;
#pragma unroll
  for (int i = 0; i < kTreeKeys / kPage; ++i) keys |= (pmask >> i) & 1u ? 0xFFFFull << (kPage * i) : 0ull;
  return keys;
}

// Sequence length as the kernels use it.
__device__ __forceinline__ int tree_len(const TreeParams &p, int T) { return max(0, min(T, p.len_limit)); }

// Work item of the split pass.
struct TreeItem {
  int b, T, split, ns;    // b < 0: no such item
  int C;                  // chunks of a split wanted in this call
  int per;                // chunks of a split of this sequence
  bool bad;               // the sequence's length was out of range
};

// Item `index` of the call, by a whole warp from the sequences' lengths.
__device__ __forceinline__ TreeItem find_item(const TreeParams &p, int index, int lane) {
  TreeItem it{-1, 0, 0, 0, kTreeMaxChunks, 0, false};
  const int first = lane < p.batch ? p.seq_lens[lane] : 0;       // a short batch is read once
  const int first_chunks = tree_ceil(tree_len(p, first), kTreeKeys);
  // splits of a sequence, and the chunks of one
  auto splits = [&](int chunks, int &per) {
    per = tree_split_chunks(chunks, it.C);
    return max(1, tree_ceil(chunks, per));
  };
  int first_per = 0, first_ns = 0, C = kTreeMaxChunks;
  if (p.slots > 0) {
    auto chunks_of = [&](int b) { return tree_ceil(tree_len(p, p.seq_lens[b]), kTreeKeys); };
    int total = first_chunks;
    for (int b = 32 + lane; b < p.batch; b += 32) total += chunks_of(b);
    total = __reduce_add_sync(0xffffffffu, total);
    int places = p.slots;
    C = tree_ceil(total, places);
    if (C > kTreeMaxChunks) {
      places *= tree_ceil(C, kTreeMaxChunks);
      C = tree_ceil(total, places);
    }
    C = min(max(C, kTreeMinChunks), kTreeMaxChunks);
    // Each sequence's last split takes a place however short it is: C grows until all fit.
    for (int trial = 0;; ++trial) {
      it.C = C;
      first_ns = splits(first_chunks, first_per);
      if (trial == kTreeTrials || C == kTreeMaxChunks) break;
      int items = lane < p.batch ? first_ns : 0, per;
      for (int b = 32 + lane; b < p.batch; b += 32) items += splits(chunks_of(b), per);
      const int over = __reduce_add_sync(0xffffffffu, items) - places;
      if (over <= 0 || over >= places) break;
      C = min(max(tree_ceil(total, places - over), C + 1), kTreeMaxChunks);
    }
  } else {
    first_ns = splits(first_chunks, first_per);
  }
  int start = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    const int b = b0 + lane, T0 = b0 == 0 ? first : b < p.batch ? p.seq_lens[b] : 0, T = tree_len(p, T0);
    int per = first_per, ns = first_ns;
    if (b0 > 0) ns = splits(tree_ceil(T, kTreeKeys), per);
    if (b >= p.batch) ns = 0;
    int incl = ns;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += up;
    }
    const int at = index - start - (incl - ns);
    const unsigned who = __ballot_sync(0xffffffffu, at >= 0 && at < ns);
    if (who) {
      const int src = __ffs(who) - 1;
      it.b = b0 + src;
      it.T = __shfl_sync(0xffffffffu, T, src);
      it.ns = __shfl_sync(0xffffffffu, ns, src);
      it.per = __shfl_sync(0xffffffffu, per, src);
      it.split = __shfl_sync(0xffffffffu, at, src);
      it.bad = __shfl_sync(0xffffffffu, T != T0 || T0 < p.n_nodes, src);
      break;
    }
    start += __shfl_sync(0xffffffffu, incl, 31);
  }
  return it;
}

template <int D, int KF, int VF, int MT>
__global__ void __launch_bounds__(TreeCfg<D, KF, VF, MT>::kThreads, 1)
    tree_kernel(const TreeParams p) {
  using C = TreeCfg<D, KF, VF, MT>;
  constexpr int KT = kTreeKeys, NP = C::kPages, RAW = C::kRaw, SW = C::kStageWarps;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bars = sb + C::kOffBar;
  auto raw_full = [&](int s) { return bars + 8 * s; };
  auto raw_empty = [&](int s) { return bars + 8 * (RAW + s); };
  enum { kKFull = 0, kKEmpty, kVFull, kVEmpty, kSFull, kPFull };
  auto bar = [&](int kind, int b) { return bars + 8 * (2 * RAW + 2 * kind + b); };
  auto pv_done = [&](int i) { return bars + 8 * (2 * RAW + 12 + i); };
  auto q_ready = [&](int i) { return bars + 8 * (2 * RAW + 14 + i); };
  const uint32_t drained = bars + 8 * (2 * RAW + 16);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffBar + 8 * (2 * RAW + 17));
  int *pid_s = reinterpret_cast<int *>(smem + C::kOffPid);

  grid_dependency_wait();
  allow_dependent_launch();
  // Items outermost: the CTAs past the last item come last, so that the others
  // fill the SMs evenly, and those of one split's pages run side by side.
  const int side = p.n_kv_heads * p.row_ctas, index = blockIdx.x / side;
  const int kvh = blockIdx.x % side / p.row_ctas, r0 = blockIdx.x % p.row_ctas * (MT * kTileRows);
  const int rows = p.n_nodes * p.group;
  // This CTA's sequence and split: items are numbered sequence by sequence
  // (one at least each).  Every warp finds it for itself.
  const TreeItem item = find_item(p, index, lane);
  const int b = item.b, T = item.T, ns = item.ns;
  if (blockIdx.x == 0 && tid == 0) *p.plan = item.C;
  if (b < 0) return;                         // fewer items than the grid's bound
  if (item.split == 0 && kvh == 0 && r0 == 0 && tid == 0 && item.bad) flag_error(p.status, MEMRA_DEVERR_BAD_SEQ_LEN);
  // Global row of row r of this KV head: node r / group, head r % group of the group.
  auto row_id = [&](int r) {
    return (static_cast<size_t>(b) * p.n_nodes + r / p.group) * p.n_heads + kvh * p.group + r % p.group;
  };
  if (T <= 0) {                              // no key at all: zeros
    for (int i = tid; i < min(MT * kTileRows, rows - r0) * (D / 8); i += C::kThreads)
      *reinterpret_cast<uint4 *>(p.out + row_id(r0 + i / (D / 8)) * D + 8 * (i % (D / 8))) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int split_len = item.per * KT, first = item.split * split_len, count = min(T - first, split_len);
  const int n_chunks = (count + KT - 1) / KT, n_pages = (count + kPage - 1) / kPage;
  // Page id of a page of the split, -1 for one left out or past the end.
  const int32_t *table = p.page_table + static_cast<size_t>(b) * p.max_pages + first / kPage;
  auto page_id = [&](int i) {
    if (i >= n_pages) return -1;
    const int pid = table[i];
    return pid >= 0 && pid < p.num_pages ? pid : -1;
  };
  // The copy warp sets the barriers up and sends for the first chunks while the others prepare.
  // Lane = (page of a chunk, K or V): one copy each, issued together (from one
  // thread the eight copies of a chunk took 1,600 clocks to issue).
  const int cp_page = lane >> 1;
  const bool cp_v = lane & 1;
  const uint32_t cp_bytes = cp_v ? C::kVSeg : C::kKSeg;
  auto copy_chunk = [&](int ci, int pid) {
    const int s = ci % RAW, n = __popc(__ballot_sync(0xffffffffu, pid >= 0)) / 2;
    if (lane == 0) {
      if (n)
        mbar_arrive_expect_tx(raw_full(s),
                              n * (C::kKSeg + C::kVSeg) + (ci == 0 && blockIdx.x == 0 ? p.test_extra_tx : 0));
      else
        mbar_arrive(raw_full(s));
    }
    __syncwarp();
    if (pid >= 0)
      bulk_copy_g2s_nohint(sb + C::kOffRaw + s * C::kRawBytes + (cp_v ? NP * C::kKSeg : 0) + cp_page * cp_bytes,
                           (cp_v ? p.v_pool : p.k_pool) + (static_cast<size_t>(pid) * p.n_kv_heads + kvh) * cp_bytes,
                           cp_bytes, raw_full(s));
  };
  int bad = 0;
  if (warp == C::kCopyWarp) {
    int pid[RAW];
#pragma unroll
    for (int ci = 0; ci < RAW; ++ci) pid[ci] = cp_page < NP ? page_id(ci * NP + cp_page) : -1;
    if (lane == 0) {
      for (int s = 0; s < RAW; ++s) {
        mbar_init(raw_full(s), 1);
        mbar_init(raw_empty(s), SW);
      }
      for (int k = 0; k < 2; ++k) {
        mbar_init(bar(kKFull, k), SW);
        mbar_init(bar(kKEmpty, k), 1);
        mbar_init(bar(kVFull, k), SW);
        mbar_init(bar(kVEmpty, k), 1);
        mbar_init(bar(kSFull, k), 1);
        mbar_init(bar(kPFull, k), 4);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(pv_done(i), 1);
        mbar_init(q_ready(i), 4);
      }
      mbar_init(drained, 1);
      fence_barrier_init();
    }
    __syncwarp();
#pragma unroll
    for (int ci = 0; ci < RAW; ++ci)
      if (ci < n_chunks) copy_chunk(ci, pid[ci]);
  } else {
    for (int i = tid; i < n_chunks * NP; i += 32 * C::kCopyWarp) {
      const int pid = page_id(i);
      pid_s[i] = pid;
      if (pid < 0 && i < n_pages) {
        flag_error(p.status, MEMRA_DEVERR_BAD_PAGE);
        bad = 1;
      }
    }
    if (warp == C::kMmaWarp) {
      tc::tmem_alloc(smem_addr(tmem_slot), C::kTCols);
      tc::tmem_relinquish();
    }
  }
  tc::fence_before_sync();
  bad = __syncthreads_or(bad);
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  // The chunk's pages, one bit each, without those left out (rows past the end are masked by position).
  auto chunk_mask = [&](int ci) {
    uint32_t m = (1u << NP) - 1u;
    if (bad) {
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (ci * NP + i < n_pages && pid_s[ci * NP + i] < 0) m &= ~(1u << i);
    }
    return m;
  };
  bool ok = true;

  if (warp == C::kCopyWarp) {
    // ----------------------------------------------------------------- copies --
    int issued = min(n_chunks, RAW);
    for (int ci = RAW; ci < n_chunks; ++ci) {
      const int pid = cp_page < NP ? pid_s[ci * NP + cp_page] : -1;
      ok = mbar_wait_suspended(raw_empty(ci % RAW), (ci / RAW - 1) & 1, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      copy_chunk(ci, pid);
      issued = ci + 1;
    }
    // every copy has landed before the CTA can leave
    for (int ci = max(0, issued - RAW); ci < issued; ++ci)
      mbar_wait_suspended(raw_full(ci % RAW), (ci / RAW) & 1, p.status);
    __syncwarp();
  } else if (warp == C::kMmaWarp) {
    // -------------------------------------------------------------------- MMA --
    if (tc::elect_one()) {
      constexpr uint32_t idesc_s = tc::idesc_f16_f32(kTileRows, KT);
      constexpr uint32_t idesc_o = C::kVRows ? tc::idesc_f16_f32_bmn(kTileRows, D) : tc::idesc_f16_f32(kTileRows, D);
      constexpr uint32_t idesc_oc = C::kMCols ? tc::idesc_f16_f32_bmn(kTileRows, C::kOCols) : idesc_o;
      auto wait = [&](int kind, int k, int phase) {
        ok = ok && mbar_wait_suspended(bar(kind, k), phase & 1, p.status);
      };
      // Score buffer and barrier of row tile i at chunk ci; its O.
      auto buf = [](int i, int ci) { return MT == 2 ? i : ci & 1; };
      auto group = [](int i, int ci) { return C::kTurns ? ci & 1 : i; };
      // S_i(ci) = Q_i K^T
      auto mma_s = [&](int i, int ci) {
        if (!ok || ci >= n_chunks) return;
        const int kb = ci % C::kKBufs, sk = buf(i, ci);
        wait(kKFull, kb, ci / C::kKBufs);
        if (!ok) return;
        tc::fence_after_sync();
        const uint32_t d = tmem + C::kSCol + sk * KT;
        const uint64_t kd = tc::smem_desc_sw128(sb + C::kOffK + kb * C::kKBuf, 16, 1024);
        const uint64_t qd = tc::smem_desc(sb + C::kOffQ + i * kTileRows * C::kQSmem * 2, 128, C::kQSmem / 8 * 128);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
          for (int lo = 0; lo < (C::kKLo ? 2 : 1); ++lo) {
            const uint64_t bd = tc::desc_at(kd, (ks / 4) * KT * 128 + (ks % 4) * 32 + lo * C::kTile);
            if (16 * ks < C::kQTmem)
              tc::mma_f16_ta(d, tmem + C::kQCol + i * (C::kQTmem / 2) + 8 * ks, bd, idesc_s, ks + lo > 0);
            else
              tc::mma_f16(d, tc::desc_at(qd, 256 * (ks - C::kQTmem / 16)), bd, idesc_s, 1);
          }
        }
        if (i == MT - 1) tc::commit(bar(kKEmpty, kb));
        tc::commit(bar(kSFull, sk));
      };
      // O_i += P_i(ci) V, P in the columns of its scores
      auto mma_o = [&](int i, int ci) {
        if (!ok) return;
        const int vb = ci % C::kVBufs, sk = buf(i, ci);
        wait(kPFull, sk, ci / C::kAhead);
        wait(kVFull, vb, ci / C::kVBufs);
        if (!ok) return;
        tc::fence_after_sync();
        const uint32_t v = sb + C::kOffV + vb * C::kVBuf, a = tmem + C::kSCol + sk * KT;
        const uint32_t d = tmem + C::kOCol + group(i, ci) * C::kOCols;
        const uint64_t vd = C::kVRows ? tc::smem_desc_sw128(v, KT * 128, 1024) : tc::smem_desc(v, 128, (KT / 8) * 128);
        constexpr uint32_t kStep = C::kVRows ? 2048 : 256;       // a K = 16 step further on
#pragma unroll
        for (int ks = 0; ks < KT / 16; ++ks) {
          tc::mma_f16_ta(d, a + 8 * ks, tc::desc_at(vd, kStep * ks), idesc_oc, ci >= C::kStep || ks > 0);
          if constexpr (C::kVLo) tc::mma_f16_ta(d, a + 8 * ks, tc::desc_at(vd, kStep * ks + C::kLoOff), idesc_o, 1);
        }
        if (i == MT - 1) tc::commit(bar(kVEmpty, vb));
        if (C::kGroups == 1 || ci + C::kStep >= n_chunks) tc::commit(pv_done(group(i, ci)));
      };
#pragma unroll
      for (int i = 0; i < C::kGroups; ++i) ok = ok && mbar_wait_suspended(q_ready(i), 0, p.status);
      for (int ci = 0; ci < C::kAhead; ++ci)
#pragma unroll
        for (int i = 0; i < MT; ++i) mma_s(i, ci);
      for (int ci = 0; ci < n_chunks && ok; ++ci)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          mma_o(i, ci);
          mma_s(i, ci + C::kAhead);          // behind the product that reads its buffer's P
        }
      tc::commit(drained);                   // what was issued completes before the CTA can leave
      mbar_wait_suspended(drained, 0, p.status);
    }
    __syncwarp();
  } else if (warp >= C::kStageWarp0) {
    // ---------------------------------------------------------------- staging --
    const int sg = (warp - C::kStageWarp0) / SW, sw = (warp - C::kStageWarp0) % SW, st = 32 * sw + lane;
    if constexpr (C::kMCols) {               // the unused columns of the centres' block, once
      for (int vb = sg; vb < C::kVBufs; vb += C::kStageGroups)
        for (uint32_t i = st; i < KT * 8u; i += 32 * SW)
          sts128(sb + C::kOffV + vb * C::kVBuf + C::kTile + 16 * i, make_uint4(0, 0, 0, 0));
      named_barrier_sync(1 + sg, 32 * SW);
    }
    // the words of all nodes together, for a split that holds rows of the tree
    const int base = T - p.n_nodes;
    uint64_t named = 0;
    if (first + n_chunks * KT > base) {
      for (int j = lane; j < p.n_nodes; j += 32)
        if (base + j >= 0) named |= p.mask[static_cast<size_t>(b) * p.n_nodes + j];
      const uint32_t lower = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(named));
      const uint32_t upper = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(named >> 32));
      named = static_cast<uint64_t>(upper) << 32 | lower;
    }
    for (int ci = sg; ci < n_chunks; ci += C::kStageGroups) {
      const int s = ci % RAW, kb = ci % C::kKBufs, vb = ci % C::kVBufs, valid = count - ci * KT;
      const uint32_t rawk = sb + C::kOffRaw + s * C::kRawBytes, rawv = rawk + NP * C::kKSeg;
      // (K^'s tile first: that its last scores are done says that the chunk RAW before this one has landed,
      // so that the raw chunk's parity names this use of its place and not the one two before)
      if (ci >= C::kKBufs) ok = mbar_wait_suspended(bar(kKEmpty, kb), (ci / C::kKBufs - 1) & 1, p.status);
      if (ok) ok = mbar_wait_suspended(raw_full(s), (ci / RAW) & 1, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      stage_k<D, KF, KT, SW>(rawk, sb + C::kOffK + kb * C::kKBuf, sw, lane);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kKFull, kb));
      if (ci >= C::kVBufs) ok = mbar_wait_suspended(bar(kVEmpty, vb), (ci / C::kVBufs - 1) & 1, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t vbuf = sb + C::kOffV + vb * C::kVBuf;
      // Tokens that any row may see; not those of a page left out, nor rows of the tree that no word names:
      // they need not have been written.
      uint64_t keep = valid < KT ? (1ull << valid) - 1ull : ~0ull;
      if (first + (ci + 1) * KT > base) keep &= seen_keys(named, first + ci * KT - base);
      if (bad) keep &= page_keys(chunk_mask(ci));
      if constexpr (C::kVRows)
        stage_v<D, VF, KT, SW, C::kMCols, C::kLoOff>(rawv, vbuf, keep, sw, lane);
      else
        stage_v_nvfp4<D, KT, SW>(rawv, vbuf, keep, st);
      if constexpr (C::kMCols) {             // 32 tokens by each of two warps, other ones each time
        const int part = (sw - 2 * ci) & (SW - 1);
        if (part < KT / 32) stage_m<D, KT>(rawv, vbuf + C::kTile, keep, 32 * part + lane);
      }
      fence_proxy_async();                   // V^ for the tensor cores, the raw chunk for the next copies
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kVFull, vb));
        mbar_arrive(raw_empty(s));
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax --
    const int g = warp >> 2, i = MT == 2 ? g : 0, rl = tid & 127;  // group, row tile, row in it
    const uint32_t tlane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int r = r0 + i * kTileRows + rl;
    const bool live = r < rows;
    uint64_t word = 0;
    if (live && T - p.n_nodes + r / p.group >= 0) word = p.mask[static_cast<size_t>(b) * p.n_nodes + r / p.group];
    if (p.n_nodes < 64) word &= (1ull << p.n_nodes) - 1ull;
    {
      // the row of Q (negated for a negative scale, zeros for scale 0: the softmax takes the largest
      // score for the largest weight): fp16 pairs into tensor memory, the last dims into core matrices
      const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (live ? row_id(r) : 0) * D);
      auto load = [&](int u) {
        const uint4 y = live ? src[u] : make_uint4(0, 0, 0, 0);
        return make_uint4((y.x & p.q_and) ^ p.q_xor, (y.y & p.q_and) ^ p.q_xor, (y.z & p.q_and) ^ p.q_xor,
                          (y.w & p.q_and) ^ p.q_xor);
      };
#pragma unroll
      for (int c = 0; c < C::kQTmem / 2; c += 16) {
        if (C::kTurns && g != (c >= 32)) continue;               // half of the row by each group
        uint32_t x[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 y = load(c / 4 + e);
          x[4 * e] = y.x, x[4 * e + 1] = y.y, x[4 * e + 2] = y.z, x[4 * e + 3] = y.w;
        }
        tc::st_32x32b_x16(tmem + tlane + C::kQCol + i * (C::kQTmem / 2) + c, x);
      }
#pragma unroll
      for (int u = 0; u < C::kQSmem / 8; ++u)
        sts128(sb + C::kOffQ + i * kTileRows * C::kQSmem * 2 + ((rl >> 3) * (C::kQSmem / 8) + u) * 128 + (rl & 7) * 16,
               load(C::kQTmem / 8 + u));
    }
    tc::wait_st();
    fence_proxy_async();
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_ready(g));
    const int base = T - p.n_nodes;          // position of the tree's first row
    const uint32_t o_col = tmem + tlane + C::kOCol + g * C::kOCols;
    float m = -INFINITY, l = 0.f;
#pragma unroll 1
    for (int ci = C::kTurns ? g : 0; ci < n_chunks; ci += C::kStep) {
      const uint32_t pmask = chunk_mask(ci);
      const int tok0 = first + ci * KT, sk = MT == 2 ? i : ci & 1;
      const uint32_t s_col = tmem + tlane + C::kSCol + sk * KT;
      ok = mbar_wait_suspended(bar(kSFull, sk), (ci / C::kAhead) & 1, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc::fence_after_sync();
      uint32_t s[KT];
#pragma unroll
      for (int c = 0; c < KT; c += 32) tc::ld_32x32b_x32(s_col + c, s + c);
      tc::wait_ld_all();
      tc::hold<KT>(s);
      if (pmask != (1u << NP) - 1u || tok0 + KT > base) {
        // bit c: the row sees key tok0 + c.  Keys before the tree, then the tree's by the word (whose
        // bits past the tree are cleared, so rows past the end are hidden too).
        const uint64_t sees = seen_keys(word, tok0 - base) & page_keys(pmask);
        const uint32_t half[2] = {static_cast<uint32_t>(sees), static_cast<uint32_t>(sees >> 32)};
#pragma unroll
        for (int c = 0; c < KT; ++c)
          if (!(half[c / 32] & (1u << (c % 32)))) s[c] = 0xff800000u;      // -inf
      }
      const float top = row_max(s) * p.scale_log2;
      float alpha = 1.f;
      if (top > m + kLazy) {                 // also the first chunk with a key (m = -inf)
        if (m != -INFINITY) alpha = fast_exp2(m - top);
        m = top;
      }
      const bool moved = ci >= C::kStep && __any_sync(0xffffffffu, alpha != 1.f);
      if (C::kGroups == 1 && ci > 0 && (moved || ci == n_chunks - 1)) {
        // The product before has completed, O is still (a group of two: these scores were issued behind it).
        // At the last chunk in any case: the wait behind the loop names the last product by its
        // parity, which the product two before has too.
        ok = mbar_wait_suspended(pv_done(i), (ci - 1) & 1, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc::fence_after_sync();
      }
      if (moved) {                           // O's rows of this warp times alpha
#pragma unroll 1
        for (int c = 0; c < C::kOCols; c += 16) {
          uint32_t o[16];
          tc::ld_32x32b_x16(o_col + c, o);
          tc::wait_ld(o);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tc::st_32x32b_x16(o_col + c, o);
        }
        l *= alpha;
      }
      const float mu = m == -INFINITY ? 0.f : m;
      uint64_t sum = 0;
#pragma unroll
      for (int c = 0; c < KT; c += 32) {
        uint32_t w[16];
        row_weights<16>(s + c, p.scale_log2, mu, w, sum);
        tc::st_32x32b_x16(s_col + c / 2, w);
      }
      float l0, l1;
      unpack_f2(sum, l0, l1);
      l += l0 + l1;
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kPFull, sk));
    }
    if constexpr (C::kGroups == 1) {
      if (ok) ok = mbar_wait_suspended(pv_done(0), (n_chunks - 1) & 1, p.status);
    } else {
      // the other group's last product too: it reads the operand tiles, and its O is joined to this one
      for (int e = 0; e < 2; ++e)
        if (ok && (!C::kTurns || e < n_chunks)) ok = mbar_wait_suspended(pv_done(e), 0, p.status);
    }
    // A length out of range (flagged) reads rows that nobody may have written: what they make of a row is left out.
    if (item.bad && !(l > 0.f)) l = 0.f;
    // (every MMA is done: the operand tiles and raw pages are free for the output rows)
    ok = __all_sync(0xffffffffu, ok);
    tc::fence_after_sync();
    // O = sum of w[e] O_e over the row's groups
    float w[C::kStep];
    if constexpr (C::kTurns) {
      // this group's (m, l) for the other
      const uint32_t ml = sb + C::kOffMl + rl * 8;
      sts64(ml + g * kTileRows * 8, __float_as_uint(m), __float_as_uint(l));
      named_barrier_sync(3, 32 * 8);
      const float m1 = __uint_as_float(lds32(ml + (g ^ 1) * kTileRows * 8));
      const float l1 = __uint_as_float(lds32(ml + (g ^ 1) * kTileRows * 8 + 4));
      // (a sum of NaN, from a query or a key that is not finite, is no empty one: the row becomes NaN)
      const float top = fmaxf(m, m1);
      const float mine = l != 0.f ? fast_exp2(m - top) : 0.f, other = l1 != 0.f ? fast_exp2(m1 - top) : 0.f;
      w[0] = g ? other : mine, w[C::kStep - 1] = g ? mine : other;
      l = l * mine + l1 * other;
      m = top;
    } else {
      w[0] = l != 0.f ? 1.f : 0.f;
    }
    const float inv = l != 0.f ? p.v_post / l : 0.f;
#pragma unroll
    for (int e = 0; e < C::kStep; ++e) w[e] *= inv;
    const uint32_t o_cols = C::kTurns ? tmem + tlane + C::kOCol : o_col;         // of the row's first group
    uint32_t ms[C::kStep][16];               // the centres' sums, per 32-dim block: hi parts, lo parts
    if constexpr (C::kMCols) {
#pragma unroll
      for (int e = 0; e < C::kStep; ++e) {
        tc::ld_32x32b_x16(o_cols + e * C::kOCols + D, ms[e]);
        tc::wait_ld(ms[e]);
      }
    }
    const uint32_t row = sb + C::kOffK + (i * kTileRows + rl) * C::kRowBytes;
#pragma unroll
    for (int c0 = 0; c0 < D / C::kStep; c0 += 16) {              // (by turns: half of the columns each)
      if (!ok) break;
      const int c = C::kTurns ? g * (D / 2) + c0 : c0;
      float x[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = 0.f;
#pragma unroll
      for (int k = 0; k < C::kStep; ++k) {
        uint32_t o[16];
        tc::ld_32x32b_x16(o_cols + k * C::kOCols + c, o);
        tc::wait_ld(o);
        float centre = 0.f;
        if constexpr (C::kMCols) {
          const float lower = __uint_as_float(ms[k][c0 / 32]) + __uint_as_float(ms[k][4 + c0 / 32]);
          centre = lower;
          if constexpr (C::kTurns) {
            const float upper = __uint_as_float(ms[k][2 + c0 / 32]) + __uint_as_float(ms[k][6 + c0 / 32]);
            centre = g ? upper : lower;
          }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e)         // (a group without a visible key: its O may hold anything)
          x[e] = w[k] != 0.f ? fmaf(__uint_as_float(o[e]) + centre, w[k], x[e]) : x[e];
      }
      if (ns == 1) {
#pragma unroll
        for (int e = 0; e < 16; e += 8)
          sts128(row + (c + e) * 2, make_uint4(pack_half2(x[e], x[e + 1]), pack_half2(x[e + 2], x[e + 3]),
                                               pack_half2(x[e + 4], x[e + 5]), pack_half2(x[e + 6], x[e + 7])));
      } else {
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          sts128(row + (c + e) * 4, make_uint4(__float_as_uint(x[e]), __float_as_uint(x[e + 1]),
                                               __float_as_uint(x[e + 2]), __float_as_uint(x[e + 3])));
      }
    }
    // The rows to memory, each by a whole warp (a bulk copy per row took 100 clocks
    // to issue, 32 of them one after another).
    constexpr int WR = 32 / C::kStep;        // rows of a warp
    const int wr = r0 + WR * warp + lane;
    const int64_t id = lane < WR && wr < rows ? static_cast<int64_t>(row_id(wr)) : -1;
    if constexpr (C::kTurns)
      ok = named_barrier_and(3, 32 * 8, ok);         // both halves of the rows are there
    else
      __syncwarp();
    if (live && ns > 1 && (!C::kTurns || g == 0))                // -inf, never weighed, without a visible key
      p.lse_part[static_cast<int64_t>(row_id(r)) * p.max_splits + item.split] =
          !ok ? __uint_as_float(kNanPair) : l != 0.f ? m + __log2f(l) : -INFINITY;
    const uint32_t row0 = sb + C::kOffK + warp * WR * C::kRowBytes;
    constexpr int BATCH = 8;                 // rows in flight
    // 16-byte units of a row, a row's address; NaN after a wait that gave up
    auto write_rows = [&](auto units, auto to_row) {
      constexpr int U = decltype(units)::value;
#pragma unroll 1
      for (int e0 = 0; e0 < WR; e0 += BATCH) {
        uint4 x[BATCH][(U + 31) / 32];
#pragma unroll
        for (int e = 0; e < BATCH; ++e)
#pragma unroll
          for (int c = 0; c < U; c += 32)
            if (U >= 32 || lane < U)
              x[e][c / 32] = ok ? lds128(row0 + (e0 + e) * C::kRowBytes + (c + lane) * 16)
                                : make_uint4(kNanPair, kNanPair, kNanPair, kNanPair);
#pragma unroll
        for (int e = 0; e < BATCH; ++e) {
          const int64_t to = __shfl_sync(0xffffffffu, id, e0 + e);
#pragma unroll
          for (int c = 0; c < U; c += 32)
            if (to >= 0 && (U >= 32 || lane < U)) to_row(to)[c + lane] = x[e][c / 32];
        }
      }
    };
    if (ns == 1)
      write_rows(std::integral_constant<int, D / 8>{}, [&](int64_t to) { return reinterpret_cast<uint4 *>(p.out + to * D); });
    else
      write_rows(std::integral_constant<int, D / 4>{}, [&](int64_t to) {
        return reinterpret_cast<uint4 *>(p.o_part + (to * p.max_splits + item.split) * D);
      });
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == C::kMmaWarp) tc::tmem_dealloc(tmem, C::kTCols);
}

// Merge of a row's partials: warp = row, each lane D / 32 consecutive outputs.
constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) tree_merge_kernel(const TreeParams p) {
  constexpr int PER = D / 32, BATCH = 8;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5);
  const int64_t per_seq = static_cast<int64_t>(p.n_nodes) * p.n_heads;
  allow_dependent_launch();
  if (row >= p.batch * per_seq) return;
  const int chunks = tree_ceil(tree_len(p, p.seq_lens[row / per_seq]), kTreeKeys);
  const float *lse = p.lse_part + row * p.max_splits;
  const float *src = p.o_part + row * p.max_splits * D + lane * PER;
  float mw = -INFINITY, L = 0.f, acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  grid_dependency_wait();                    // the partials and the plan are complete
  // BATCH partials in flight.  The first ones are read before the plan says how
  // many there are: what is behind them is never weighed.
  int ns = p.max_splits;
  for (int k0 = 0; k0 < ns; k0 += BATCH) {
    float ls[BATCH];
    float4 x[BATCH][PER / 4];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const bool in = k0 + u < ns;
      ls[u] = in ? lse[k0 + u] : -INFINITY;
      const float4 *at = reinterpret_cast<const float4 *>(src + static_cast<size_t>(in ? k0 + u : 0) * D);
#pragma unroll
      for (int e = 0; e < PER / 4; ++e) x[u][e] = in ? at[e] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (k0 == 0) {
      ns = tree_ceil(chunks, tree_split_chunks(chunks, *p.plan));
      if (ns <= 1) return;                   // the split pass wrote this row
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      if (k0 + u >= ns || ls[u] == -INFINITY) continue;      // its row may hold anything
      if (ls[u] > mw) {
        const float sc = fast_exp2(mw - ls[u]);
        L *= sc;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] *= sc;
        mw = ls[u];
      }
      const float w = fast_exp2(ls[u] - mw);
      L += w;
#pragma unroll
      for (int e = 0; e < PER / 4; ++e) {
        acc[4 * e + 0] = fmaf(w, x[u][e].x, acc[4 * e + 0]);
        acc[4 * e + 1] = fmaf(w, x[u][e].y, acc[4 * e + 1]);
        acc[4 * e + 2] = fmaf(w, x[u][e].z, acc[4 * e + 2]);
        acc[4 * e + 3] = fmaf(w, x[u][e].w, acc[4 * e + 3]);
      }
    }
  }
  const float inv = L != 0.f ? 1.f / L : 0.f;          // (0: no visible key; a NaN stays one)
  uint32_t y[PER / 2];
#pragma unroll
  for (int e = 0; e < PER / 2; ++e) y[e] = pack_half2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  __half *dst = p.out + row * D + lane * PER;
  if constexpr (PER == 4)
    *reinterpret_cast<uint2 *>(dst) = make_uint2(y[0], y[1]);
  else
    *reinterpret_cast<uint4 *>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
}

template <int D, int KF, int VF, int MT>
cudaError_t launch_one(const TreeParams &p, cudaStream_t st) {
  using C = TreeCfg<D, KF, VF, MT>;
  auto kernel = tree_kernel<D, KF, VF, MT>;
  static bool ready[64] = {};                // the shared-memory limit, set once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  // Items of the call at most: the waves' worth and one more per sequence; and
  // no sequence has more than the longest can have.
  const int64_t chunks = p.batch * static_cast<int64_t>(tree_ceil(p.max_seq_len, kTreeKeys));
  const int64_t per_wave = static_cast<int64_t>(std::max(p.slots, 1)) * kTreeMaxChunks;
  const int64_t items = std::min<int64_t>(
      p.batch + std::max(p.slots, 1) * std::max<int64_t>((chunks + per_wave - 1) / per_wave, 1),
      static_cast<int64_t>(p.batch) * std::max(1, p.max_splits));
  const int64_t ctas = items * p.n_kv_heads * p.row_ctas;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(ctas));
  return launch_pdl(kernel, grid, dim3(C::kThreads), C::kSmem, st, p);
}

template <int D, int KF, int VF>
cudaError_t launch_tiles(const TreeParams &p, cudaStream_t st) {
  if constexpr (D == 128)
    if (tree_tiles(D, p.n_nodes * p.group) == 2) return launch_one<D, KF, VF, 2>(p, st);
  return launch_one<D, KF, VF, 1>(p, st);
}

template <int D>
cudaError_t launch_formats(int kf, int vf, const TreeParams &p, cudaStream_t st) {
  auto by_v = [&](auto kc) -> cudaError_t {
    constexpr int K = decltype(kc)::value;
    switch (vf) {
      case MEMRA_KV_Q5_1: return launch_tiles<D, K, MEMRA_KV_Q5_1>(p, st);
      case MEMRA_KV_Q4_0: return launch_tiles<D, K, MEMRA_KV_Q4_0>(p, st);
      case MEMRA_KV_FP8_E4M3: return launch_tiles<D, K, MEMRA_KV_FP8_E4M3>(p, st);
      case MEMRA_KV_NVFP4: return launch_tiles<D, K, MEMRA_KV_NVFP4>(p, st);
      default: return cudaErrorInvalidValue;
    }
  };
  switch (kf) {
    case MEMRA_KV_Q8_0: return by_v(std::integral_constant<int, MEMRA_KV_Q8_0>{});
    case MEMRA_KV_FP8_E4M3: return by_v(std::integral_constant<int, MEMRA_KV_FP8_E4M3>{});
    case MEMRA_KV_NVFP4: return by_v(std::integral_constant<int, MEMRA_KV_NVFP4>{});
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_tree(int D, int kf, int vf, const TreeParams &p, cudaStream_t st) {
  return D == 128 ? launch_formats<128>(kf, vf, p, st) : launch_formats<256>(kf, vf, p, st);
}

cudaError_t launch_tree_merge(int D, const TreeParams &p, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(p.batch) * p.n_nodes * p.n_heads;
  const dim3 grid(static_cast<unsigned>((rows + kMergeWarps - 1) / kMergeWarps));
  if (D == 128) return launch_pdl(tree_merge_kernel<128>, grid, dim3(32 * kMergeWarps), 0, st, p);
  return launch_pdl(tree_merge_kernel<256>, grid, dim3(32 * kMergeWarps), 0, st, p);
}

}  // namespace memra
