// Tree attention: a tree of up to 64 drafted nodes per sequence against the
// block-quantized paged cache.  Node i sees every key before the tree's rows
// and, of the tree's own, those whose bit its mask word holds:
//
//   o_i = sum_u p_iu V^_u / sum_u p_iu,  p_iu = 2^(q_i . K^_u * scale * log2(e) - m_i)
//
// The rows of one KV head, nodes x the group's query heads, 128 to a tile, are
// the M side of tcgen05 MMAs, so a page is read and dequantized once for all of
// them (twice or more only past 256 rows).  CTA = (split of the keys, KV head,
// sequence and row tiles):
//   * a producer thread copies raw pages into a ring of three chunks;
//   * eight staging warps dequantize a chunk's K and V into double-buffered
//     fp16 operand tiles (core-matrix order): exact hi + lo pairs for q8_0,
//     q5_1 and q4_0, single values for fp8 and NVFP4 (kv_stage.cuh), so only P
//     is rounded (fp16, relative 2^-11 a weight);
//   * one MMA thread: S = Q K^T with Q in tensor memory, O += P V with P in
//     tensor memory over its scores; neither A operand touches shared memory,
//     whose bandwidth the staged tiles need;
//   * four softmax warps, thread = row (of each tile in turn).
// One tile: two score buffers, the scores run a chunk ahead.  Two tiles
// (head_dim 128): one buffer each, the tensor cores work on one tile while the
// softmax takes the other.
// A sequence of one split writes its rows directly; the others leave (o, lse)
// partials that tree_merge_kernel joins.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "kv_stage.cuh"
#include "tcgen05.cuh"
#include "tree.cuh"

namespace memra {
namespace {

constexpr int kTileRows = 128;
constexpr float kLazy = 8.f;               // log2 units: P stays <= 256 between rescales
constexpr int kStageWarps = 8;
constexpr int kStageThreads = 32 * kStageWarps;
constexpr int kMmaWarp = 4 + kStageWarps, kCopyWarp = kMmaWarp + 1;
constexpr int kTreeThreads = 32 * (kCopyWarp + 1);
constexpr int kRaw = 3;                    // chunks of raw pages

template <int D, int KF, int VF, int MT>
struct TreeCfg {
  static constexpr int kKeys = tree_chunk_tokens(D);
  static constexpr int kPages = kKeys / kPage;
  static constexpr int kBufs = MT == 1 ? 2 : 1;                 // score buffers of a tile
  static constexpr bool kKLo = KF == MEMRA_KV_Q8_0;
  static constexpr bool kVLo = VF == MEMRA_KV_Q5_1 || VF == MEMRA_KV_Q4_0;
  static constexpr int kKSeg = k_seg_bytes(KF, D), kVSeg = v_seg_bytes(VF, D);
  static constexpr uint32_t kTile = kKeys * D * 2;              // one operand tile: 16 KB
  static constexpr uint32_t kKBuf = kTile * (kKLo ? 2 : 1), kVBuf = kTile * (kVLo ? 2 : 1);
  static constexpr uint32_t kRawBytes = kPages * (kKSeg + kVSeg);
  // barriers and page ids, then two K^ buffers, two V^T buffers and the raw chunks; the output rows
  // reuse everything behind the page ids
  static constexpr uint32_t kOffBar = 0, kOffPid = 256, kOffK = kOffPid + 4 * kSplitPagesMax;
  static constexpr uint32_t kOffV = kOffK + 2 * kKBuf, kOffRaw = kOffV + 2 * kVBuf;
  static constexpr uint32_t kEnd = kOffRaw + kRaw * kRawBytes;
  static constexpr uint32_t kRowBytes = D * 4 + 16;             // padded output row
  static constexpr uint32_t kEndRows = kOffK + MT * kTileRows * kRowBytes;
  // One CTA per SM, whatever runs beside it: a CTA takes all 512 tensor-memory
  // columns, and one that shares an SM with another holder of them would wait.
  static constexpr uint32_t kNeed = kEnd > kEndRows ? kEnd : kEndRows;
  static constexpr uint32_t kSmem = kNeed < 116 * 1024 ? 116 * 1024 : kNeed;
  static constexpr uint32_t kQCol = 0, kOCol = MT * D / 2, kSCol = kOCol + MT * D;   // tensor-memory columns
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kSCol + MT * kBufs * kKeys <= 512, "tensor memory");
  static_assert(kRawBytes % 16 == 0 && kOffRaw % 16 == 0 && kOffK % 256 == 0, "alignment");
};

// K^ and V^T operand tiles of one chunk, written by the staging warps.
// `valid`: tokens of the chunk that exist; `pmask`: its pages that do.
template <int D, int KF, int KEYS>
__device__ __forceinline__ void stage_k(uint32_t raw, uint32_t buf, uint32_t lo_off, uint32_t pmask, int st) {
  constexpr int KSEG = k_seg_bytes(KF, D), IT = KEYS * (D / 8) / kStageThreads;
  static_assert(IT * kStageThreads == KEYS * (D / 8), "whole items");
  KRaw kr[IT];
#pragma unroll
  for (int it = 0; it < IT; ++it) {      // item i = (token group, 8-dim group, token in group), byte 16 i
    const int i = st + it * kStageThreads, n = ((i >> 3) / (D / 8)) * 8 + (i & 7);
    kr[it] = load_k8<D, KF>(raw + (n / kPage) * KSEG, n % kPage, (i >> 3) % (D / 8));
  }
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int i = st + it * kStageThreads, n = ((i >> 3) / (D / 8)) * 8 + (i & 7);
    uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
    if ((pmask >> (n / kPage)) & 1u) convert_k8<KF>(kr[it], n % kPage, hi, lo);
    sts128(buf + 16 * i, make_uint4(hi[0], hi[1], hi[2], hi[3]));
    if constexpr (KF == MEMRA_KV_Q8_0) sts128(buf + lo_off + 16 * i, make_uint4(lo[0], lo[1], lo[2], lo[3]));
  }
}

// Eight tokens (pairs in words) of which the first n exist; the others become zeros.
__device__ __forceinline__ uint4 keep_tokens(const uint32_t (&x)[4], int n) {
  uint32_t y[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) y[c] = x[c] & (n >= 2 * c + 2 ? 0xFFFFFFFFu : n == 2 * c + 1 ? 0xFFFFu : 0u);
  return make_uint4(y[0], y[1], y[2], y[3]);
}

template <int D, int VF, int KEYS>
__device__ __forceinline__ void stage_v(uint32_t raw, uint32_t buf, uint32_t lo_off, uint32_t pmask, int valid,
                                        int st) {
  constexpr int NB = D / 32, VSEG = v_seg_bytes(VF, D), PAGES = KEYS / kPage;
  constexpr bool kLo = VF == MEMRA_KV_Q5_1 || VF == MEMRA_KV_Q4_0;
  constexpr int TASKS = VF == MEMRA_KV_NVFP4 ? PAGES * 2 * (D / 16) * 8 : PAGES * 2 * NB * 8 * 2;
  constexpr int IT = TASKS / kStageThreads;
  static_assert(IT * kStageThreads == TASKS, "whole tasks");
  // dim dd, token group g (8 tokens): one 16-byte row of a core matrix
  auto store = [&](int dd, int g, uint4 h, uint4 l) {
    const uint32_t off = ((dd >> 3) * (KEYS / 8) + g) * 128 + (dd & 7) * 16;
    sts128(buf + off, h);
    if constexpr (kLo) sts128(buf + lo_off + off, l);
  };
  const uint4 z = make_uint4(0, 0, 0, 0);
  if constexpr (VF == MEMRA_KV_NVFP4) {
    // task (page, half page, 16-dim block b16, rr): dims 16 b16 + rr and + 8
    uint32_t cw[IT][4], sw[IT][4];
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int task = st + it * kStageThreads, rr = task & 7, b16 = (task >> 3) % (D / 16);
      const uint32_t seg = raw + task / (16 * (D / 16)) * VSEG;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        cw[it][c] = lds32(seg + ((b16 >> 2) * 32 + 4 * rr + c) * 16 + (b16 & 3) * 4);
        sw[it][c] = lds32(seg + 8 * D + (c * (D / 16) + b16) * 4);
      }
    }
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int task = st + it * kStageThreads, rr = task & 7, b16 = (task >> 3) % (D / 16),
                ph = (task / (8 * (D / 16))) & 1, ps = task / (16 * (D / 16)), g = 2 * ps + ph;
      uint32_t h0[4], h1[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        __half2 v[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int sh = 8 * (f + 2 * ph);
          v[f] = __hmul2(bits_h2(e2m1x2_to_half2((cw[it][c] >> sh) & 0xFFu)), e4m3_scale_h2(sw[it][c] >> sh));
        }
        h0[c] = h2_bits(__lows2half2(v[0], v[1]));
        h1[c] = h2_bits(__highs2half2(v[0], v[1]));
      }
      const int n = (pmask >> ps) & 1u ? valid - 8 * g : 0;
      store(16 * b16 + rr, g, keep_tokens(h0, n), z);
      store(16 * b16 + rr + 8, g, keep_tokens(h1, n), z);
    }
  } else {
    // task (page, half page, block b, vg, pair h): dims 32 b + 4 vg + 2 h + s, tokens 8 half + 2 c + f
    VRaw vr[IT];
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int task = st + it * kStageThreads;
      vr[it] = load_v_task<D, VF>(raw + task / (32 * NB) * VSEG, (task / (16 * NB)) & 1, (task >> 4) % NB,
                                  (task >> 1) & 7, task & 1);
    }
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int task = st + it * kStageThreads, h = task & 1, vg = (task >> 1) & 7, b = (task >> 4) % NB,
                ph = (task / (16 * NB)) & 1, ps = task / (32 * NB), g = 2 * ps + ph;
      uint32_t hi[2][4], lo[2][4];
      convert_v_task<VF>(vr[it], ph, b, h, hi, lo);
      const int n = (pmask >> ps) & 1u ? valid - 8 * g : 0;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        store(32 * b + 4 * vg + 2 * h + e, g, keep_tokens(hi[e], n), kLo ? keep_tokens(lo[e], n) : z);
    }
  }
}

template <int D, int KF, int VF, int MT>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(const TreeParams p) {
  using C = TreeCfg<D, KF, VF, MT>;
  constexpr int KT = C::kKeys, NP = C::kPages, NBUF = C::kBufs;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bars = sb + C::kOffBar;
  auto raw_full = [&](int s) { return bars + 8 * s; };
  auto raw_empty = [&](int s) { return bars + 8 * (kRaw + s); };
  enum { kKFull = 0, kKEmpty, kVFull, kVEmpty, kSFull, kPFull, kPvDone };
  auto bar = [&](int kind, int b) { return bars + 8 * (2 * kRaw + 2 * kind + b); };
  const uint32_t drained = bars + 8 * (2 * kRaw + 14), q_ready = drained + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffBar + 8 * (2 * kRaw + 16));
  int *pid_s = reinterpret_cast<int *>(smem + C::kOffPid);

  grid_dependency_wait();
  allow_dependent_launch();
  const int kvh = blockIdx.y, b = blockIdx.z / p.row_ctas, rc = blockIdx.z % p.row_ctas;
  const int rows = p.n_nodes * p.group, r0 = rc * MT * kTileRows;
  const int T0 = p.seq_lens[b];
  const int T = max(0, min(min(T0, p.max_seq_len),
                           static_cast<int>(min(static_cast<long long>(p.max_pages) * kPage, 2147483647ll))));
  if (blockIdx.x == 0 && kvh == 0 && rc == 0 && tid == 0 && (T != T0 || T0 < p.n_nodes))
    flag_error(p.status, MEMRA_DEVERR_BAD_SEQ_LEN);
  const int split_len = tree_split_tokens(T, p.target);
  const int ns = tree_ceil(T, split_len);
  // Global row of row r of this KV head: node r / group, head r % group of the group.
  auto row_id = [&](int r) {
    return (static_cast<size_t>(b) * p.n_nodes + r / p.group) * p.n_heads + kvh * p.group + r % p.group;
  };
  if (static_cast<int>(blockIdx.x) >= ns) {
    if (T <= 0 && blockIdx.x == 0)           // no key at all: zeros
      for (int i = tid; i < min(MT * kTileRows, rows - r0) * (D / 8); i += kTreeThreads)
        *reinterpret_cast<uint4 *>(p.out + row_id(r0 + i / (D / 8)) * D + 8 * (i % (D / 8))) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int first = blockIdx.x * split_len, count = min(T - first, split_len);
  const int n_chunks = (count + KT - 1) / KT, n_pages = (count + kPage - 1) / kPage;
  for (int i = tid; i < n_chunks * NP; i += kTreeThreads) {
    int pid = -1;
    if (i < n_pages) {
      pid = p.page_table[static_cast<size_t>(b) * p.max_pages + first / kPage + i];
      if (pid < 0 || pid >= p.num_pages) {
        flag_error(p.status, MEMRA_DEVERR_BAD_PAGE);
        pid = -1;
      }
    }
    pid_s[i] = pid;
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(smem_addr(tmem_slot), 512);
    tc::tmem_relinquish();
  }
  if (tid == 32 * kCopyWarp) {
    for (int s = 0; s < kRaw; ++s) {
      mbar_init(raw_full(s), 1);
      mbar_init(raw_empty(s), kStageWarps);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(bar(kKFull, k), kStageWarps);
      mbar_init(bar(kKEmpty, k), 1);
      mbar_init(bar(kVFull, k), kStageWarps);
      mbar_init(bar(kVEmpty, k), 1);
      mbar_init(bar(kSFull, k), 1);
      mbar_init(bar(kPFull, k), 128);
      mbar_init(bar(kPvDone, k), 1);
    }
    mbar_init(drained, 1);
    mbar_init(q_ready, 128);
    fence_barrier_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  auto chunk_mask = [&](int ci) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) m |= (pid_s[ci * NP + i] >= 0 ? 1u : 0u) << i;
    return m;
  };
  bool ok = true;

  if (warp == kCopyWarp) {
    // ----------------------------------------------------------------- copies --
    if (lane == 0) {
      const size_t kstride = static_cast<size_t>(p.n_kv_heads) * C::kKSeg;
      const size_t vstride = static_cast<size_t>(p.n_kv_heads) * C::kVSeg;
      int issued = 0;
      for (int ci = 0; ci < n_chunks; ++ci) {
        const int s = ci % kRaw;
        if (ci >= kRaw) ok = mbar_wait_bounded(raw_empty(s), (ci / kRaw - 1) & 1, p.status);
        if (!ok) break;
        const uint32_t m = chunk_mask(ci), buf = sb + C::kOffRaw + s * C::kRawBytes;
        if (m) {
          mbar_arrive_expect_tx(raw_full(s), __popc(m) * (C::kKSeg + C::kVSeg));
          for (int i = 0; i < NP; ++i) {
            const int pg = pid_s[ci * NP + i];
            if (pg < 0) continue;
            bulk_copy_g2s_nohint(buf + i * C::kKSeg, p.k_pool + pg * kstride + static_cast<size_t>(kvh) * C::kKSeg,
                                 C::kKSeg, raw_full(s));
            bulk_copy_g2s_nohint(buf + NP * C::kKSeg + i * C::kVSeg,
                                 p.v_pool + pg * vstride + static_cast<size_t>(kvh) * C::kVSeg, C::kVSeg, raw_full(s));
          }
        } else {
          mbar_arrive(raw_full(s));
        }
        issued = ci + 1;
      }
      // every copy has landed before the CTA can leave
      for (int ci = max(0, issued - kRaw); ci < issued; ++ci)
        mbar_wait_bounded(raw_full(ci % kRaw), (ci / kRaw) & 1, p.status);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // -------------------------------------------------------------------- MMA --
    if (lane == 0) {
      constexpr uint32_t idesc_s = tc::idesc_f16_f32(kTileRows, KT);
      constexpr uint32_t idesc_o = tc::idesc_f16_f32(kTileRows, D);
      auto wait = [&](int kind, int k, int phase) {
        ok = ok && mbar_wait_bounded(bar(kind, k), phase & 1, p.status);
      };
      // S_i(ci) = Q_i K^T into score buffer sbuf of tile i
      auto mma_s = [&](int i, int ci) {
        const int kb = ci & 1, sbuf = NBUF > 1 ? ci & 1 : 0;
        wait(kKFull, kb, ci >> 1);
        if (!ok) return;
        tc::fence_after_sync();
        const uint32_t k = sb + C::kOffK + kb * C::kKBuf, d = tmem + C::kSCol + (i * NBUF + sbuf) * KT;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t a = tmem + C::kQCol + i * (D / 2) + 8 * ks;
          tc::mma_f16_ta(d, a, tc::smem_desc(k + 256 * ks, 128, (D / 8) * 128), idesc_s, ks > 0);
          if constexpr (C::kKLo)
            tc::mma_f16_ta(d, a, tc::smem_desc(k + C::kTile + 256 * ks, 128, (D / 8) * 128), idesc_s, 1);
        }
        if (i == MT - 1) tc::commit(bar(kKEmpty, kb));
        tc::commit(bar(kSFull, MT == 1 ? sbuf : i));
      };
      // O_i += P_i(ci) V
      auto mma_o = [&](int i, int ci) {
        const int vb = ci & 1, sbuf = NBUF > 1 ? ci & 1 : 0;
        wait(kPFull, MT == 1 ? sbuf : i, MT == 1 ? ci >> 1 : ci);
        wait(kVFull, vb, ci >> 1);
        if (!ok) return;
        tc::fence_after_sync();
        const uint32_t v = sb + C::kOffV + vb * C::kVBuf, a0 = tmem + C::kSCol + (i * NBUF + sbuf) * KT;
        const uint32_t d = tmem + C::kOCol + i * D;
#pragma unroll
        for (int ks = 0; ks < KT / 16; ++ks) {
          tc::mma_f16_ta(d, a0 + 8 * ks, tc::smem_desc(v + 256 * ks, 128, (KT / 8) * 128), idesc_o,
                         ci > 0 || ks > 0);
          if constexpr (C::kVLo)
            tc::mma_f16_ta(d, a0 + 8 * ks, tc::smem_desc(v + C::kTile + 256 * ks, 128, (KT / 8) * 128), idesc_o, 1);
        }
        if (i == MT - 1) tc::commit(bar(kVEmpty, vb));
        if (NBUF > 1 || ci == n_chunks - 1) tc::commit(bar(kPvDone, i));
      };
      ok = mbar_wait_bounded(q_ready, 0, p.status);
      if constexpr (MT == 1) {
        if (ok) mma_s(0, 0);
        if (ok && n_chunks > 1) mma_s(0, 1);
        for (int ci = 0; ci < n_chunks && ok; ++ci) {
          mma_o(0, ci);
          if (ok && ci + 2 < n_chunks) mma_s(0, ci + 2);   // behind the product that reads its buffer's P
        }
      } else {
        for (int i = 0; i < MT && ok; ++i) mma_s(i, 0);
        for (int ci = 0; ci < n_chunks && ok; ++ci)
          for (int i = 0; i < MT && ok; ++i) {
            mma_o(i, ci);
            if (ok && ci + 1 < n_chunks) mma_s(i, ci + 1);
          }
      }
      tc::commit(drained);                   // what was issued completes before the CTA can leave
      mbar_wait_bounded(drained, 0, p.status);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- staging --
    const int st = tid - 128;
    for (int ci = 0; ci < n_chunks; ++ci) {
      const int s = ci % kRaw, k = ci & 1;
      const uint32_t rawk = sb + C::kOffRaw + s * C::kRawBytes, pmask = chunk_mask(ci);
      ok = mbar_wait_bounded(raw_full(s), (ci / kRaw) & 1, p.status);
      if (ok && ci >= 2) ok = mbar_wait_bounded(bar(kKEmpty, k), ((ci >> 1) - 1) & 1, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      stage_k<D, KF, KT>(rawk, sb + C::kOffK + k * C::kKBuf, C::kTile, pmask, st);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kKFull, k));
      if (ci >= 2) ok = mbar_wait_bounded(bar(kVEmpty, k), ((ci >> 1) - 1) & 1, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      stage_v<D, VF, KT>(rawk + NP * C::kKSeg, sb + C::kOffV + k * C::kVBuf, C::kTile, pmask, count - ci * KT, st);
      fence_proxy_async();                   // V^T for the tensor cores, the raw chunk for the next copies
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kVFull, k));
        mbar_arrive(raw_empty(s));
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax --
    const uint32_t tlane = static_cast<uint32_t>(warp * 32) << 16;
    uint64_t word[MT];
    float m[MT], l[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int r = r0 + i * kTileRows + tid;
      m[i] = -INFINITY;
      l[i] = 0.f;
      word[i] = 0;
      if (r < rows && T - p.n_nodes + r / p.group >= 0) word[i] = p.mask[static_cast<size_t>(b) * p.n_nodes + r / p.group];
      // the row of Q, fp16 pairs as they lie, into tensor memory
      const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (r < rows ? row_id(r) : 0) * D);
#pragma unroll
      for (int c = 0; c < D / 2; c += 32) {
        uint32_t x[32];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint4 y = r < rows ? src[c / 4 + e] : make_uint4(0, 0, 0, 0);
          x[4 * e] = y.x, x[4 * e + 1] = y.y, x[4 * e + 2] = y.z, x[4 * e + 3] = y.w;
        }
        tc::st_32x32b_x32(tmem + tlane + C::kQCol + i * (D / 2) + c, x);
      }
    }
    tc::wait_st();
    tc::fence_before_sync();
    mbar_arrive(q_ready);
    const int base = T - p.n_nodes;          // position of the tree's first row
#pragma unroll 1
    for (int ci = 0; ci < n_chunks && ok; ++ci) {
      const uint32_t pmask = chunk_mask(ci);
      const int tok0 = first + ci * KT, sbuf = NBUF > 1 ? ci & 1 : 0;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int sk = MT == 1 ? sbuf : i;
        const uint32_t s_col = tmem + tlane + C::kSCol + (i * NBUF + sbuf) * KT;
        ok = mbar_wait_bounded(bar(kSFull, sk), (MT == 1 ? ci >> 1 : ci) & 1, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc::fence_after_sync();
        uint32_t s[KT];
#pragma unroll
        for (int c = 0; c < KT; c += 32) tc::ld_32x32b_x32(s_col + c, s + c);
        tc::wait_ld_all();
        tc::hold<KT>(s);
#pragma unroll
        for (int c = 0; c < KT; ++c) s[c] = __float_as_uint(__uint_as_float(s[c]) * p.scale_log2);
        if (pmask != (1u << NP) - 1u || tok0 + KT > base) {
#pragma unroll
          for (int c = 0; c < KT; ++c) {
            const int j = tok0 + c - base;   // the tree's row, if >= 0
            const bool sees = ((pmask >> (c / kPage)) & 1u) && (j < 0 || (j < p.n_nodes && ((word[i] >> j) & 1u)));
            if (!sees) s[c] = 0xff800000u;   // -inf
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < KT; c += 4)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], __uint_as_float(s[c + e]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        float alpha = 1.f;
        if (top > m[i] + kLazy) {            // also the first chunk with a key (m = -inf)
          if (m[i] != -INFINITY) alpha = fast_exp2(m[i] - top);
          m[i] = top;
        }
        if (ci > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // O's rows of this warp times alpha, once the product before has
          // completed (one score buffer: these scores were issued behind it)
          if (NBUF > 1) {
            ok = mbar_wait_bounded(bar(kPvDone, i), (ci - 1) & 1, p.status);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc::fence_after_sync();
          }
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tc::ld_32x32b_x32(tmem + tlane + C::kOCol + i * D + c, o);
            tc::wait_ld_all();
            tc::hold<32>(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc::st_32x32b_x32(tmem + tlane + C::kOCol + i * D + c, o);
          }
          l[i] *= alpha;
        }
        const float mu = m[i] == -INFINITY ? 0.f : m[i];
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int c = 0; c < KT; c += 32) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float p0 = fast_exp2(__uint_as_float(s[c + 2 * e]) - mu);
            const float p1 = fast_exp2(__uint_as_float(s[c + 2 * e + 1]) - mu);
            l0 += p0;
            l1 += p1;
            w[e] = pack_half2(p0, p1);
          }
          tc::st_32x32b_x16(s_col + c / 2, w);
        }
        l[i] += l0 + l1;
        tc::wait_st();
        tc::fence_before_sync();
        mbar_arrive(bar(kPFull, sk));
      }
    }
    // The last product of each tile.  Two score buffers: the product before it may still be
    // running, so its phase comes first (a parity names only the next phase).
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (NBUF > 1 && n_chunks > 1 && ok) ok = mbar_wait_bounded(bar(kPvDone, i), (n_chunks - 2) & 1, p.status);
      if (ok) ok = mbar_wait_bounded(bar(kPvDone, i), NBUF > 1 ? (n_chunks - 1) & 1 : 0, p.status);
    }
    // (every tile's last product is done: the operand tiles and raw pages are free for the output rows)
    ok = __all_sync(0xffffffffu, ok);
    tc::fence_after_sync();
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int r = r0 + i * kTileRows + tid;
      const float inv = l[i] > 0.f ? p.v_post / l[i] : 0.f;
      const uint32_t row = sb + C::kOffK + (i * kTileRows + tid) * C::kRowBytes;
#pragma unroll 1
      for (int c = 0; ok && c < D; c += 32) {
        uint32_t o[32];
        tc::ld_32x32b_x32(tmem + tlane + C::kOCol + i * D + c, o);
        tc::wait_ld_all();
        tc::hold<32>(o);
        float x[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = l[i] > 0.f ? __uint_as_float(o[e]) * inv : 0.f;
        if (ns == 1) {
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            sts128(row + (c + e) * 2, make_uint4(pack_half2(x[e], x[e + 1]), pack_half2(x[e + 2], x[e + 3]),
                                                 pack_half2(x[e + 4], x[e + 5]), pack_half2(x[e + 6], x[e + 7])));
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            sts128(row + (c + e) * 4, make_uint4(__float_as_uint(x[e]), __float_as_uint(x[e + 1]),
                                                 __float_as_uint(x[e + 2]), __float_as_uint(x[e + 3])));
        }
      }
      // the row by one bulk copy; a partial's lse by a plain store (-inf, never weighed, without a
      // visible key or after a wait that gave up)
      if (r < rows) {
        const size_t id = row_id(r), slot = id * p.max_splits + blockIdx.x;
        if (ok) {
          fence_proxy_async();
          if (ns == 1)
            bulk_store_s2g(p.out + id * D, row, D * 2);
          else
            bulk_store_s2g(p.o_part + slot * D, row, D * 4);
        }
        if (ns > 1) p.lse_part[slot] = ok && l[i] > 0.f ? m[i] + __log2f(l[i]) : -INFINITY;
      }
    }
    bulk_store_wait();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// Merge of a row's partials: warp = row, each lane D / 32 consecutive outputs.
constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) tree_merge_kernel(const TreeParams p) {
  constexpr int PER = D / 32, BATCH = 8;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5);
  const int64_t per_seq = static_cast<int64_t>(p.n_nodes) * p.n_heads;
  if (row >= p.batch * per_seq) return;
  const int T0 = p.seq_lens[row / per_seq];
  const int T = max(0, min(min(T0, p.max_seq_len),
                           static_cast<int>(min(static_cast<long long>(p.max_pages) * kPage, 2147483647ll))));
  const int split_len = tree_split_tokens(T, p.target), ns = tree_ceil(T, split_len);
  grid_dependency_wait();                    // the partials are complete
  if (ns <= 1) return;                       // the split pass wrote this row
  const float *lse = p.lse_part + row * p.max_splits;
  const float *src = p.o_part + row * p.max_splits * D + lane * PER;
  float mw = -INFINITY, L = 0.f, acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  for (int k0 = 0; k0 < ns; k0 += BATCH) {   // BATCH partials in flight
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
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      if (ls[u] == -INFINITY) continue;      // its row may hold anything
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
  const float inv = L > 0.f ? 1.f / L : 0.f;
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
    ready[dev] = true;
  }
  const int most = std::max(1, tree_most_splits(p.max_seq_len, p.target));
  const dim3 grid(static_cast<unsigned>(most), static_cast<unsigned>(p.n_kv_heads),
                  static_cast<unsigned>(p.batch * p.row_ctas));
  return launch_pdl(kernel, grid, dim3(kTreeThreads), C::kSmem, st, p);
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
