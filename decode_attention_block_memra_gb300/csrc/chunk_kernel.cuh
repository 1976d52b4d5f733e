// Chunk attention: a chunk of new tokens of every sequence, from one to thousands,
// against the block-quantized paged cache that holds their context and themselves.
// The row of token t (position s = T - n + t) and head h sees keys max(0, s - W + 1) .. s:
//
//   o = sum_u p_u V^_u / sum_u p_u,  p_u = 2^(q . K^_u * scale * log2(e) - m)
//
// The rows of one KV head, tokens x the group's query heads, 128 to a tile, are
// the M side of tcgen05 MMAs, so a page is read and dequantized once for 256 of
// them (128 at head_dim 256).  A CTA walks its share of the call's blocks
// (chunk.cuh) from end to end, its roles each at their own pace:
//   * a copy warp brings raw pages into a ring of chunks (64 keys);
//   * two groups of staging warps dequantize the chunks by turns into fp16 tiles;
//   * one MMA thread: S = Q K^T with Q in tensor memory, O += P V with P in
//     tensor memory over its scores;
//   * groups of four softmax warps, thread = row.
// Head_dim 128 has two softmax groups, each with a score buffer and an O of its own:
// one for each row tile, or, where a block has one tile, taking its chunks by
// turns, their O joined at the end.  Either way the groups take the units (a row
// tile at a chunk) alternately, and one's softmax fills the gaps of the other's MMAs.
// head_dim 256: one group, two score buffers.
//
// Roundings.  K^ and V^ enter exactly, or as fp16 hi + lo pairs (q8_0, q5_1, q4_0: a single fp16
// value of either would cost as much as the output's own rounding, 4.2e-4 instead of 3.0e-4
// with both).  P is fp16, everything else float32.  P is lifted by 2^7: weights below 2^-21 of a row's largest are off by up to
// 2^-32 of it, those below 2^-32 are lost (2^-25 with P at 1: 262,143 keys that weigh 2^-25.1 of one other are 0.7% of the
// row, and all of it was lost).  The tensor cores cut an accumulator's last bits
// at every step, so an O takes kSumUnits chunks at most; then it is added to a
// float32 row in the workspace.
//
// What it measured (q8_0/q5_1, D 128, 32/4 heads).  2,048 tokens behind 30,000: 1.36 ms, with the pairs' products 81% of
// the rate of a large library product, the tensor pipe 69% active; fp8/fp8, which has no pairs and half of the products, 0.95 ms
// with the pipe 47% active.  So the chain bounds it, from a score to its P and to the next score over it, which two groups
// do not quite hide.  512 tokens beside 15 single ones over 60,000 keys: 109 us.  One token over 255
// keys: 11 us, a chain of latencies.  Not faster: an MMA thread for each group (1,818 us), P in columns
// of its own with most of Q in shared memory (1,507 us).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "chunk.cuh"
#include "page_tiles.cuh"
#include "softmax_tile.cuh"
#include "tcgen05.cuh"

namespace memra {
namespace {

// log2 units: a row's maximum passes its reference m by no more between rescales; and P is 2^(s - m + kLift), so
// that it uses fp16's range: 2^15 at most, and 2^7 at least for the row's largest.
constexpr float kLazy = 8.f, kLift = 7.f;
constexpr float kLarge = 1048576.f;        // log2 units: float32 holds smaller scores to 2^-4
constexpr int kSumUnits = 120;             // chunks of one sum of the tensor cores: 7,680 keys

// Where a CTA's share of the line begins, or ends.
struct ChunkPlace {
  int h, b, j, k;
};

// A block, or the part of one, that a CTA takes.  The copy warp finds them one
// after another and leaves them in a ring in shared memory, some ahead of the other warps.
constexpr int kChunkPieces = 4;
struct ChunkPiece {
  int first, tokens;            // row of the block's first token in the call, and its tokens
  int pos0, T;                  // that token's position; keys of the sequence
  int h, b;
  int step0, steps;             // steps over the keys; steps < 0: there is no more piece
  int tiles;
  int whole, head;              // all of the block's steps; its first ones
  int key0;                     // first key that a row of the block sees
};

// Walks a CTA's share.
struct ChunkWalk {
  const ChunkParams &p;
  int h, b, j, k, h1, b1, j1, k1, tpb, seen;
  ChunkSeq s;
  __device__ __forceinline__ ChunkWalk(const ChunkParams &p_, const ChunkPlace &from, const ChunkPlace &to, int tpb_)
      : p(p_), h(from.h), b(from.b), j(from.j), k(from.k), h1(to.h), b1(to.b), j1(to.j), k1(to.k), tpb(tpb_), seen(-1) {}
  __device__ __forceinline__ bool next(ChunkPiece &x) {
    while (true) {
      if (h > h1 || (h == h1 && (b > b1 || (b == b1 && (j > j1 || (j == j1 && k >= k1)))))) return false;
      if (seen != b) {
        s = chunk_seq(p, b);
        seen = b;
      }
      if (j * static_cast<int64_t>(tpb) >= s.n) {
        j = k = 0;
        if (++b == p.batch) b = 0, ++h;
        continue;
      }
      const ChunkBlock block = chunk_block(p, s, j, tpb);
      const int steps = max(0, block.hi - block.lo);
      const bool last = h == h1 && b == b1 && j == j1;
      const int from = k, to = last ? k1 : steps;
      x.first = s.first + block.t0;
      x.tokens = block.t1 - block.t0;
      x.pos0 = s.T - s.n + block.t0;
      x.T = s.T;
      x.h = h, x.b = b;
      x.step0 = block.lo + from;
      x.steps = to - from;
      x.tiles = x.tokens > p.tpt ? 2 : 1;
      x.whole = from == 0 && to == steps;
      x.head = from == 0;
      x.key0 = block.key0;
      if (last) k = k1; else ++j, k = 0;
      if (from < to || steps == 0) return true;
    }
  }
};

template <int D, int KF, int VF>
struct ChunkCfg {
  static constexpr int kTiles = chunk_tiles(D), kGroups = D == 128 ? 2 : 1;
  static constexpr bool kKLo = KF == MEMRA_KV_Q8_0;
  static constexpr bool kVLo = VF == MEMRA_KV_Q5_1 || VF == MEMRA_KV_Q4_0;
  // (pairs of 256 dims leave room for one tile of theirs)
  static constexpr int kStageGroups = D == 256 && (kKLo || kVLo) ? 1 : 2, kStageWarps = 8 / kStageGroups;
  static constexpr int kStageWarp0 = 4 * kGroups, kMmaWarp = kStageWarp0 + 8, kCopyWarp = kMmaWarp + 1;
  static constexpr int kThreads = 32 * (kCopyWarp + 1);
  static constexpr int kPages = kChunkKeys / kPage;
  static constexpr int kKSeg = k_seg_bytes(KF, D), kVSeg = v_seg_bytes(VF, D);
  // q5_1's d q + m as d (q - 16) and, in 16 more columns of V^, the blocks' centres m + 16 d (hi and lo parts),
  // joined to O at the end: three operations a pair instead of ten, and no large sums that nearly cancel.  (The
  // MMA is at most 256 wide, so at head_dim 256 it is the pair of d q + m.)
  static constexpr bool kMCols = VF == MEMRA_KV_Q5_1 && D == 128;
  static constexpr int kOCols = D + (kMCols ? 16 : 0);
  static constexpr bool kVRows = VF != MEMRA_KV_NVFP4;          // V staged as token rows (MN-major)
  static constexpr uint32_t kTile = kChunkKeys * D * 2;
  static constexpr uint32_t kLoOff = kTile + (kMCols ? kChunkKeys * 128 : 0);     // V: hi, centres, lo
  static constexpr uint32_t kKBuf = kTile * (kKLo ? 2 : 1), kVBuf = kVLo ? kLoOff + kTile : kTile;
  static constexpr uint32_t kRawBytes = kPages * (kKSeg + kVSeg);
  // Q in tensor memory; with the centres' columns, two row tiles fill it with 48 columns of Q, 144 of O and 64 of
  // scores each: Q's last 32 dims lie in shared memory.
  static constexpr int kQTmem = kMCols ? 96 : D, kQSmem = D - kQTmem;
  static constexpr int kKBufs = kStageGroups, kVBufs = kStageGroups == 2 || !kVLo ? 2 : 1;
  // barriers, masks of the chunks' pages, the share, the pieces, (m, l) of two groups; then Q's last dims, the tiles
  // and the raw chunks
  static constexpr uint32_t kOffBar = 0, kOffMask = 384, kOffCut = 400, kOffPiece = 448;
  static constexpr uint32_t kOffMl = 1024, kOffQ = 4096;
  static constexpr uint32_t kOffK = kOffQ + kTiles * kChunkRows * kQSmem * 2;
  static constexpr uint32_t kOffV = kOffK + kKBufs * kKBuf, kOffRaw = kOffV + kVBufs * kVBuf;
  static constexpr uint32_t kRoom = 227 * 1024;
  static constexpr int kRaw = (kRoom - kOffRaw) / kRawBytes < 6 ? (kRoom - kOffRaw) / kRawBytes : 6;
  // Tensor memory: a CTA that found its columns taken would wait in its allocation, so
  // no more CTAs of the library's tensor-memory kernels may fit an SM than its 512 columns hold.
  static constexpr uint32_t kTCols = 512, kNeed = kOffRaw + kRaw * kRawBytes, kFloor = 150 * 1024;
  static constexpr uint32_t kSmem = kNeed < kFloor ? kFloor : kNeed;
  // tensor-memory columns: Q of each row tile, O of each group, two score buffers
  static constexpr uint32_t kQCol = 0, kOCol = kTiles * kQTmem / 2, kSCol = kOCol + kGroups * kOCols;
  // barriers: the raw chunks', six pairs for the tiles, scores and weights, then
  enum Bar { kPvDone = 2 * kRaw + 12, kQReady = kPvDone + 2, kDrained = kQReady + 2, kPieceFull, kPieceFree = kPieceFull + kChunkPieces,
             kBars = kPieceFree + kChunkPieces };
  static_assert(kRaw >= 2 && kRaw <= 8, "a chunk ahead; the masks' ring");
  static_assert(kOffBar + 8 * kBars + 4 <= kOffMask, "barriers and the tensor-memory address");
  static_assert(kOffPiece + kChunkPieces * sizeof(ChunkPiece) <= kOffMl, "pieces");
  static_assert(kOffMl + 2 * kChunkRows * 8 <= kOffQ, "maxima and sums");
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kSCol + 2 * kChunkKeys <= kTCols, "tensor memory");
  static_assert(kRawBytes % 16 == 0 && kOffRaw % 16 == 0 && kOffK % 1024 == 0 && kTile % 1024 == 0, "alignment");
};

// The keys of the chunk's pages whose bit is set.
__device__ __forceinline__ uint64_t chunk_page_keys(uint32_t pmask) {
  uint64_t keys = 0;
#pragma unroll
  for (int i = 0; i < kChunkKeys / kPage; ++i) keys |= (pmask >> i) & 1u ? 0xFFFFull << (kPage * i) : 0ull;
  return keys;
}

// Bit c: a row `last` keys past the chunk's first sees key c of the chunk (the last `window` up to its own; 0: all).
__device__ __forceinline__ uint64_t chunk_seen(int last, int window) {
  uint64_t keys = last >= 63 ? ~0ull : last < 0 ? 0ull : (2ull << last) - 1ull;
  if (window > 0) {
    const int low = last - window + 1;
    keys &= low >= 64 ? 0ull : low > 0 ? ~0ull << low : ~0ull;
  }
  return keys;
}

template <int D, int KF, int VF>
__global__ void __launch_bounds__(ChunkCfg<D, KF, VF>::kThreads, 1) chunk_kernel(const ChunkParams p) {
  using C = ChunkCfg<D, KF, VF>;
  constexpr int KT = kChunkKeys, NP = C::kPages, RAW = C::kRaw, SW = C::kStageWarps, G = C::kGroups;
  constexpr uint32_t kAllPages = (1u << NP) - 1u;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bars = sb + C::kOffBar;
  auto raw_full = [&](int s) { return bars + 8 * s; };
  auto raw_empty = [&](int s) { return bars + 8 * (RAW + s); };
  enum { kKFull = 0, kKEmpty, kVFull, kVEmpty, kSFull, kPFull };
  auto bar = [&](int kind, int b) { return bars + 8 * (2 * RAW + 2 * kind + b); };
  auto pv_done = [&](int i) { return bars + 8 * (C::kPvDone + i); };
  auto q_ready = [&](int i) { return bars + 8 * (C::kQReady + i); };
  auto piece_full = [&](int i) { return bars + 8 * (C::kPieceFull + i); };
  auto piece_free = [&](int i) { return bars + 8 * (C::kPieceFree + i); };
  const uint32_t drained = bars + 8 * C::kDrained;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffBar + 8 * C::kBars);
  ChunkPiece *pieces = reinterpret_cast<ChunkPiece *>(smem + C::kOffPiece);
  // a byte for each chunk in flight: the pages that exist
  volatile uint8_t *page_mask = smem + C::kOffMask;
  ChunkPlace *share = reinterpret_cast<ChunkPlace *>(smem + C::kOffCut);
  const int tpb = C::kTiles * p.tpt;

  if (warp == C::kCopyWarp) {
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
        mbar_init(pv_done(k), 1);
        mbar_init(q_ready(k), 4);
      }
      mbar_init(drained, 1);
      for (int k = 0; k < kChunkPieces; ++k) {
        mbar_init(piece_full(k), 1);
        mbar_init(piece_free(k), C::kCopyWarp);        // every other warp
      }
      fence_barrier_init();
    }
  } else if (warp == C::kMmaWarp) {
    tc::tmem_alloc(smem_addr(tmem_slot), C::kTCols);
    tc::tmem_relinquish();
  }
  grid_dependency_wait();
  allow_dependent_launch();
  if (warp < 2) {                                      // the share's two ends, by a warp each
    const int64_t head = chunk_head_cost<C::kTiles>(p, tpb, lane);
    const int n = chunk_shares<C::kTiles>(p, head), c = blockIdx.x + warp;
    const bool some = head > 0 && static_cast<int>(blockIdx.x) < n;
    ChunkPlace at{warp == 0 ? 0 : some ? p.n_kv_heads : -1, 0, 0, 0};
    if (some && c > 0 && c < n) {
      const ChunkCut x = chunk_cut<C::kTiles>(p, head, head * p.n_kv_heads * c / n, tpb, lane);
      at = ChunkPlace{x.h, x.b, x.j, x.k};
    }
    if (lane == 0) share[warp] = at;
  } else if (warp == 2 && blockIdx.x == 0) {           // one CTA checks every length
    for (int b = lane; b < p.batch; b += 32)
      if (chunk_seq(p, b).bad) flag_error(p.status, MEMRA_DEVERR_BAD_SEQ_LEN);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;
  int cc = 0, piece = 0;                     // chunks and pieces before the present one, in this CTA
  // The next piece, for the warps that are told of it (one thread of the MMA warp); and that this warp is done with one.
  auto next_piece = [&]() -> const volatile ChunkPiece * {
    const int i = piece % kChunkPieces;
    ok = ok && mbar_wait_suspended(piece_full(i), (piece / kChunkPieces) & 1, p.status);
    return pieces + i;
  };
  auto free_piece = [&] {
    mbar_arrive(piece_free(piece % kChunkPieces));
    ++piece;
  };

  if (warp == C::kCopyWarp) {
    // ----------------------------------------------------------------- copies --
    // Lane = (page of a chunk, K or V): one copy each, issued together.  Page ids are
    // read for eight chunks at a time, a lane each, eight chunks ahead.
    const int cp_page = lane >> 1;
    const bool cp_v = lane & 1;
    const uint32_t cp_bytes = cp_v ? C::kVSeg : C::kKSeg;
    ChunkWalk walk(p, share[0], share[1], tpb);
    ChunkPiece x;
    while (ok) {
      const bool more = walk.next(x);
      if (!more) x.steps = -1;
      const int at = piece % kChunkPieces;
      if (piece >= kChunkPieces) ok = mbar_wait_suspended(piece_free(at), (piece / kChunkPieces - 1) & 1, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) {
        pieces[at] = x;
        mbar_arrive(piece_full(at));
      }
      __syncwarp();
      ++piece;
      if (!more) break;
      const int32_t *table = p.page_table + static_cast<size_t>(x.b) * p.max_pages;
      // Page id of a logical page, -1: none (past the keys, before the first one seen, or outside the pool).
      auto page_id = [&](int step) {
        const int i = (x.step0 + step) * NP + (lane & (NP - 1));
        if (step >= x.steps || i > (x.T - 1) / kPage || i < x.key0 / kPage) return -1;
        const int pid = table[p.window > 0 ? i % p.max_pages : i];
        if (pid >= 0 && pid < p.num_pages) return pid;
        flag_error(p.status, MEMRA_DEVERR_BAD_PAGE);
        return -1;
      };
      int ids = page_id(lane / NP), ahead = page_id(8 + lane / NP);
      for (int i = 0; i < x.steps; ++i, ++cc) {
        if (i > 0 && i % 8 == 0) {
          ids = ahead;
          ahead = page_id(i + 8 + lane / NP);
        }
        int pid = __shfl_sync(0xffffffffu, ids, (i % 8) * NP + (cp_page & (NP - 1)));
        if (cp_page >= NP) pid = -1;
        const int s = cc % RAW;
        if (cc >= RAW) ok = mbar_wait_suspended(raw_empty(s), (cc / RAW - 1) & 1, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t there = __ballot_sync(0xffffffffu, pid >= 0);
        if (lane == 0) {
          uint32_t m = 0;
#pragma unroll
          for (int e = 0; e < NP; ++e) m |= (there >> (2 * e) & 1u) << e;
          page_mask[cc & 15] = static_cast<uint8_t>(m);
          const int n = __popc(there) / 2;
          if (n)
            mbar_arrive_expect_tx(raw_full(s),
                                  n * (C::kKSeg + C::kVSeg) + (cc == 0 && blockIdx.x == 0 ? p.test_extra_tx : 0));
          else
            mbar_arrive(raw_full(s));
        }
        __syncwarp();
        if (pid >= 0)
          bulk_copy_g2s_nohint(sb + C::kOffRaw + s * C::kRawBytes + (cp_v ? NP * C::kKSeg : 0) + cp_page * cp_bytes,
                               (cp_v ? p.v_pool : p.k_pool) + (static_cast<size_t>(pid) * p.n_kv_heads + x.h) * cp_bytes,
                               cp_bytes, raw_full(s));
      }
    }
    // every copy has landed before the CTA can leave
    for (int c = max(0, cc - RAW); c < cc; ++c) mbar_wait_suspended(raw_full(c % RAW), (c / RAW) & 1, p.status);
    __syncwarp();
  } else if (warp == C::kMmaWarp) {
    // -------------------------------------------------------------------- MMA --
    if (tc::elect_one()) {
      constexpr uint32_t idesc_s = tc::idesc_f16_f32(kChunkRows, KT);
      constexpr uint32_t idesc_o = C::kVRows ? tc::idesc_f16_f32_bmn(kChunkRows, D) : tc::idesc_f16_f32(kChunkRows, D);
      constexpr uint32_t idesc_oc = C::kMCols ? tc::idesc_f16_f32_bmn(kChunkRows, C::kOCols) : idesc_o;
      int used[2] = {0, 0};                  // uses of the score buffers
      while (true) {
        const volatile ChunkPiece *x = next_piece();
        const int steps = ok ? x->steps : -1, shift = ok ? x->tiles - 1 : 0, units = steps << shift;
        if (steps < 0) break;
        auto wait = [&](int kind, int k, int phase) {
          ok = ok && mbar_wait_suspended(bar(kind, k), phase & 1, p.status);
        };
        // Unit u: row tile (two of them: u's last bit) at chunk u >> shift; score buffer u & 1, and O of the same
        // group where there are two.
        // S(u) = Q K^T
        auto mma_s = [&](int u) {
          if (!ok || u >= units) return;
          const int c = cc + (u >> shift), kb = c % C::kKBufs, sk = u & 1;
          wait(kKFull, kb, c / C::kKBufs);
          if (!ok) return;
          tc::fence_after_sync();
          const uint32_t d = tmem + C::kSCol + sk * KT;
          const int tile = shift ? sk : 0;
          const uint64_t kd = tc::smem_desc_sw128(sb + C::kOffK + kb * C::kKBuf, 16, 1024);
          const uint64_t qd = tc::smem_desc(sb + C::kOffQ + tile * kChunkRows * C::kQSmem * 2, 128, C::kQSmem / 8 * 128);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
            for (int lo = 0; lo < (C::kKLo ? 2 : 1); ++lo) {
              const uint64_t bd = tc::desc_at(kd, (ks / 4) * KT * 128 + (ks % 4) * 32 + lo * C::kTile);
              if (16 * ks < C::kQTmem)
                tc::mma_f16_ta(d, tmem + C::kQCol + tile * (C::kQTmem / 2) + 8 * ks, bd, idesc_s, ks + lo > 0);
              else
                tc::mma_f16(d, tc::desc_at(qd, 256 * (ks - C::kQTmem / 16)), bd, idesc_s, 1);
            }
          }
          if (!shift || sk) tc::commit(bar(kKEmpty, kb));
          tc::commit(bar(kSFull, sk));
        };
        // O += P(u) V, P in the columns of its scores
        auto mma_o = [&](int u) {
          if (!ok) return;
          const int c = cc + (u >> shift), vb = c % C::kVBufs, sk = u & 1;
          wait(kPFull, sk, used[sk]);
          wait(kVFull, vb, c / C::kVBufs);
          if (!ok) return;
          ++used[sk];
          tc::fence_after_sync();
          const uint32_t v = sb + C::kOffV + vb * C::kVBuf, a = tmem + C::kSCol + sk * KT;
          const uint32_t d = tmem + C::kOCol + (G == 2 ? sk * C::kOCols : 0);
          const uint64_t vd = C::kVRows ? tc::smem_desc_sw128(v, KT * 128, 1024) : tc::smem_desc(v, 128, (KT / 8) * 128);
          constexpr uint32_t kStep = C::kVRows ? 2048 : 256;       // a K = 16 step further on
          const bool anew = (G == 2 ? u >> 1 : u) % kSumUnits == 0;
#pragma unroll
          for (int ks = 0; ks < KT / 16; ++ks) {
            tc::mma_f16_ta(d, a + 8 * ks, tc::desc_at(vd, kStep * ks), idesc_oc, !anew || ks > 0);
            if constexpr (C::kVLo) tc::mma_f16_ta(d, a + 8 * ks, tc::desc_at(vd, kStep * ks + C::kLoOff), idesc_o, 1);
          }
          if (!shift || sk) tc::commit(bar(kVEmpty, vb));
          if (G == 1 || u + 2 >= units) tc::commit(pv_done(G == 2 ? sk : 0));
        };
#pragma unroll
        for (int i = 0; i < G; ++i) ok = ok && mbar_wait_suspended(q_ready(i), piece & 1, p.status);
        mma_s(0);
        mma_s(1);
        for (int u = 0; u < units && ok; ++u) {
          mma_o(u);
          mma_s(u + 2);                      // behind the product that reads its buffer's P
        }
        cc += steps;
        free_piece();
      }
      tc::commit(drained);                   // what was issued completes before the CTA can leave
      mbar_wait_suspended(drained, 0, p.status);
    }
    __syncwarp();
  } else if (warp >= C::kStageWarp0) {
    // ---------------------------------------------------------------- staging --
    if constexpr (D == 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int sg = (warp - C::kStageWarp0) / SW, sw = (warp - C::kStageWarp0) % SW, st = 32 * sw + lane;
    if constexpr (C::kMCols) {               // the unused columns of the centres' block, once
      for (int vb = sg; vb < C::kVBufs; vb += C::kStageGroups)
        for (uint32_t i = st; i < KT * 8u; i += 32 * SW)
          sts128(sb + C::kOffV + vb * C::kVBuf + C::kTile + 16 * i, make_uint4(0, 0, 0, 0));
      named_barrier_sync(1 + sg, 32 * SW);
    }
    while (true) {
      const volatile ChunkPiece *x = next_piece();
      ok = __all_sync(0xffffffffu, ok);
      const int steps = ok ? x->steps : -1;
      if (steps < 0) break;
      const int keys = x->T - x->step0 * KT; // from the first step on
      __syncwarp();
      if (lane == 0) free_piece(); else ++piece;
      for (int i = 0; i < steps; ++i) {
        const int c = cc + i;
        if (C::kStageGroups == 2 && (c & 1) != sg) continue;
        const int s = c % RAW, kb = c % C::kKBufs, vb = c % C::kVBufs, valid = keys - i * KT;
        const uint32_t rawk = sb + C::kOffRaw + s * C::kRawBytes, rawv = rawk + NP * C::kKSeg;
        // (K^'s tile first: that its last scores are done says that the chunk RAW before this one has landed,
        // so that the raw chunk's parity names this use of its place and not the one two before)
        if (c >= C::kKBufs) ok = mbar_wait_suspended(bar(kKEmpty, kb), (c / C::kKBufs - 1) & 1, p.status);
        if (ok) ok = mbar_wait_suspended(raw_full(s), (c / RAW) & 1, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        stage_k<D, KF, KT, SW>(rawk, sb + C::kOffK + kb * C::kKBuf, sw, lane);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kKFull, kb));
        if (c >= C::kVBufs) ok = mbar_wait_suspended(bar(kVEmpty, vb), (c / C::kVBufs - 1) & 1, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // Tokens that exist; the others need not have been written, and 0 * (what their bytes stand for) may be NaN.
        uint64_t keep = valid < KT ? (1ull << valid) - 1ull : ~0ull;
        const uint32_t pages = page_mask[c & 15];
        if (pages != kAllPages) keep &= chunk_page_keys(pages);
        const uint32_t vbuf = sb + C::kOffV + vb * C::kVBuf;
        if constexpr (C::kVRows)
          stage_v<D, VF, KT, SW, C::kMCols, C::kLoOff>(rawv, vbuf, keep, sw, lane);
        else
          stage_v_nvfp4<D, KT, SW>(rawv, vbuf, keep, st);
        if constexpr (C::kMCols) {           // 32 tokens by each of two warps, other ones each time
          const int part = (sw - 2 * c) & (SW - 1);
          if (part < KT / 32) stage_m<D, KT>(rawv, vbuf + C::kTile, keep, 32 * part + lane);
        }
        fence_proxy_async();                 // V^ for the tensor cores, the raw chunk for the next copies
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kVFull, vb));
          mbar_arrive(raw_empty(s));
        }
      }
      cc += steps;
    }
  } else {
    // ---------------------------------------------------------------- softmax --
    if constexpr (D == 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
    const int g = warp >> 2, rl = tid & 127;           // group, row of its tile
    const uint32_t tlane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t o_col = tmem + tlane + C::kOCol + g * C::kOCols;
    const int tl = rl / p.group, head = rl % p.group;
    float4 *const far = reinterpret_cast<float4 *>(p.far) +
                        (static_cast<size_t>(blockIdx.x) * G + g) * (kChunkFarCols(D) / 4) * kChunkRows + rl;
    int used[2] = {0, 0}, done = 0;                    // uses of the score buffers; phases of pv_done
    while (true) {
      const volatile ChunkPiece *x = next_piece();
      // All softmax warps go on together, or none; and both groups' rows are out: Q and the maxima may be this piece's.
      tc::fence_before_sync();
      ok = named_barrier_and(3, 32 * 4 * G, ok);
      tc::fence_after_sync();
      if (!ok || x->steps < 0) break;
      const int shift = x->tiles - 1, units = x->steps << shift;
      const bool turns = G == 2 && shift == 0;
      const int tile = turns ? 0 : g, t = tile * p.tpt + tl;       // the row's token in the block
      const bool live = tl < p.tpt && t < x->tokens;
      // from the first step's first key: the row's own position (rows that do not exist see nothing), the tile's first
      // and last
      const int origin = x->step0 * KT;
      const int pos = live ? x->pos0 + t - origin : -1;
      const int pos_first = x->pos0 + tile * p.tpt - origin;
      const int pos_last = x->pos0 + min(x->tokens, (tile + 1) * p.tpt) - 1 - origin;
      {
        // the row of Q: fp16 pairs into tensor memory, the last dims into core matrices
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q + (live ? (x->first + t) * p.q_stride + static_cast<int64_t>(x->h * p.group + head) * D : 0));
        auto load = [&](int u) {
          const uint4 v = live ? src[u] : make_uint4(0, 0, 0, 0);
          return make_uint4(nan_for_inf(v.x), nan_for_inf(v.y), nan_for_inf(v.z), nan_for_inf(v.w));
        };
#pragma unroll
        for (int c = 0; c < C::kQTmem / 2; c += 16) {
          if (turns && g != (c >= 32)) continue;       // a part of the row by each group
          uint32_t y[16];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4 v = load(c / 4 + e);
            y[4 * e] = v.x, y[4 * e + 1] = v.y, y[4 * e + 2] = v.z, y[4 * e + 3] = v.w;
          }
          tc::st_32x32b_x16(tmem + tlane + C::kQCol + tile * (C::kQTmem / 2) + c, y);
        }
#pragma unroll
        for (int u = 0; u < C::kQSmem / 8; ++u) {
          if (turns && g == 0) continue;
          sts128(sb + C::kOffQ + tile * kChunkRows * C::kQSmem * 2 + ((rl >> 3) * (C::kQSmem / 8) + u) * 128 + (rl & 7) * 16,
                 load(C::kQTmem / 8 + u));
        }
      }
      if constexpr (C::kQSmem > 0) fence_proxy_async();
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready(g));
      float m = -INFINITY, l = 0.f, m_far = -INFINITY;
      bool large = false;                    // of the warp: some row's reference is
      // O plus what lies in `far`, to `far` (or back to O, at the end)
      auto join = [&](bool back) {
        const bool held = m_far != -INFINITY;
        const float scale = held ? fast_exp2(m_far - m) : 0.f;
#pragma unroll 1
        for (int c = 0; c < C::kOCols; c += 16) {
          uint32_t o[16];
          tc::ld_32x32b_x16(o_col + c, o);
          float4 f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = held ? far[(c / 4 + e) * kChunkRows] : make_float4(0.f, 0.f, 0.f, 0.f);
          tc::wait_ld(o);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[e].x = fmaf(f[e].x, scale, __uint_as_float(o[4 * e]));
            f[e].y = fmaf(f[e].y, scale, __uint_as_float(o[4 * e + 1]));
            f[e].z = fmaf(f[e].z, scale, __uint_as_float(o[4 * e + 2]));
            f[e].w = fmaf(f[e].w, scale, __uint_as_float(o[4 * e + 3]));
          }
          if (back) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[4 * e] = __float_as_uint(f[e].x), o[4 * e + 1] = __float_as_uint(f[e].y);
              o[4 * e + 2] = __float_as_uint(f[e].z), o[4 * e + 3] = __float_as_uint(f[e].w);
            }
            tc::st_32x32b_x16(o_col + c, o);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) far[(c / 4 + e) * kChunkRows] = f[e];
          }
        }
        if (back) tc::wait_st();
      };
#pragma unroll 1
      for (int u = g; u < units && ok; u += G) {
        const int i = u >> shift, nth = G == 2 ? u >> 1 : u, sk = u & 1;
        const int tok0 = i * KT;
        const uint32_t s_col = tmem + tlane + C::kSCol + sk * KT;
        ok = mbar_wait_suspended(bar(kSFull, sk), used[sk] & 1, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++used[sk];
        tc::fence_after_sync();
        uint32_t s[KT];
#pragma unroll
        for (int c = 0; c < KT; c += 32) tc::ld_32x32b_x32(s_col + c, s + c);
        const uint32_t pages = page_mask[(cc + i) & 15];
        tc::wait_ld_all();
        tc::hold<KT>(s);
        if (pages != kAllPages || tok0 + KT - 1 > pos_first || (p.window > 0 && tok0 < pos_last - p.window + 1)) {
          const uint64_t sees = chunk_seen(pos - tok0, p.window) & chunk_page_keys(pages);
          const uint32_t half[2] = {static_cast<uint32_t>(sees), static_cast<uint32_t>(sees >> 32)};
#pragma unroll
          for (int c = 0; c < KT; ++c)
            if (!(half[c / 32] & (1u << (c % 32)))) s[c] = 0xff800000u;      // -inf
        }
        const float most = row_max(s), top = __fmul_rn(most, p.scale_log2);      // (rounded: not a part of a fused sum below)
        if (G == 1 && nth > 0 && nth % kSumUnits == 0) {
          ok = mbar_wait_suspended(pv_done(0), (done + nth - 1) & 1, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc::fence_after_sync();
        }
        if (nth > 0 && nth % kSumUnits == 0) {         // (a group of two: these scores were issued behind its product)
          join(false);
          m_far = m;
        }
        float alpha = 1.f;
        const bool passed = __any_sync(0xffffffffu, top - m > kLazy), moved = nth > 0 && passed;
        if (passed) {
          if (top - m > kLazy) {             // also the first chunk with a key (m = -inf)
            if (m != -INFINITY) alpha = fast_exp2(m - top);
            m = top;
          }
          large = __any_sync(0xffffffffu, fabsf(m) > kLarge && m != -INFINITY);
        }
        if (G == 1 && nth > 0 && (moved || nth == units - 1)) {
          // The product before has completed, O is still (a group of two: these scores were issued behind it).
          // At the last chunk in any case: the wait behind the loop names the last product by its
          // parity, which the product two before has too.
          ok = mbar_wait_suspended(pv_done(0), (done + nth - 1) & 1, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc::fence_after_sync();
        }
        if (moved) {                         // O's rows of this warp times alpha
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
        float mu = m == -INFINITY ? 0.f : m - kLift;
        if (large) {
          // s * scale - m may be off by more than P has room for: the difference from the chunk's largest first, which is exact
          // for what lies near it
          const float from = most == -INFINITY ? 0.f : most;
#pragma unroll
          for (int c = 0; c < KT; ++c) s[c] = __float_as_uint(__uint_as_float(s[c]) - from);
          if (most != -INFINITY) mu = (m - top) - kLift;
        }
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
      if (G == 1) {
        if (ok && units > 0) ok = mbar_wait_suspended(pv_done(0), (done + units - 1) & 1, p.status);
        done += units;
      } else {
        // the other group's last product too, where O of both make one row
        for (int e = 0; e < 2; ++e) {
          const bool any = e < units;
          if (ok && any && (turns || e == g)) ok = mbar_wait_suspended(pv_done(e), (e ? done >> 1 : done) & 1, p.status);
        }
        // (low bit: phases of the first group's barrier; next: the second's)
        done ^= (units > 0 ? 1 : 0) | (units > 1 ? 2 : 0);
      }
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
      if (ok && __any_sync(0xffffffffu, m_far != -INFINITY)) join(true);
      // O = sum of w[e] O_e over the row's groups
      float w[2] = {0.f, 0.f};
      if (turns) {
        const uint32_t ml = sb + C::kOffMl + rl * 8;
        sts64(ml + g * kChunkRows * 8, __float_as_uint(m), __float_as_uint(l));
        tc::fence_before_sync();
        ok = named_barrier_and(3, 32 * 4 * G, ok);
        tc::fence_after_sync();
        const float m1 = __uint_as_float(lds32(ml + (g ^ 1) * kChunkRows * 8));
        const float l1 = __uint_as_float(lds32(ml + (g ^ 1) * kChunkRows * 8 + 4));
        // (a sum of NaN, from a query or a key that is not finite, is no empty one: the row becomes NaN)
        const float top = fmaxf(m, m1);
        const float mine = l != 0.f ? fast_exp2(m - top) : 0.f, other = l1 != 0.f ? fast_exp2(m1 - top) : 0.f;
        w[0] = g ? other : mine, w[1] = g ? mine : other;
        l = l * mine + l1 * other;
        m = top;
      } else {
        w[0] = l != 0.f ? 1.f : 0.f;
      }
      const float inv = l != 0.f ? p.v_post / l : 0.f;
      w[0] *= inv, w[1] *= inv;
      const uint32_t o_first = turns ? tmem + tlane + C::kOCol : o_col;      // of the row's first group
      const int parts = turns ? 2 : 1;
      const bool whole = x->whole;
      const int slot = 2 * blockIdx.x + (x->head ? 1 : 0), part_row = tile * kChunkRows + rl;
      const int64_t row = static_cast<int64_t>(x->first + t) * p.n_heads + x->h * p.group + head;
      float4 *const part = reinterpret_cast<float4 *>(p.o_part) +
                           static_cast<size_t>(slot) * (D / 4) * (C::kTiles * kChunkRows) + part_row;
      uint4 *const to = reinterpret_cast<uint4 *>(p.out + row * D);
      // the centres' sums (hi and lo parts together) of this group's 32-dim blocks
      float centre[D / 32];
      if constexpr (C::kMCols) {
#pragma unroll
        for (int e = 0; e < D / 32; ++e) centre[e] = 0.f;
        for (int k = 0; k < parts; ++k) {
          uint32_t o[16];
          tc::ld_32x32b_x16(o_first + k * C::kOCols + D, o);
          tc::wait_ld(o);
#pragma unroll
          for (int e = 0; e < D / 32; ++e)
            centre[e] = w[k] != 0.f ? fmaf(__uint_as_float(o[e]) + __uint_as_float(o[D / 32 + e]), w[k], centre[e]) : centre[e];
        }
      }
#pragma unroll
      for (int c = 0; c < D; c += 16) {
        if (!ok || (turns && g != (c >= D / 2))) continue;                   // (by turns: half of the columns each)
        float y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = C::kMCols ? centre[c / 32] : 0.f;
        for (int k = 0; k < parts; ++k) {
          uint32_t o[16];
          tc::ld_32x32b_x16(o_first + k * C::kOCols + c, o);
          tc::wait_ld(o);
#pragma unroll
          for (int e = 0; e < 16; ++e)       // (a group without a visible key: its O may hold anything)
            y[e] = w[k] != 0.f ? fmaf(__uint_as_float(o[e]), w[k], y[e]) : y[e];
        }
        if (!live) continue;
        if (whole) {
#pragma unroll
          for (int e = 0; e < 16; e += 8)
            to[(c + e) / 8] = make_uint4(pack_half2(y[e], y[e + 1]), pack_half2(y[e + 2], y[e + 3]),
                                         pack_half2(y[e + 4], y[e + 5]), pack_half2(y[e + 6], y[e + 7]));
        } else {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            part[static_cast<size_t>((c + e) / 4) * (C::kTiles * kChunkRows)] = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
        }
      }
      if (ok && live && (!turns || g == 0)) {
        // base 2; -inf, never weighed, without a visible key
        const float lse = l != 0.f ? m - kLift + log2f(l) : -INFINITY;
        if (!whole)
          p.lse_part[static_cast<size_t>(slot) * (C::kTiles * kChunkRows) + part_row] = lse;
        else if (p.lse)
          p.lse[row] = lse * 0.69314718055994531f;
      }
      cc += x->steps;
      __syncwarp();
      if (lane == 0) free_piece(); else ++piece;
    }
    if (!ok) {
      // A wait gave up: every row of the CTA's share becomes NaN.
      ChunkWalk walk(p, share[0], share[1], tpb);
      ChunkPiece x;
      while (walk.next(x)) {
        const int tile = x.tiles == 2 ? g : 0, t = tile * p.tpt + tl;
        if (tl >= p.tpt || t >= x.tokens || (G == 2 && x.tiles == 1 && g == 1)) continue;
        const int64_t row = static_cast<int64_t>(x.first + t) * p.n_heads + x.h * p.group + head;
        const float nan = __uint_as_float(kNanPair);
        if (!x.whole) {
          p.lse_part[static_cast<size_t>(2 * blockIdx.x + (x.head ? 1 : 0)) * (C::kTiles * kChunkRows) + tile * kChunkRows + rl] = nan;
          continue;
        }
        if (p.lse) p.lse[row] = nan;
        for (int u = 0; u < D / 8; ++u)
          reinterpret_cast<uint4 *>(p.out + row * D)[u] = make_uint4(kNanPair, kNanPair, kNanPair, kNanPair);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == C::kMmaWarp) tc::tmem_dealloc(tmem, C::kTCols);
}

template <int D, int KF, int VF>
cudaError_t launch_chunk_one(const ChunkParams &p, cudaStream_t st) {
  using C = ChunkCfg<D, KF, VF>;
  auto kernel = chunk_kernel<D, KF, VF>;
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
  return launch_pdl(kernel, dim3(p.ctas), dim3(C::kThreads), C::kSmem, st, p);
}

template <int KF>
cudaError_t launch_chunk_formats(int D, int vf, const ChunkParams &p, cudaStream_t st) {
  auto by_dim = [&](auto v) -> cudaError_t {
    constexpr int V = decltype(v)::value;
    return D == 128 ? launch_chunk_one<128, KF, V>(p, st) : launch_chunk_one<256, KF, V>(p, st);
  };
  switch (vf) {
    case MEMRA_KV_Q5_1: return by_dim(std::integral_constant<int, MEMRA_KV_Q5_1>{});
    case MEMRA_KV_Q4_0: return by_dim(std::integral_constant<int, MEMRA_KV_Q4_0>{});
    case MEMRA_KV_FP8_E4M3: return by_dim(std::integral_constant<int, MEMRA_KV_FP8_E4M3>{});
    case MEMRA_KV_NVFP4: return by_dim(std::integral_constant<int, MEMRA_KV_NVFP4>{});
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
}  // namespace memra
