// Key weights: how much attention each cached key collects from a chunk of query
// rows whose log-sum-exp is known, summed over the rows and the heads of a group.
//
//   w_u <- keep * w_u + sum over rows t, heads h that see key u of 2^(q_th . K^_u * scale * log2(e) - lse_th * log2(e))
//
// One pass over K, no V and no softmax state: the log-sum-exp makes every weight
// final as its score is.  The keys are the M side of the tcgen05 MMAs, the query
// rows the N side, so that a thread of the epilogue holds one key and adds up its
// weights over all rows in a register: no sum crosses threads, and none is
// atomic.  K^ is dequantized once (q8_0 as exact fp16 pairs: the weights are float32) and meets
// every row tile while it lies in shared memory.
//   * a copy warp brings raw pages into a ring;
//   * eight staging warps dequantize them into tiles of 128 keys, one tile after the
//     other: while one is made, the tensor cores are at the other;
//   * a load warp brings row tiles of Q by TMA; where all rows of the chunk
//     fit their ring, once for all keys of a CTA's run;
//   * an MMA thread for each key tile: S^T = K^ Q^T, two key tiles beside one another for
//     each row tile (one thread for both took longer to issue than the MMAs run: 205 us);
//   * four groups of four warps, two for each key tile, which take its row tiles by
//     turns: thread = key (at head_dim 256 with q8_0 there is room for one tile of
//     K^, and two groups).
// Row tiles have 128 rows (64 at head_dim 256).  With many rows the epilogue bounds it, an exponential for
// every score: 64 tokens of 32 heads over 262,144 keys of 4, q8_0, take 183 us, 78% of the rate of
// the tensor cores' fp16 products, pairs counted (one group to a key tile: 252).  With few, each key is staged
// for a handful of rows: tiles of 32 rows then, 16 staging warps, one group to a key tile.  8 sequences
// of one token over 6,316 keys each take 19 us, 23 in tiles of 128 (and those 64 tokens 379 us in tiles of 32).  The choice goes by
// the rows of a sequence on average, which the host knows: 64 single tokens over 4,000 keys 65 us, 86 in tiles of 128;
// but with 190 tokens behind 30,000 among them, still 32 rows on average, 288 us, where tiles of 128 take 168.
// Of the 19 some 5 pass before the first page is there; then a tile is staged in 1,300 clocks, and 28 MB
// arrive in 10 us.
// The (key tile, KV head, sequence) items of the call lie behind one another on a line
// that the CTAs, one to an SM, share by their cost.
#include <algorithm>
#include <type_traits>

#include "key_weights.cuh"
#include "page_tiles.cuh"
#include "softmax_tile.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace memra {
namespace {

constexpr int kPieces = 4;
constexpr int kLseRows = 1024;             // rows of a chunk whose log-sum-exps stay in shared memory for a whole run of tiles

// A run of key tiles of one KV head of a sequence.
struct WeightPiece {
  int first, n;                 // rows of the chunk
  int T;
  int h, b;
  int tile0, tiles;             // tiles < 0: there is no more piece
  int row_tiles;
};

struct WeightSeq {
  int first, n, T;
  bool bad;
};

__device__ __forceinline__ WeightSeq weight_seq(const WeightParams &p, int b) {
  const int cs = p.cu_seqlens[b], ce = p.cu_seqlens[b + 1], T = p.seq_lens[b];
  WeightSeq s;
  s.first = min(max(cs, 0), p.total);
  s.n = min(max(ce, s.first), p.total) - s.first;
  s.T = max(0, min(T, p.len_limit));
  s.bad = s.first != cs || s.first + s.n != ce || s.T != T || T < s.n;
  return s;
}

// Tiles of a sequence's keys (none where the chunk has no row), and the cost of one: its row tiles and a fixed part.
__device__ __forceinline__ int weight_tiles(const WeightSeq &s) { return s.n > 0 && s.T > 0 ? (s.T - 1) / kWeightKeys + 1 : 0; }
__device__ __forceinline__ int weight_row_tiles(const WeightParams &p, int n) { return ((n - 1) / p.tpt + 1) * p.subs; }
__device__ __forceinline__ int64_t weight_cost(const WeightParams &p, const WeightSeq &s) {
  return s.n > 0 ? weight_row_tiles(p, s.n) + 1 : 1;
}

// Where a share begins: before a tile of a (head, sequence).
struct WeightPlace {
  int h, b, tile;
};

__device__ __forceinline__ int64_t weight_sum(int64_t x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// Whole warp: the cost of one KV head's tiles.
__device__ __forceinline__ int64_t weight_head_cost(const WeightParams &p, int lane) {
  int64_t sum = 0;
  for (int b = lane; b < p.batch; b += 32) {
    const WeightSeq s = weight_seq(p, b);
    sum += weight_tiles(s) * weight_cost(p, s);
  }
  return weight_sum(sum);
}

// Whole warp: the first tile that starts at `pos` of the line or behind it.
__device__ __forceinline__ WeightPlace weight_place(const WeightParams &p, int64_t head_cost, int64_t pos, int lane) {
  WeightPlace w{static_cast<int>(pos / head_cost), 0, 0};
  const int64_t rest = pos % head_cost;
  int64_t start = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    const int b = b0 + lane;
    int64_t mine = 0, per = 1;
    if (b < p.batch) {
      const WeightSeq s = weight_seq(p, b);
      per = weight_cost(p, s);
      mine = weight_tiles(s) * per;
    }
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += up;
    }
    const int64_t at = rest - start - (incl - mine);
    const unsigned who = __ballot_sync(0xffffffffu, at >= 0 && at < mine);
    if (who) {
      const int src = __ffs(who) - 1;
      w.b = b0 + src;
      w.tile = static_cast<int>(__shfl_sync(0xffffffffu, (at + per - 1) / per, src));
      break;
    }
    start += __shfl_sync(0xffffffffu, incl, 31);
  }
  return w;
}

// Walks a CTA's share.
struct WeightWalk {
  const WeightParams &p;
  WeightPlace at, end;
  __device__ __forceinline__ bool next(WeightPiece &x) {
    while (true) {
      if (at.h > end.h || (at.h == end.h && (at.b > end.b || (at.b == end.b && at.tile >= end.tile)))) return false;
      const WeightSeq s = weight_seq(p, at.b);
      const int tiles = weight_tiles(s);
      const bool last = at.h == end.h && at.b == end.b;
      x.first = s.first, x.n = s.n, x.T = s.T;
      x.h = at.h, x.b = at.b;
      x.tile0 = at.tile;
      x.tiles = (last ? min(end.tile, tiles) : tiles) - at.tile;
      x.row_tiles = s.n > 0 ? weight_row_tiles(p, s.n) : 0;
      if (last)
        at.tile = end.tile;
      else {
        at.tile = 0;
        if (++at.b == p.batch) at.b = 0, ++at.h;
      }
      if (x.tiles > 0) return true;
    }
  }
};

template <int D, int KF, int N>
struct WeightCfg {
  static constexpr bool kKLo = KF == MEMRA_KV_Q8_0;
  static constexpr int kRows = N;          // query rows of a tile
  // Few rows: a key tile's time is its staging, so that twice as many warps stage, and one group takes its row tiles.
  static constexpr bool kFew = N == kWeightRowsFew;
  static constexpr int kStageWarps = kFew ? 16 : 8, kGroups = kFew ? 1 : 2;     // groups of the epilogue to a tile of K^
  // Keys of a raw chunk: as many as fit, for the loads that a staging warp has in flight between two waits.
  static constexpr int kStepKeys = (D == 128 ? 64 : 32) * (kFew ? 2 : 1), kTileSteps = kWeightKeys / kStepKeys;
  static constexpr int kTiles = D == 256 && kKLo ? 1 : 2;       // tiles of K^
  static constexpr int kEpilogue = 128 * kGroups * kTiles;      // threads
  static constexpr int kStageWarp0 = kEpilogue / 32, kMmaWarp = kStageWarp0 + kStageWarps, kLoadWarp = kMmaWarp + kTiles;
  static constexpr int kCopyWarp = kLoadWarp + 1, kThreads = 32 * (kCopyWarp + 1);
  static constexpr int kPages = kStepKeys / kPage;
  static constexpr int kKSeg = k_seg_bytes(KF, D);
  static constexpr int kBlocks = D / 64;                // 64-element column blocks of a row
  static constexpr uint32_t kTile = kWeightKeys * D * 2, kKBuf = kTile * (kKLo ? 2 : 1);
  static constexpr uint32_t kQBuf = kRows * D * 2, kRawBytes = kPages * kKSeg;
  static constexpr uint32_t kRoom = 227 * 1024;
  // barriers, page masks, the share, the pieces; log-sum-exps (of the run's rows, or two row tiles of each group); half of
  // the sums of two tiles for each tile of K^; tiles of K^; Q; raw chunks
  static constexpr uint32_t kOffBar = 0, kOffMask = 384, kOffShare = 448, kOffPiece = 480, kOffLse = 1024;
  static constexpr uint32_t kOffSum = kOffLse + 4096, kOffK = kOffSum + 2048;
  static constexpr uint32_t kOffQ = kOffK + kTiles * kKBuf;
  // (two raw chunks at least beside the row tiles)
  static constexpr int kQMost = kFew ? 2 : 4, kQFit = (kRoom - 1024 - kOffQ - 2 * kRawBytes) / kQBuf;
  static constexpr int kQBufs = kQFit < kQMost ? kQFit : kQMost;
  static constexpr uint32_t kOffRaw = kOffQ + kQBufs * kQBuf;
  static constexpr int kRaw = (kRoom - 1024 - kOffRaw) / kRawBytes < 8 ? (kRoom - 1024 - kOffRaw) / kRawBytes : 8;
  static constexpr uint32_t kTCols = 512, kNeed = kOffRaw + kRaw * kRawBytes + 1024, kFloor = 150 * 1024;      // (1024: aligning the base)
  static constexpr uint32_t kSmem = kNeed < kFloor ? kFloor : kNeed;
  enum Bar { kRawFull = 0, kRawEmpty = kRawFull + kRaw, kKFull = kRawEmpty + kRaw, kKFree = kKFull + 2, kQFull = kKFree + 2,
             kQFree = kQFull + kQBufs, kSFull = kQFree + kQBufs, kSFree = kSFull + 4, kDrained = kSFree + 4, kPieceFull = kDrained + 2,
             kPieceFree = kPieceFull + kPieces, kBars = kPieceFree + kPieces };
  static_assert(kQBufs >= 1 && kRaw >= 1, "rings");
  static_assert(kOffBar + 8 * kBars + 4 <= kOffMask, "barriers and the tensor-memory address");
  static_assert(kOffPiece + kPieces * sizeof(WeightPiece) <= kOffLse, "pieces");
  static_assert(kTiles * 4 * kRows <= kLseRows && kLseRows * 4 <= 4096 && kTiles * 2 * kWeightKeys * 4 <= 2048, "log-sum-exps, sums");
  static_assert(kTiles * 2 * kRows <= 512, "tensor memory");
  static_assert(kOffK % 1024 == 0 && kQBuf % 1024 == 0 && kOffRaw % 16 == 0 && kSmem <= 232448, "alignment, shared memory");
};

// Row tiles of a chunk that may see the keys from `key0` on: the first of them.
__device__ __forceinline__ int weight_first_row_tile(const WeightParams &p, int n, int T, int key0) {
  const int t = key0 - (T - n);                        // the first token that sees key0
  return t > 0 ? t / p.tpt * p.subs : 0;
}

template <int D, int KF, int N>
__global__ void __launch_bounds__(WeightCfg<D, KF, N>::kThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap qmap, const WeightParams p) {
  using C = WeightCfg<D, KF, N>;
  constexpr int G = C::kTiles, GP = C::kGroups, SW = C::kStageWarps, NP = C::kPages, RAW = C::kRaw, QB = C::kQBufs;
  constexpr int kStepKeys = C::kStepKeys, kTileSteps = C::kTileSteps;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](int which, int i) { return sb + C::kOffBar + 8 * (which + i); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffBar + 8 * C::kBars);
  volatile uint8_t *page_mask = smem + C::kOffMask;
  WeightPlace *share = reinterpret_cast<WeightPlace *>(smem + C::kOffShare);
  WeightPiece *pieces = reinterpret_cast<WeightPiece *>(smem + C::kOffPiece);

  if (warp == C::kCopyWarp) {
    if (lane == 0) {
      for (int i = 0; i < RAW; ++i) {
        mbar_init(bar(C::kRawFull, i), 1);
        mbar_init(bar(C::kRawEmpty, i), SW);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(C::kKFull, i), SW);
        mbar_init(bar(C::kKFree, i), 1);
      }
      for (int i = 0; i < QB; ++i) {
        mbar_init(bar(C::kQFull, i), 1);
        mbar_init(bar(C::kQFree, i), G);
      }
      for (int i = 0; i < 4; ++i) {
        mbar_init(bar(C::kSFull, i), 1);
        mbar_init(bar(C::kSFree, i), 4);
      }
      for (int i = 0; i < G; ++i) mbar_init(bar(C::kDrained, i), 1);
      for (int i = 0; i < kPieces; ++i) {
        mbar_init(bar(C::kPieceFull, i), 1);
        mbar_init(bar(C::kPieceFree, i), C::kCopyWarp);          // every other warp
      }
      fence_barrier_init();
    }
  } else if (warp == C::kMmaWarp) {
    tc::tmem_alloc(smem_addr(tmem_slot), C::kTCols);
    tc::tmem_relinquish();
  }
  grid_dependency_wait();
  allow_dependent_launch();
  // The share's two ends, by a warp each.
  if (warp < 2) {
    const int64_t head = weight_head_cost(p, lane), all = head * p.n_kv_heads;
    const int c = blockIdx.x + warp, n = p.ctas;
    WeightPlace at = warp == 0 ? WeightPlace{0, 0, 0} : WeightPlace{head > 0 ? p.n_kv_heads : -1, 0, 0};
    if (head > 0 && c > 0 && c < n) at = weight_place(p, head, all * c / n, lane);
    if (lane == 0) share[warp] = at;
  } else if (warp == 2 && blockIdx.x == 0) {           // one CTA checks every length
    for (int b = lane; b < p.batch; b += 32)
      if (weight_seq(p, b).bad) flag_error(p.status, MEMRA_DEVERR_BAD_SEQ_LEN);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;
  int piece = 0;
  // The next piece, for the warps that are told of it (one thread of some); and that this warp is done with one.
  auto next_piece = [&]() -> const volatile WeightPiece * {
    const int i = piece % kPieces;
    ok = ok && mbar_wait_suspended(bar(C::kPieceFull, i), (piece / kPieces) & 1, p.status);
    return pieces + i;
  };
  auto free_piece = [&] {
    mbar_arrive(bar(C::kPieceFree, piece % kPieces));
    ++piece;
  };
  // Row tile rt: its first token in the chunk, the first of its heads, and its rows.
  // (a token's heads are one tile's but for groups wider than a tile: no division then)
  auto tokens_of = [&](int rt) { return (p.subs == 1 ? rt : rt / p.subs) * p.tpt; };
  auto heads_of = [&](int rt) { return p.subs == 1 ? 0 : rt % p.subs * p.hpt; };
  auto rows_of = [&](int rt, int n) {
    return min(p.tpt, n - tokens_of(rt)) * p.hpt - max(0, heads_of(rt) + p.hpt - p.group);
  };

  if (warp == C::kCopyWarp) {
    // ----------------------------------------------------------------- copies --
    WeightWalk walk{p, share[0], share[1]};
    WeightPiece x;
    int cc = 0;                              // raw chunks so far
    while (ok) {
      const bool more = walk.next(x);
      if (!more) x.tiles = -1;
      const int at = piece % kPieces;
      if (piece >= kPieces) ok = mbar_wait_suspended(bar(C::kPieceFree, at), (piece / kPieces - 1) & 1, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) {
        pieces[at] = x;
        mbar_arrive(bar(C::kPieceFull, at));
      }
      __syncwarp();
      ++piece;
      if (!more) break;
      const int32_t *table = p.page_table + static_cast<size_t>(x.b) * p.max_pages;
      const int steps = kTileSteps * x.tiles;
      // Page id of a logical page, -1: none (past the keys or outside the pool); 32 pages are read at a time, ahead.
      auto page_id = [&](int step) {
        const int i = (kTileSteps * x.tile0 + step) * NP + (lane & (NP - 1));
        if (step >= steps || i > (x.T - 1) / kPage) return -1;
        const int pid = table[i];
        if (pid >= 0 && pid < p.num_pages) return pid;
        flag_error(p.status, MEMRA_DEVERR_BAD_PAGE);
        return -1;
      };
      constexpr int kAhead = 32 / NP;
      int ids = page_id(lane / NP), ahead = page_id(kAhead + lane / NP);
      for (int i = 0; i < steps; ++i, ++cc) {
        if (i > 0 && i % kAhead == 0) {
          ids = ahead;
          ahead = page_id(i + kAhead + lane / NP);
        }
        int pid = __shfl_sync(0xffffffffu, ids, (i % kAhead) * NP + (lane & (NP - 1)));
        if (lane >= NP) pid = -1;
        const int s = cc % RAW;
        if (cc >= RAW) ok = mbar_wait_suspended(bar(C::kRawEmpty, s), (cc / RAW - 1) & 1, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t there = __ballot_sync(0xffffffffu, pid >= 0);
        if (lane == 0) {
          page_mask[cc & 63] = static_cast<uint8_t>(there);
          if (there)
            mbar_arrive_expect_tx(bar(C::kRawFull, s),
                                  __popc(there) * C::kKSeg + (cc == 0 && blockIdx.x == 0 ? p.test_extra_tx : 0));
          else
            mbar_arrive(bar(C::kRawFull, s));
        }
        __syncwarp();
        if (pid >= 0)
          bulk_copy_g2s_nohint(sb + C::kOffRaw + s * C::kRawBytes + lane * C::kKSeg,
                               p.k_pool + (static_cast<size_t>(pid) * p.n_kv_heads + x.h) * C::kKSeg, C::kKSeg,
                               bar(C::kRawFull, s));
      }
    }
    // every copy has landed before the CTA can leave
    for (int c = max(0, cc - RAW); c < cc; ++c) mbar_wait_suspended(bar(C::kRawFull, c % RAW), (c / RAW) & 1, p.status);
    __syncwarp();
  } else if (warp == C::kLoadWarp) {
    // ---------------------------------------------------------------- Q tiles --
    if (tc::elect_one()) {
      int qn = 0;                            // loads so far
      auto load = [&](const volatile WeightPiece *x, int rt) {
        const int s = qn % QB;
        if (ok && qn >= QB) ok = mbar_wait_suspended(bar(C::kQFree, s), (qn / QB - 1) & 1, p.status);
        if (!ok) return;
        mbar_arrive_expect_tx(bar(C::kQFull, s), static_cast<uint32_t>(p.hpt * p.tpt) * 128 * C::kBlocks);
#pragma unroll
        for (int c = 0; c < C::kBlocks; ++c)
          tma_load_3d(sb + C::kOffQ + s * C::kQBuf + c * N * 128, &qmap, 64 * c, x->h * p.group + heads_of(rt),
                      x->first + tokens_of(rt), bar(C::kQFull, s));
        ++qn;
      };
      while (true) {
        const volatile WeightPiece *x = next_piece();
        if (!ok || x->tiles < 0) break;
        const int tiles = x->tiles, rts = x->row_tiles, n = x->n, T = x->T, tile0 = x->tile0;
        const int first = weight_first_row_tile(p, n, T, tile0 * kWeightKeys);
        if (rts - first <= QB) {             // all that the run needs fit: once
          for (int rt = first; rt < rts && ok; ++rt) load(x, rt);
        } else {
          for (int t = 0; t < tiles && ok; t += G)
            for (int rt = weight_first_row_tile(p, n, T, (tile0 + t) * kWeightKeys); rt < rts && ok; ++rt) load(x, rt);
        }
        free_piece();
      }
      for (int c = max(0, qn - QB); c < qn; ++c) mbar_wait_suspended(bar(C::kQFull, c % QB), (c / QB) & 1, p.status);
    }
    __syncwarp();
  } else if (warp >= C::kMmaWarp) {
    // -------------------------------------------------------------------- MMA --
    if (tc::elect_one()) {
      const int g = warp - C::kMmaWarp;                // the tile of K^
      const uint64_t kd = tc::smem_desc_sw128(sb + C::kOffK + g * C::kKBuf, 16, 1024);
      const uint64_t qd0 = tc::smem_desc_sw128(sb + C::kOffQ, 16, 1024);
      int qn = 0, kn = 0, sn = 0;                      // loads of Q, tiles of K^ and score buffers used
      auto wait = [&](int which, int i, int phase) { ok = ok && mbar_wait_suspended(bar(which, i), phase & 1, p.status); };
      while (true) {
        const volatile WeightPiece *x = next_piece();
        if (!ok || x->tiles < 0) break;
        const int tiles = x->tiles, rts = x->row_tiles, n = x->n, T = x->T, tile0 = x->tile0;
        const int first = weight_first_row_tile(p, n, T, tile0 * kWeightKeys);
        const bool held = rts - first <= QB;
        for (int t = 0; t < tiles && ok; t += G) {
          const int low = weight_first_row_tile(p, n, T, (tile0 + t) * kWeightKeys);
          const bool any = t + g < tiles;
          for (int rt = low; rt < rts; ++rt) {
            const int use = held ? qn + rt - first : qn, qs = use % QB, sbuf = 2 * g + (sn & 1);
            // (Without a tile too: a slot is freed once by each for every load, and only after it.)
            wait(C::kQFull, qs, use / QB);
            if (!ok) break;
            if (any) {
              const uint32_t idesc = tc::idesc_f16_f32(kWeightKeys, (rows_of(rt, n) + 15) & ~15);
              const uint64_t qd = tc::desc_at(qd0, qs * C::kQBuf);
              if (rt == low) wait(C::kKFull, g, kn);
              if (sn >= 2) wait(C::kSFree, sbuf, (sn >> 1) - 1);
              if (!ok) break;
              tc::fence_after_sync();
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint64_t bd = tc::desc_at(qd, (ks / 4) * N * 128 + (ks % 4) * 32);
#pragma unroll
                for (int lo = 0; lo < (C::kKLo ? 2 : 1); ++lo)
                  tc::mma_f16(tmem + sbuf * N, tc::desc_at(kd, (ks / 4) * kWeightKeys * 128 + (ks % 4) * 32 + lo * C::kTile),
                              bd, idesc, ks + lo > 0);
              }
              tc::commit(bar(C::kSFull, sbuf));
              ++sn;
              if (rt == rts - 1) {
                tc::commit(bar(C::kKFree, g));
                ++kn;
              }
            }
            if (!held) {
              tc::commit(bar(C::kQFree, qs));
              ++qn;
            }
          }
        }
        if (held && ok) {
          for (int rt = first; rt < rts; ++rt) tc::commit(bar(C::kQFree, (qn + rt - first) % QB));
          qn += rts - first;
        }
        free_piece();
      }
      tc::commit(bar(C::kDrained, g));       // what was issued completes before the CTA can leave
      mbar_wait_suspended(bar(C::kDrained, g), 0, p.status);
    }
    __syncwarp();
  } else if (warp >= C::kStageWarp0) {
    // ---------------------------------------------------------------- staging --
    const int sw = warp - C::kStageWarp0;
    int cc = 0, kn[2] = {0, 0};              // raw chunks, and uses of each tile of K^ so far
    while (true) {
      const volatile WeightPiece *x = next_piece();
      ok = __all_sync(0xffffffffu, ok);
      const int tiles = ok ? x->tiles : -1;
      if (tiles < 0) break;
      __syncwarp();
      if (lane == 0) free_piece(); else ++piece;
      for (int t = 0; t < tiles && ok; ++t) {
        const int g = t % G;
        if (kn[g] > 0) ok = mbar_wait_suspended(bar(C::kKFree, g), (kn[g] - 1) & 1, p.status);
        ++kn[g];
#pragma unroll 1
        for (int i = 0; i < kTileSteps; ++i, ++cc) {
          const int s = cc % RAW;
          if (ok) ok = mbar_wait_suspended(bar(C::kRawFull, s), (cc / RAW) & 1, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          stage_k<D, KF, kStepKeys, SW, kWeightKeys>(sb + C::kOffRaw + s * C::kRawBytes,
                                                    sb + C::kOffK + g * C::kKBuf + i * kStepKeys * 128, sw, lane);
          fence_proxy_async();               // K^ for the tensor cores, the raw chunk for the next copies
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kRawEmpty, s));
        }
        if (ok && lane == 0) mbar_arrive(bar(C::kKFull, g));
      }
    }
  } else {
    // --------------------------------------------------------------- epilogue --
    // Group, its tile of K^ and which of the tile's units it takes, key of the tile.
    const int group = warp >> 2, g = group / GP, turn = group % GP, kl = tid & 127;
    const uint32_t tlane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float *const lse_all = reinterpret_cast<float *>(smem + C::kOffLse), *const lse_two = lse_all + group * 2 * N;
    float *const half_s = reinterpret_cast<float *>(smem + C::kOffSum) + g * 2 * kWeightKeys + kl;
    const uint64_t scale2 = pack_f2(p.scale_log2, p.scale_log2);
    int sn = 0, cc = 0, tn = 0;              // units of this tile of K^ so far, raw chunks, tiles
    while (true) {
      const volatile WeightPiece *x = next_piece();
      ok = named_barrier_and(7, C::kEpilogue, ok);          // all groups go on together, or none
      if (!ok || x->tiles < 0) break;
      const int tiles = x->tiles, rts = x->row_tiles, n = x->n, T = x->T, tile0 = x->tile0;
      float *const row = p.weights + (static_cast<int64_t>(x->b) * p.n_kv_heads + x->h) * p.weight_stride;
      const float *const lse_rows = p.lse + static_cast<int64_t>(x->first) * p.n_heads + x->h * p.group;
      // log-sum-exp of a column of a row tile, base 2, negated; none: -inf
      auto lse_of = [&](int rt, int col) {
        if (rt >= rts || col >= rows_of(rt, n)) return -INFINITY;
        return lse_rows[static_cast<int64_t>(tokens_of(rt) + col / p.hpt) * p.n_heads + heads_of(rt) + col % p.hpt] *
               -1.4426950408889634f;
      };
      // Where they fit, the run's are there once for all tiles.
      const int run_low = weight_first_row_tile(p, n, T, tile0 * kWeightKeys);
      const bool cached = (rts - run_low) * N <= kLseRows;
      if (cached) {
        for (int i = tid; i < (rts - run_low) * N; i += C::kEpilogue) lse_all[i] = lse_of(run_low + i / N, i % N);
        named_barrier_sync(7, C::kEpilogue);
      }
      for (int t = g; t < tiles; t += G, ++tn) {
        const int key = (tile0 + t) * kWeightKeys + kl;
        const int low = weight_first_row_tile(p, n, T, (tile0 + t / G * G) * kWeightKeys);
        int rt = low + (GP == 2 ? (sn ^ turn) & 1 : 0);          // this group's first
        float old = 0.f, next = 0.f, sum = 0.f;
        if (p.keep != 0.f && key < T) old = row[key];
        if (!cached && kl < N) next = lse_of(rt, kl);
        for (; rt < rts && ok; rt += GP) {
          const int nth = sn + rt - low, sbuf = 2 * g + (nth & 1);     // the unit's number
          const int live = rows_of(rt, n);
          const float *lse = lse_all + (rt - run_low) * N;
          if (!cached) {
            float *const mine = lse_two + (nth / GP & 1) * N;
            if (kl < N) {
              mine[kl] = next;
              next = lse_of(rt + GP, kl);
            }
            lse = mine;
          }
          ok = mbar_wait_suspended(bar(C::kSFull, sbuf), (nth >> 1) & 1, p.status);
          ok = cached ? __all_sync(0xffffffffu, ok) : named_barrier_and(1 + group, 128, ok);
          if (!ok) break;
          tc::fence_after_sync();
          const bool here = key < T && (page_mask[(cc + kTileSteps * t + kl / kStepKeys) & 63] >> (kl % kStepKeys / kPage) & 1);
          // columns from `from` on belong to tokens that see the key
          const int from = here ? min(max(0, key - (T - n) - tokens_of(rt)), N) * p.hpt : INT32_MAX;
          const bool whole = __all_sync(0xffffffffu, from <= 0);
          const uint32_t s_col = tmem + tlane + sbuf * N;
          uint64_t acc[2] = {0, 0};
          // 16 columns; `masked`: those that a key does not see, or behind the last, add nothing
          auto add = [&](const uint32_t(&s)[16], int c, auto masked) {
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 l = *reinterpret_cast<const float4 *>(lse + c + e);
              float w[4];
              unpack_f2(fma_f2(pack_f2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), scale2, pack_f2(l.x, l.y)), w[0], w[1]);
              unpack_f2(fma_f2(pack_f2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), scale2, pack_f2(l.z, l.w)), w[2], w[3]);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                w[k] = fast_exp2(w[k]);
                if constexpr (decltype(masked)::value) w[k] = c + e + k >= from && c + e + k < live ? w[k] : 0.f;
              }
              acc[0] = add_f2(acc[0], pack_f2(w[0], w[1]));
              acc[1] = add_f2(acc[1], pack_f2(w[2], w[3]));
            }
          };
          // the next columns' load in flight beside these ones' sums
          auto all = [&](auto masked) {
            uint32_t s0[16], s1[16];
            tc::ld_32x32b_x16(s_col, s0);
#pragma unroll 1
            for (int c = 0; c < live; c += 32) {
              tc::wait_ld(s0);
              tc::ld_32x32b_x16(s_col + c + 16, s1);
              add(s0, c, masked);
              tc::wait_ld(s1);
              if (c + 32 < live) tc::ld_32x32b_x16(s_col + c + 32, s0);
              add(s1, c + 16, masked);
            }
          };
          if (whole && live % 32 == 0) all(std::false_type{}); else all(std::true_type{});
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kSFree, sbuf));
          float a0, a1;
          unpack_f2(add_f2(acc[0], acc[1]), a0, a1);
          sum += a0 + a1;
        }
        // A tile of one unit is its group's; else the groups' sums are joined.
        const int units = rts - low;
        const bool mine = GP == 1 || (units > 1 ? turn == 0 : ((sn ^ turn) & 1) == 0);
        if (GP == 2 && units > 1) {
          float *const half = half_s + (tn & 1) * kWeightKeys;
          if (turn == 1) *half = sum;
          ok = named_barrier_and(5 + g, 256, ok);
          if (turn == 0) sum += *half;
        }
        sn += units;
        if (ok && mine && key < T) row[key] = p.keep != 0.f ? fmaf(p.keep, old, sum) : sum;
      }
      cc += kTileSteps * tiles;
      __syncwarp();
      if (lane == 0) free_piece(); else ++piece;
    }
    if (!ok) {
      // A wait gave up: every key of the CTA's share becomes NaN (some hold their new weights, others the old ones).
      WeightWalk walk{p, share[0], share[1]};
      WeightPiece x;
      while (walk.next(x)) {
        float *const row = p.weights + (static_cast<int64_t>(x.b) * p.n_kv_heads + x.h) * p.weight_stride;
        const int end = min(x.T, (x.tile0 + x.tiles) * kWeightKeys);
        for (int key = x.tile0 * kWeightKeys + tid; key < end; key += C::kEpilogue) row[key] = __uint_as_float(kNanPair);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == C::kMmaWarp) tc::tmem_dealloc(tmem, C::kTCols);
}

template <int D, int KF, int N>
cudaError_t launch_one(const WeightParams &p, cudaStream_t st) {
  using C = WeightCfg<D, KF, N>;
  auto kernel = key_weights_kernel<D, KF, N>;
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
  CUtensorMap qm;
  if (!encode_rows(&qm, p.q, D, p.n_heads, p.total, p.q_stride, p.hpt, p.tpt)) return cudaErrorInvalidValue;
  return launch_pdl(kernel, dim3(p.ctas), dim3(C::kThreads), C::kSmem, st, qm, p);
}

template <int D, int N>
cudaError_t launch_formats(int kf, const WeightParams &p, cudaStream_t st) {
  switch (kf) {
    case MEMRA_KV_Q8_0: return launch_one<D, MEMRA_KV_Q8_0, N>(p, st);
    case MEMRA_KV_FP8_E4M3: return launch_one<D, MEMRA_KV_FP8_E4M3, N>(p, st);
    case MEMRA_KV_NVFP4: return launch_one<D, MEMRA_KV_NVFP4, N>(p, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_key_weights(int D, int rows, int kf, const WeightParams &p, cudaStream_t st) {
  if (rows == kWeightRowsFew)
    return D == 128 ? launch_formats<128, kWeightRowsFew>(kf, p, st) : launch_formats<256, kWeightRowsFew>(kf, p, st);
  return D == 128 ? launch_formats<128, weight_rows(128)>(kf, p, st) : launch_formats<256, weight_rows(256)>(kf, p, st);
}

}  // namespace memra
