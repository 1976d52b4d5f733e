// Chunk attention over the paged cache: how the work is cut, the parameters of its
// two kernels (the pass over the keys and the merge) and their launchers.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "memra_device.cuh"

namespace memra {

// Keys of one step (the N of the score MMA).
constexpr int kChunkKeys = 64;
constexpr int kChunkRows = 128;            // query rows of a tile: tokens x the group's heads
// Row tiles of a block (what a CTA holds at a time): two at head_dim 128.
__host__ __device__ constexpr int chunk_tiles(int D) { return D == 128 ? 2 : 1; }
// Columns of a row in the workspace: the output's, and at head_dim 128 those of the q5_1 blocks' centres.
__host__ __device__ constexpr int kChunkFarCols(int D) { return D + (D == 128 ? 16 : 0); }

// How the work is cut.  A block is a run of a sequence's tokens (its rows fill the
// row tiles) under one KV head, and costs a fixed part and its keys.  All blocks
// of the call, head by head and sequence by sequence, lie behind one another on a
// line that the CTAs share equally: a CTA takes whole blocks and, at either end of
// its share, a part of one, whose rows it leaves as partial sums.  So the GPU is
// evenly loaded whatever the lengths, one CTA to an SM, and no CTA leaves more
// than two partial blocks.
// A block's fixed cost, in keys (head_dim 128: 192 and 512 are within 4%; 256, chunks of 700, 1, 257 and 512 tokens that
// see 1,024 keys: 48 us with 704, 52 with 320 or 1,024).
__host__ __device__ constexpr int kChunkFixed(int tiles) { return tiles == 2 ? 320 : 704; }
// Least share of a CTA, in keys: the fixed cost and three steps.
__host__ __device__ constexpr int kChunkShareMin(int tiles) { return kChunkFixed(tiles) + 192; }
// A step of a block that has one row tile where there is room for two costs half of another's (512 tokens beside 15 single
// ones over 60,000 keys: 130 us; 138 with 3/4, 143 with 1,
// 151 with 3/8; the merge took 8 more than now).
constexpr int kChunkOneTileStep = kChunkKeys / 2;
// A block is cut at least this many steps from either end.
constexpr int kChunkSnap = 3;
constexpr int kChunkCtasMax = 160;

struct ChunkParams {
  const uint8_t *k_pool;
  const uint8_t *v_pool;
  const __half *q;              // token t's heads at q + t * q_stride
  int64_t q_stride;
  const int32_t *cu_seqlens;    // [batch + 1]
  const int32_t *page_table;    // [batch][max_pages]; a ring for a window
  const int32_t *seq_lens;
  __half *out;                  // [total][n_heads][D]
  float *lse;                   // [total][n_heads], or null
  float *o_part;                // [2 * CTAs][D / 4][rows of a block][4]: the partial blocks at a CTA's start and end
  float *lse_part;              // [2 * CTAs][rows of a block], base 2
  int4 *merges;                 // [CTAs]: the block that was cut where a CTA's share begins (chunk_merge_of)
  float *far;                   // [CTAs][row tiles][columns / 4][128][4]: what earlier sums of a long block came to
  int32_t *status;
  int batch, total, n_heads, group, n_kv_heads, num_pages, max_pages, window;
  int len_limit;                // lengths are clamped to it
  int tpt;                      // tokens of a row tile: 128 / group
  int ctas;                     // CTAs of the pass at most
  float scale_log2;             // sm_scale * (post-scale of the staged K values) * log2(e)
  float v_post;                 // post-scale of the staged V values
  int test_extra_tx;            // the test hook's: bytes that CTA 0 expects beyond its first chunk's (0 elsewhere)
};

// A sequence as the kernels use it.
struct ChunkSeq {
  int first, n;                 // first row and rows of its chunk
  int T;                        // keys: the context and the chunk
  bool bad;
};

__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams &p, int b) {
  const int cs = p.cu_seqlens[b], ce = p.cu_seqlens[b + 1], T = p.seq_lens[b];
  ChunkSeq s;
  s.first = min(max(cs, 0), p.total);
  s.n = min(max(ce, s.first), p.total) - s.first;
  s.T = max(0, min(T, p.len_limit));
  s.bad = s.first != cs || s.first + s.n != ce || s.T != T || T < s.n;
  // a ring must hold every key that the chunk sees
  if (p.window > 0 && s.T > 0 && s.n > 0) {
    const int low = max(0, s.T - s.n - p.window + 1);
    s.bad = s.bad || (s.T - 1) / kPage - low / kPage + 1 > p.max_pages;
  }
  return s;
}

// Block j of a sequence: its tokens and its steps over the keys.
struct ChunkBlock {
  int t0, t1;                   // tokens of the chunk
  int lo, hi;                   // steps of kChunkKeys keys; hi <= lo: no row sees a key
  int key0;                     // first key that a row sees
};

__device__ __forceinline__ ChunkBlock chunk_block(const ChunkParams &p, const ChunkSeq &s, int j, int tpb) {
  ChunkBlock k;
  k.t0 = j * tpb;
  k.t1 = min(s.n, k.t0 + tpb);
  const int last = s.T - s.n + k.t1;                   // keys that the last row sees end here
  k.key0 = p.window > 0 ? max(0, s.T - s.n + k.t0 - p.window + 1) : 0;
  k.lo = k.key0 / kChunkKeys;
  k.hi = last > 0 ? (last - 1) / kChunkKeys + 1 : 0;
  return k;
}

// Cost of a sequence's blocks: the fixed cost + 128 + min(A + (j + 1) tpb, M) for block
// j, which is more than its steps have keys, in a form that adds up without a loop.
template <int TILES>
struct ChunkCost {
  int64_t A, M, less;           // less: what the last block has not
  int tpb, blocks;
  static constexpr int kFixed = kChunkFixed(TILES);
  __device__ __forceinline__ ChunkCost(const ChunkParams &p, const ChunkSeq &s, int tpb_) : tpb(tpb_) {
    blocks = s.n > 0 ? (s.n - 1) / tpb + 1 : 0;
    A = max(0, s.T - s.n);
    M = p.window > 0 ? static_cast<int64_t>(p.window) + tpb : INT64_MAX;
    less = TILES == 2 && s.n - static_cast<int64_t>(blocks - 1) * tpb <= p.tpt ? min(A + static_cast<int64_t>(blocks) * tpb, M) / 2 : 0;
  }
  // of a step of block j
  __device__ __forceinline__ int step(int j) const { return less > 0 && j == blocks - 1 ? kChunkOneTileStep : kChunkKeys; }
  // of the first j blocks
  __device__ __forceinline__ int64_t upto(int j) const {
    const int64_t rising = M > A ? (M - A - 1) / tpb : 0, i = min(static_cast<int64_t>(j), rising);
    return j * static_cast<int64_t>(kFixed + 128) + i * A + tpb * (i * (i + 1) / 2) + (j - i ? (j - i) * M : 0) -
           (j == blocks ? less : 0);
  }
};

// A place where the line of all blocks is cut: before step `k` of a block, counted
// from the block's first; k = 0: between blocks.
struct ChunkCut {
  int h, b, j, k;
  int steps, step;              // of the block, and what one costs
  int64_t start, cost;          // of the block, on the line
};

// Steps of a block before a cut `off` behind its start: a block is cut only well inside.
template <int TILES>
__device__ __forceinline__ int chunk_cut_step(int64_t off, int steps, int step) {
  constexpr int fixed = kChunkFixed(TILES);
  const int64_t at = (off - fixed) / step;
  const int k = off <= fixed ? 0 : static_cast<int>(min(at, static_cast<int64_t>(steps)));
  if (steps < 2 * kChunkSnap) return 2 * k > steps ? steps : 0;
  return k < kChunkSnap ? 0 : steps - k < kChunkSnap ? steps : k;
}

// Whole warp: the cost of one KV head's blocks.
template <int TILES>
__device__ __forceinline__ int64_t chunk_head_cost(const ChunkParams &p, int tpb, int lane) {
  int64_t sum = 0;
  for (int b = lane; b < p.batch; b += 32) {
    const ChunkCost<TILES> c(p, chunk_seq(p, b), tpb);
    sum += c.upto(c.blocks);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return sum;
}

// CTAs that share the line, and where the c-th share begins.
template <int TILES>
__device__ __forceinline__ int chunk_shares(const ChunkParams &p, int64_t head_cost) {
  const int64_t want = head_cost * p.n_kv_heads / kChunkShareMin(TILES);
  return static_cast<int>(max(static_cast<int64_t>(1), min(want, static_cast<int64_t>(p.ctas))));
}

// Whole warp: the cut at `pos` of the line (0 <= pos < n_kv_heads * head_cost).
template <int TILES>
__device__ __forceinline__ ChunkCut chunk_cut(const ChunkParams &p, int64_t head_cost, int64_t pos, int tpb, int lane) {
  ChunkCut c{};
  c.h = static_cast<int>(pos / head_cost);
  int64_t rest = pos % head_cost, start = 0;
  c.start = pos - rest;
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    const int b = b0 + lane;
    int64_t mine = 0;
    if (b < p.batch) {
      const ChunkCost<TILES> cost(p, chunk_seq(p, b), tpb);
      mine = cost.upto(cost.blocks);
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
      rest = __shfl_sync(0xffffffffu, at, src);
      c.start += start + __shfl_sync(0xffffffffu, incl - mine, src);
      c.b = b0 + src;
      break;
    }
    start += __shfl_sync(0xffffffffu, incl, 31);
  }
  const ChunkSeq s = chunk_seq(p, c.b);
  const ChunkCost<TILES> cost(p, s, tpb);
  int lo = 0, hi = cost.blocks;              // upto(lo) <= rest < upto(hi)
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (cost.upto(mid) <= rest) lo = mid; else hi = mid;
  }
  c.j = lo;
  c.start += cost.upto(lo);
  c.cost = cost.upto(lo + 1) - cost.upto(lo);
  const ChunkBlock k = chunk_block(p, s, lo, tpb);
  c.steps = max(0, k.hi - k.lo);
  c.step = cost.step(lo);
  c.k = chunk_cut_step<TILES>(rest - cost.upto(lo), c.steps, c.step);
  return c;
}

cudaError_t launch_chunk(int D, int kf, int vf, const ChunkParams &p, cudaStream_t st);
cudaError_t launch_chunk_merge(int D, const ChunkParams &p, cudaStream_t st);

// of one K format each: a translation unit of its own
cudaError_t launch_chunk_q8(int D, int vf, const ChunkParams &p, cudaStream_t st);
cudaError_t launch_chunk_fp8(int D, int vf, const ChunkParams &p, cudaStream_t st);
cudaError_t launch_chunk_nvfp4(int D, int vf, const ChunkParams &p, cudaStream_t st);

}  // namespace memra
