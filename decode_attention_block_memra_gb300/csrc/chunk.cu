// Chunk attention: the dispatch of the pass over the keys (chunk_kernel.cuh) and the
// merge of the blocks that more than one CTA worked on.
#include "chunk.cuh"
#include "softmax_tile.cuh"

namespace memra {
namespace {

// Whole warp: what the merge joins at the cut where CTA c's share begins (c > 0): pieces (0: nothing was cut
// there, or the cut is a later one of its block), KV head, first row and tokens.
template <int TILES>
__device__ __forceinline__ int4 chunk_merge_of(const ChunkParams &p, int c, int tpb, int lane) {
  const int64_t head = chunk_head_cost<TILES>(p, tpb, lane), all = head * p.n_kv_heads;
  const int n = chunk_shares<TILES>(p, head);
  if (head <= 0 || c >= n) return make_int4(0, 0, 0, 0);
  const ChunkCut x = chunk_cut<TILES>(p, head, all * c / n, tpb, lane);
  const int64_t before = all * (c - 1) / n - x.start;
  if (x.k <= 0 || x.k >= x.steps || (before > 0 && chunk_cut_step<TILES>(before, x.steps, x.step) != 0))
    return make_int4(0, 0, 0, 0);
  // the CTA before this cut has the block's head, the others a piece from their own cut on
  int pieces = 2;
  for (int d = c + 1; d < n; ++d) {
    const int64_t off = all * d / n - x.start;
    if (off >= x.cost || chunk_cut_step<TILES>(off, x.steps, x.step) >= x.steps) break;
    ++pieces;
  }
  const ChunkSeq s = chunk_seq(p, x.b);
  const ChunkBlock block = chunk_block(p, s, x.j, tpb);
  return make_int4(pieces, x.h, s.first + block.t0, block.t1 - block.t0);
}

// A warp for each cut.  A kernel of its own: the merge's CTAs, several one after another on an SM, would each find their
// cut in front of their loads (512 tokens beside 15 single ones over 60,000 keys: 123 us for 111), and in the pass it takes
// registers from the loops over the keys (2,048 tokens behind 30,000: 1,410 us for 1,350).
constexpr int kCutWarps = 8;
template <int D>
__global__ void __launch_bounds__(32 * kCutWarps) chunk_cuts_kernel(const ChunkParams p) {
  allow_dependent_launch();
  const int c = 1 + blockIdx.x * kCutWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  // (the pass has begun, so that what it reads is there, and what a call before has left is used up)
  const int4 merge = chunk_merge_of<chunk_tiles(D)>(p, c, chunk_tiles(D) * p.tpt, lane);
  if (lane == 0 && c < p.ctas) p.merges[c] = merge;
  grid_dependency_wait();                    // with this kernel the pass has ended
}

// CTA = 32 rows of a cut block, warp = 16 columns, thread = row.  The CTA of the
// block's first cut merges it, the pieces in their order along the keys.
template <int D>
__global__ void __launch_bounds__(2 * D) chunk_merge_kernel(const ChunkParams p) {
  constexpr int kRows = chunk_tiles(D) * kChunkRows, kSides = kRows / 32, BATCH = 2;
  const int c = 1 + blockIdx.x / kSides, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part_row = blockIdx.x % kSides * 32 + lane;
  const int rl = part_row % kChunkRows, tl = rl / p.group;
  grid_dependency_wait();                    // the partial blocks are complete
  allow_dependent_launch();
  const int4 merge = p.merges[c];
  const int pieces = merge.x, t = part_row / kChunkRows * p.tpt + tl;       // the row's token in the block
  const bool live = tl < p.tpt && t < merge.w;
  if (pieces == 0 || !__any_sync(0xffffffffu, live)) return;
  float mw = -INFINITY, L = 0.f, acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  for (int k0 = 0; k0 < pieces; k0 += BATCH) {
    float ls[BATCH];
    float4 x[BATCH][4];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const bool in = live && k0 + u < pieces;
      const int slot = k0 + u == 0 ? 2 * (c - 1) + 1 : 2 * (c + k0 + u - 1);
      ls[u] = in ? p.lse_part[static_cast<size_t>(slot) * kRows + part_row] : -INFINITY;
      const float4 *at = reinterpret_cast<const float4 *>(p.o_part) +
                         (static_cast<size_t>(slot) * (D / 4) + 4 * warp) * kRows + part_row;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[u][e] = in ? at[e * kRows] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      if (ls[u] == -INFINITY) continue;                // no visible key: its row may hold anything
      if (ls[u] > mw) {
        const float sc = fast_exp2(mw - ls[u]);
        L *= sc;
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] *= sc;
        mw = ls[u];
      }
      const float w = fast_exp2(ls[u] - mw);
      L += w;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[4 * e + 0] = fmaf(w, x[u][e].x, acc[4 * e + 0]);
        acc[4 * e + 1] = fmaf(w, x[u][e].y, acc[4 * e + 1]);
        acc[4 * e + 2] = fmaf(w, x[u][e].z, acc[4 * e + 2]);
        acc[4 * e + 3] = fmaf(w, x[u][e].w, acc[4 * e + 3]);
      }
    }
  }
  if (!live) return;
  const float inv = L != 0.f ? 1.f / L : 0.f;          // (0: no visible key; a NaN stays one)
  const int64_t row = static_cast<int64_t>(merge.z + t) * p.n_heads + merge.y * p.group + rl % p.group;
  uint4 *to = reinterpret_cast<uint4 *>(p.out + row * D + 16 * warp);
#pragma unroll
  for (int e = 0; e < 16; e += 8)
    to[e / 8] = make_uint4(pack_half2(acc[e] * inv, acc[e + 1] * inv), pack_half2(acc[e + 2] * inv, acc[e + 3] * inv),
                           pack_half2(acc[e + 4] * inv, acc[e + 5] * inv), pack_half2(acc[e + 6] * inv, acc[e + 7] * inv));
  if (warp == 0 && p.lse) p.lse[row] = L != 0.f ? (mw + log2f(L)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

cudaError_t launch_chunk(int D, int kf, int vf, const ChunkParams &p, cudaStream_t st) {
  switch (kf) {
    case MEMRA_KV_Q8_0: return launch_chunk_q8(D, vf, p, st);
    case MEMRA_KV_FP8_E4M3: return launch_chunk_fp8(D, vf, p, st);
    case MEMRA_KV_NVFP4: return launch_chunk_nvfp4(D, vf, p, st);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_chunk_merge(int D, const ChunkParams &p, cudaStream_t st) {
  if (p.ctas < 2) return cudaSuccess;
  const dim3 cuts((p.ctas - 1 + kCutWarps - 1) / kCutWarps), grid((p.ctas - 1) * (chunk_tiles(D) * kChunkRows / 32));
  auto run = [&](auto find, auto merge) {
    const cudaError_t e = launch_pdl(find, cuts, dim3(32 * kCutWarps), 0, st, p);
    return e != cudaSuccess ? e : launch_pdl(merge, grid, dim3(2 * D), 0, st, p);
  };
  return D == 128 ? run(chunk_cuts_kernel<128>, chunk_merge_kernel<128>) : run(chunk_cuts_kernel<256>, chunk_merge_kernel<256>);
}

}  // namespace memra
