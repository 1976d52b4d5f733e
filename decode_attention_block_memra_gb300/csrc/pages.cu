// Upkeep of the paged cache: copies of whole pages inside the pools (a fork's
// partial last page, copy on write, compaction of a pool) and the compaction
// of a verified tree (the accepted nodes' rows move to the front of the
// tree's rows).  Bytes move as they are: no value is decoded.
#include <cuda_runtime.h>

#include "pages.cuh"

namespace memra {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;                      // 16-byte units in flight per thread

// One page of a pool is n_kv_heads consecutive segments, so a page copy is one
// contiguous run per pool.  CTA = one page's run of kCopyThreads * kCopyUnroll
// 16-byte units (K's first, then V's), every load of a thread in flight before
// its first store.  Bound by HBM: 16,384 pages of 14,848 bytes in 73.2 us (6,650
// GB/s, 98% of the copy peak); a list of 16 pages takes 1.5 us in a replayed graph and
// 4.8 to 5.9 us as a call, which is the host's launch.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const CopyPagesParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  const uint32_t units = p.k_units + p.v_units;
  for (long long item = blockIdx.x; item < static_cast<long long>(p.n) * p.runs; item += gridDim.x) {
    const int i = static_cast<int>(item / p.runs), run = static_cast<int>(item % p.runs);
    const int src = p.src[i], dst = p.dst[i];
    if (src < 0 || dst < 0) continue;                // padding of the list
    if (src >= p.num_pages || dst >= p.num_pages) {
      if (threadIdx.x == 0) flag_error(p.status, MEMRA_DEVERR_BAD_PAGE);
      continue;
    }
    uint4 x[kCopyUnroll];
    uint4 *to[kCopyUnroll];
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j) {
      const uint32_t u = (run * kCopyUnroll + j) * kCopyThreads + threadIdx.x;
      to[j] = nullptr;
      if (u < units) {
        const bool v = u >= p.k_units;
        uint4 *pool = v ? p.v_pool : p.k_pool;
        const size_t per = v ? p.v_units : p.k_units, at = v ? u - p.k_units : u;
        x[j] = pool[src * per + at];
        to[j] = pool + dst * per + at;
      }
    }
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j)
      if (to[j]) *to[j] = x[j];
  }
}

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

// Thread = one byte of the row, for every moved row of a (sequence, KV head):
// it reads them all into registers, then writes them all, and no other thread
// touches its bytes, so the accepted list may hold any order and nothing waits.
// (A row's bytes are scattered over all of its page's sectors, so a page costs
// its whole traffic whatever moves; what counts is that the reads overlap.)  256
// sequences x up to 64 of 64 nodes, 2 heads, D 256, nvfp4/q4_0: 5 us, against 24.5
// us through shared memory with the byte's place computed for every row.
constexpr int kCompactThreads = 128;
constexpr int kRowsMax = MEMRA_MAX_TREE_NODES;

template <int D>
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactParams p) {
  __shared__ int s_from[kRowsMax], s_to[kRowsMax];           // pages of the moved rows
  __shared__ uint8_t s_from_t[kRowsMax], s_to_t[kRowsMax];
  __shared__ int s_n;
  grid_dependency_wait();
  allow_dependent_launch();
  const int b = blockIdx.y, tid = threadIdx.x;
  const int h = blockIdx.x / p.parts, x0 = blockIdx.x % p.parts * kCompactThreads + tid;
  const bool report = blockIdx.x == 0;
  if (tid < 32) {
    // one warp lists the rows that move, in any order of the list
    const int T = p.seq_lens[b], Tc = max(0, min(min(T, p.max_seq_len), static_cast<int>(min(
        static_cast<long long>(p.max_pages) * kPage, 2147483647ll))));
    const int n_acc = p.n_accepted[b], n = max(0, min(n_acc, p.max_accepted));
    const int base = Tc - p.n_nodes;
    if (report && tid == 0 && (Tc != T || T < p.n_nodes || n != n_acc)) flag_error(p.status, MEMRA_DEVERR_BAD_SEQ_LEN);
    int moved = 0;
#pragma unroll
    for (int i0 = 0; i0 < kRowsMax; i0 += 32) {
      const int i = i0 + tid;
      int fp = -1, tp = -1, node = 0;
      if (i < n) {
        node = p.accepted[static_cast<size_t>(b) * p.max_accepted + i];
        if (node < 0 || node >= p.n_nodes) {
          if (report) flag_error(p.status, MEMRA_DEVERR_BAD_SLOT);
        } else if (node != i && base + node >= 0 && base + i >= 0) {
          const int32_t *row = p.page_table + static_cast<size_t>(b) * p.max_pages;
          fp = row[(base + node) / kPage];
          tp = row[(base + i) / kPage];
          if (fp < 0 || fp >= p.num_pages || tp < 0 || tp >= p.num_pages) {
            if (report) flag_error(p.status, MEMRA_DEVERR_BAD_PAGE);
            fp = -1;
          }
        }
      }
      const unsigned m = __ballot_sync(0xffffffffu, fp >= 0);
      if (fp >= 0) {
        const int at = moved + __popc(m & ((1u << tid) - 1u));
        s_from[at] = fp;
        s_to[at] = tp;
        s_from_t[at] = static_cast<uint8_t>((base + node) & (kPage - 1));
        s_to_t[at] = static_cast<uint8_t>((base + i) & (kPage - 1));
      }
      moved += __popc(m);
    }
    if (tid == 0) s_n = moved;
  }
  __syncthreads();
  const int n = s_n, kb = p.k_seg / kPage, rb = kb + p.v_seg / kPage;
  if (x0 >= rb || n == 0) return;
  int part;
  const bool v = x0 >= kb;
  const int at = v ? v_byte<D>(p.v_fmt, x0 - kb, part) : k_byte<D>(p.k_fmt, x0, part);
  const int seg = v ? p.v_seg : p.k_seg;
  uint8_t *mine = (v ? p.v_pool : p.k_pool) + static_cast<size_t>(h) * seg + at;
  const size_t stride = static_cast<size_t>(p.n_kv_heads) * seg;
  uint8_t y[kRowsMax];
#pragma unroll
  for (int r0 = 0; r0 < kRowsMax; r0 += 8)
    if (r0 < n) {
#pragma unroll
      for (int r = r0; r < r0 + 8; ++r)
        if (r < n) y[r] = mine[s_from[r] * stride + token_offset<D>(part, s_from_t[r])];
    }
#pragma unroll
  for (int r0 = 0; r0 < kRowsMax; r0 += 8)
    if (r0 < n) {
#pragma unroll
      for (int r = r0; r < r0 + 8; ++r)
        if (r < n) mine[s_to[r] * stride + token_offset<D>(part, s_to_t[r])] = y[r];
    }
}

}  // namespace

cudaError_t launch_copy_pages(CopyPagesParams p, cudaStream_t st) {
  constexpr uint32_t kRun = kCopyThreads * kCopyUnroll;
  p.runs = (p.k_units + p.v_units + kRun - 1) / kRun;
  const long long items = static_cast<long long>(p.n) * p.runs;
  const unsigned grid = static_cast<unsigned>(items < (1ll << 30) ? items : (1ll << 30));
  return launch_pdl(copy_pages_kernel, dim3(grid), dim3(kCopyThreads), 0, st, p);
}

cudaError_t launch_compact(int D, CompactParams p, int batch, cudaStream_t st) {
  p.parts = ((p.k_seg + p.v_seg) / kPage + kCompactThreads - 1) / kCompactThreads;
  const dim3 grid(static_cast<unsigned>(p.n_kv_heads) * p.parts, static_cast<unsigned>(batch));
  if (D == 128) return launch_pdl(compact_kernel<128>, grid, dim3(kCompactThreads), 0, st, p);
  return launch_pdl(compact_kernel<256>, grid, dim3(kCompactThreads), 0, st, p);
}

}  // namespace memra
