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
// its first store.
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

// Byte x (0 .. seg / 16 - 1) of token t's row in a page segment, by the layout
// of memra.h; x means the same part of the row for every t.
template <int D>
__device__ __forceinline__ int k_row_byte(int fmt, int t, int x) {
  constexpr int NB = D / 32;
  if (fmt == MEMRA_KV_NVFP4) {
    if (x < D / 2)
      return ((x >> 5) * 32 + 4 * (t & 7) + ((x >> 3) & 3)) * 16 + ((x >> 1) & 3) * 4 + (t >> 3) + 2 * (x & 1);
    return 8 * D + t * (D / 16) + (x - D / 2);
  }
  if (x < D) {
    const int b = x >> 5, r = x & 31;
    return (((t >> 3) * (NB / 2) + (b >> 1)) * 32 + 4 * (t & 7) + (r >> 3)) * 16 + (b & 1) * 8 + (r & 7);
  }
  return 16 * D + t * NB * 2 + (x - D);             // q8_0 scales
}

template <int D>
__device__ __forceinline__ int v_row_byte(int fmt, int t, int x) {
  constexpr int NB = D / 32;
  const int c = (t & 7) >> 1, f = t & 1, p = t >> 3, k = 2 * f + p;
  if (fmt == MEMRA_KV_FP8_E4M3)
    return ((x >> 5) * 32 + 4 * ((x >> 2) & 7) + c) * 16 + 8 * ((x >> 1) & 1) + 2 * (2 * p + (x & 1)) + f;
  if (fmt == MEMRA_KV_NVFP4) {
    if (x < D / 2) return ((x >> 5) * 32 + 4 * ((x >> 2) & 7) + c) * 16 + (x & 3) * 4 + f + 2 * p;
    return 8 * D + (c * (D / 16) + (x - D / 2)) * 4 + f + 2 * p;
  }
  if (x < D / 2) return ((x >> 5) * 32 + 4 * ((x >> 2) & 7) + c) * 16 + ((x >> 1) & 1) * 8 + 4 * (x & 1) + k;
  x -= D / 2;
  if (fmt == MEMRA_KV_Q5_1) {
    if (x < D / 8) return 8 * D + ((4 * (x / (NB / 2)) + c) * (NB / 2) + x % (NB / 2)) * 4 + k;
    x -= D / 8;
    const int m = x >= 2 * NB ? D : 0;               // the minima lie D bytes behind the scales
    x -= m ? 2 * NB : 0;
    return 10 * D + m + ((c * NB + (x >> 1)) * 4 + 2 * p + f) * 2 + (x & 1);
  }
  return 8 * D + ((c * NB + (x >> 1)) * 4 + 2 * p + f) * 2 + (x & 1);
}

constexpr int kCompactThreads = 256;

// CTA (KV head, sequence): every byte of the moved rows is read into shared
// memory before the first is written, so the accepted list may hold any order.
template <int D>
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactParams p) {
  extern __shared__ uint8_t buf[];
  __shared__ int from_page[MEMRA_MAX_TREE_NODES], to_page[MEMRA_MAX_TREE_NODES];
  __shared__ uint8_t from_t[MEMRA_MAX_TREE_NODES], to_t[MEMRA_MAX_TREE_NODES];
  grid_dependency_wait();
  allow_dependent_launch();
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int T = p.seq_lens[b], Tc = max(0, min(min(T, p.max_seq_len), static_cast<int>(min(
      static_cast<long long>(p.max_pages) * kPage, 2147483647ll))));
  const int n_acc = p.n_accepted[b], n = max(0, min(n_acc, p.max_accepted));
  const int base = Tc - p.n_nodes;
  const bool report = h == 0;
  if (report && tid == 0 && (Tc != T || T < p.n_nodes || n != n_acc)) flag_error(p.status, MEMRA_DEVERR_BAD_SEQ_LEN);
  if (tid < n) {
    const int node = p.accepted[static_cast<size_t>(b) * p.max_accepted + tid];
    int fp = -1, tp = -1;
    if (node < 0 || node >= p.n_nodes) {
      if (report) flag_error(p.status, MEMRA_DEVERR_BAD_SLOT);
    } else if (node != tid && base + node >= 0 && base + tid >= 0) {
      const int32_t *row = p.page_table + static_cast<size_t>(b) * p.max_pages;
      fp = row[(base + node) / kPage];
      tp = row[(base + tid) / kPage];
      if (fp < 0 || fp >= p.num_pages || tp < 0 || tp >= p.num_pages) {
        if (report) flag_error(p.status, MEMRA_DEVERR_BAD_PAGE);
        fp = -1;
      }
    }
    from_page[tid] = fp;
    to_page[tid] = tp;
    from_t[tid] = static_cast<uint8_t>((base + node) & (kPage - 1));
    to_t[tid] = static_cast<uint8_t>((base + tid) & (kPage - 1));
  }
  __syncthreads();
  const int kb = p.k_seg / kPage, rb = kb + p.v_seg / kPage;
  for (int i = tid; i < n * rb; i += kCompactThreads) {
    const int r = i / rb, x = i % rb;
    if (from_page[r] < 0) continue;
    const size_t at = static_cast<size_t>(from_page[r]) * p.n_kv_heads + h;
    buf[i] = x < kb ? p.k_pool[at * p.k_seg + k_row_byte<D>(p.k_fmt, from_t[r], x)]
                    : p.v_pool[at * p.v_seg + v_row_byte<D>(p.v_fmt, from_t[r], x - kb)];
  }
  __syncthreads();
  for (int i = tid; i < n * rb; i += kCompactThreads) {
    const int r = i / rb, x = i % rb;
    if (from_page[r] < 0) continue;
    const size_t at = static_cast<size_t>(to_page[r]) * p.n_kv_heads + h;
    if (x < kb)
      p.k_pool[at * p.k_seg + k_row_byte<D>(p.k_fmt, to_t[r], x)] = buf[i];
    else
      p.v_pool[at * p.v_seg + v_row_byte<D>(p.v_fmt, to_t[r], x - kb)] = buf[i];
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

cudaError_t launch_compact(int D, const CompactParams &p, int batch, cudaStream_t st) {
  // at most 64 rows of 2 x 272 bytes: within the 48 KB every launch may use
  const size_t smem = static_cast<size_t>(p.max_accepted) * (p.k_seg + p.v_seg) / kPage;
  const dim3 grid(static_cast<unsigned>(p.n_kv_heads), static_cast<unsigned>(batch));
  if (D == 128) return launch_pdl(compact_kernel<128>, grid, dim3(kCompactThreads), smem, st, p);
  return launch_pdl(compact_kernel<256>, grid, dim3(kCompactThreads), smem, st, p);
}

}  // namespace memra
