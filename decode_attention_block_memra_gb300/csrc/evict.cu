// Eviction: of each KV head's rows of a sequence, those with the largest weight
// move, in order, to the rows of other pages.
//
// n = min(T, budget) rows stay: the last `recent` of them, the first `sink`, and of
// the others (the middle) the m with the largest weight, the lower index where
// two weigh the same.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "evict.cuh"
#include "page_rows.cuh"

namespace memra {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBits = 11, kBins = 1 << kBits, kDigits = 3;       // 11 + 11 + 10 bits of a weight's key
constexpr int kClusterMax = 8;

// What a sequence keeps.
struct Share {
  int T, n, sink, recent;
  bool bad;
};

__device__ __forceinline__ Share share_of(const EvictParams &p, int b) {
  const int T = p.seq_lens[b], budget = p.budgets[b];
  Share s;
  s.T = max(0, min(T, p.len_limit));
  const int most = max(0, min(budget, p.max_budget));
  s.bad = s.T != T || most != budget;
  s.n = min(s.T, most);
  s.recent = min(p.recent, s.n);
  s.sink = min(p.sink, s.n - s.recent);
  return s;
}

// A weight as an integer of the same order; NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return w != w ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Inclusive sum over the CTA's threads; `total` the whole.
__device__ __forceinline__ int block_scan(int x, int *warp_sums, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += up;
  }
  __syncthreads();                         // (the sums of the scan before have been read)
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int s = warp_sums[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += up;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
  return x + (warp > 0 ? before : 0);
}

// The m-th largest key by digits, the highest first: a histogram of the digit over
// the keys that agree with the digits found, and the digit where the count from
// above passes m.  A cluster holds one (sequence, KV head), each CTA a run of the
// middle; the CTAs add up each other's histograms through shared memory.  The
// weights are read once a digit, from L2 after the first time.
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictParams p) {
  __shared__ int hist[kDigits][kBins];
  __shared__ int warp_sums[kWarps];
  __shared__ int found[2];                 // the digit, and how many of its keys are wanted
  __shared__ int counts[2];                // of this CTA's run: keys above the last one taken, keys equal to it
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = cluster.block_rank(), ranks = cluster.num_blocks();
  const int row = blockIdx.x / ranks, b = row / p.n_kv_heads;
  for (int i = tid; i < kDigits * kBins; i += kThreads) hist[i / kBins][i % kBins] = 0;
  if (tid < 2) counts[tid] = 0;
  grid_dependency_wait();
  allow_dependent_launch();
  const Share s = share_of(p, b);
  if (row % p.n_kv_heads == 0 && rank == 0 && tid == 0) {
    if (s.bad) flag_error(p.status, MEMRA_DEVERR_BAD_SEQ_LEN);
    if (p.new_lens) p.new_lens[b] = s.n;
  }
  const float *w = p.weights + static_cast<int64_t>(row) * p.weight_stride;
  const int middle = s.T - s.sink - s.recent, m = s.n - s.sink - s.recent;
  const int run = (middle + ranks - 1) / ranks, lo = s.sink + min(rank * run, middle),
            hi = s.sink + min((rank + 1) * run, middle);
  __syncthreads();

  // every key from `last` up is taken, and the first `ties` equal to it
  uint32_t last = 0;
  int ties = middle;
  if (m < middle) {                        // (the same for the whole cluster)
    uint32_t prefix = 0;
    int want = m;
#pragma unroll
    for (int digit = 0; digit < kDigits; ++digit) {
      constexpr int kShift[kDigits] = {21, 10, 0};
      const int shift = kShift[digit], bits = digit < 2 ? kBits : 10;
      for (int i = lo + tid; i < hi; i += kThreads) {
        const uint32_t key = key_of(w[i]);
        if (digit == 0 || (key >> (shift + bits)) == (prefix >> (shift + bits)))
          atomicAdd(&hist[digit][(key >> shift) & ((1 << bits) - 1)], 1);
      }
      cluster.sync();
      // two bins of each thread, from the highest down
      int count[2] = {0, 0};
      const int top = (1 << bits) - 1 - 2 * tid;
      if (top > 0) {
        for (int r = 0; r < ranks; ++r) {
          const int *h = cluster.map_shared_rank(&hist[digit][0], r);
          count[0] += h[top];
          count[1] += h[top - 1];
        }
      }
      int all;
      const int upto = block_scan(count[0] + count[1], warp_sums, all), above = upto - count[0] - count[1];
      if (want > above && want <= upto) {
        const bool one = want <= above + count[0];
        found[0] = one ? top : top - 1;
        found[1] = want - above - (one ? 0 : count[0]);
      }
      __syncthreads();
      if (want > 0) {
        prefix |= static_cast<uint32_t>(found[0]) << shift;
        want = found[1];
      }
    }
    last = prefix;
    ties = want;
    if (m == 0) last = 0xFFFFFFFFu, ties = 0;
  }
  // How many this CTA's run holds, and with those of the runs before it, where its rows go.
  int over = 0, equal = 0;
  for (int i = lo + tid; i < hi; i += kThreads) {
    const uint32_t key = key_of(w[i]);
    over += key > last;
    equal += key == last;
  }
  over = __reduce_add_sync(0xffffffffu, over);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if ((tid & 31) == 0) {
    atomicAdd(&counts[0], over);
    atomicAdd(&counts[1], equal);
  }
  cluster.sync();
  int over_before = 0, equal_before = 0;
  for (int r = 0; r < rank; ++r) {
    const int *c = cluster.map_shared_rank(&counts[0], r);
    over_before += c[0];
    equal_before += c[1];
  }
  cluster.sync();                          // no CTA leaves while another reads its shared memory

  int32_t *kept = p.kept + static_cast<int64_t>(row) * p.max_budget;
  float *new_w = p.new_weights ? p.new_weights + static_cast<int64_t>(row) * p.new_stride : nullptr;
  auto keep = [&](int at, int i, float x) {
    kept[at] = i;
    if (new_w) new_w[at] = x;
  };
  if (rank == 0) {
    for (int i = tid; i < s.sink; i += kThreads) keep(i, i, w[i]);
    for (int i = tid; i < s.recent; i += kThreads) keep(s.n - s.recent + i, s.T - s.recent + i, w[s.T - s.recent + i]);
    for (int i = s.n + tid; i < p.max_budget; i += kThreads) kept[i] = -1;
  }
  for (int i0 = lo; i0 < hi; i0 += kThreads) {
    const int i = i0 + tid;
    const float x = i < hi ? w[i] : 0.f;
    const uint32_t key = key_of(x);
    const bool above = i < hi && key > last, same = i < hi && key == last;
    int all;
    // (both counts in one scan: a CTA has 1,024 threads)
    const int sum = block_scan(above | same << 16, warp_sums, all);
    const int overs = over_before + (sum & 0xFFFF), equals = equal_before + (sum >> 16);
    if (above || (same && equals <= ties))
      keep(s.sink + overs + min(equals, ties) - 1, i, x);
    over_before += all & 0xFFFF;
    equal_before += all >> 16;
  }
}

// The kept rows to their new pages, byte for byte.  CTA = one page of one KV head,
// thread = one byte position of a row, which it reads for the page's 16 rows before
// it writes any.
constexpr int kMoveThreads = 128;

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
  __shared__ int s_page[kPage], s_token[kPage];
  grid_dependency_wait();
  allow_dependent_launch();
  const int tid = threadIdx.x, page = blockIdx.x, h = blockIdx.y % p.n_kv_heads, b = blockIdx.y / p.n_kv_heads;
  const int n = share_of(p, b).n;
  if (page * kPage >= n) return;
  const int rows = min(kPage, n - page * kPage);
  const int to = p.dst_table[static_cast<int64_t>(b) * p.dst_pages + page];
  const bool to_ok = to >= 0 && to < p.num_pages;
  if (tid < kPage) {
    int from = -1, t = 0;
    if (tid < rows) {
      const int i = p.kept[(static_cast<int64_t>(b) * p.n_kv_heads + h) * p.max_budget + page * kPage + tid];
      from = p.page_table[static_cast<int64_t>(b) * p.max_pages + i / kPage];
      t = i % kPage;
      if (from < 0 || from >= p.num_pages) from = -1;
      if (from < 0 || !to_ok) flag_error(p.status, MEMRA_DEVERR_BAD_PAGE);
    }
    s_page[tid] = from;
    s_token[tid] = t;
  }
  __syncthreads();
  if (!to_ok) return;
  const int kb = p.k_seg / kPage, rb = kb + p.v_seg / kPage;
  for (int x = tid; x < rb; x += kMoveThreads) {
    int part;
    const bool v = x >= kb;
    const int at = v ? v_byte<D>(p.v_fmt, x - kb, part) : k_byte<D>(p.k_fmt, x, part);
    const int seg = v ? p.v_seg : p.k_seg;
    uint8_t *mine = (v ? p.v_pool : p.k_pool) + static_cast<size_t>(h) * seg + at;
    const size_t stride = static_cast<size_t>(p.n_kv_heads) * seg;
    uint8_t y[kPage];
#pragma unroll
    for (int r = 0; r < kPage; ++r)
      if (s_page[r] >= 0) y[r] = mine[s_page[r] * stride + token_offset<D>(part, s_token[r])];
#pragma unroll
    for (int r = 0; r < kPage; ++r)
      if (s_page[r] >= 0) mine[to * stride + token_offset<D>(part, r)] = y[r];
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictParams &p, int sms, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(p.batch) * p.n_kv_heads;
  // CTAs for the weights of one row: 4,096 of them each, as long as there are SMs
  int ranks = 1;
  while (ranks < kClusterMax && 4096ll * ranks < p.max_seq_len && 2 * ranks * rows <= 2 * sms) ranks *= 2;
  if (rows * ranks > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
}

cudaError_t launch_evict_move(int D, const EvictParams &p, cudaStream_t st) {
  const dim3 grid((p.max_budget + kPage - 1) / kPage, static_cast<unsigned>(p.batch) * p.n_kv_heads);
  if (D == 128) return launch_pdl(evict_move_kernel<128>, grid, dim3(kMoveThreads), 0, st, p);
  return launch_pdl(evict_move_kernel<256>, grid, dim3(kMoveThreads), 0, st, p);
}

}  // namespace memra
