// Eviction: of each KV head's rows of a sequence, those with the largest weight
// move, in order, to the rows of other pages.
//
// n = min(T, budget) rows stay: the last `recent` of them, the first `sink`, and of
// the others (the middle) the m with the largest weight, the lower index where
// two weigh the same.
//
// Two kernels: who stays, which is a chain of latencies (a read of the weights, four rounds over a
// cluster), and their rows' move, which is bytes.  q8_0/q5_1, D 128, with the graph's launches:
// 262,144 keys of 4 heads to 16,384 35 us (16 to select, 19 to move 15 MB), 16 sequences of up to
// 8,192 to 2,048 24 us (7 and 17 for 29 MB), one of 512 with 2 heads to 256 8 us.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "evict.cuh"

namespace memra {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBits = 8, kBins = 1 << kBits, kDigits = 32 / kBits;     // digits of a weight's key
constexpr int kClusterMax = 16;             // (more than 8 needs the kernel's leave)

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

// Inclusive sum over the CTA's threads.
template <class T>
__device__ __forceinline__ T block_scan(T x, T *warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T up = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += up;
  }
  __syncthreads();                         // (the sums of the scan before have been read)
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  T s = warp_sums[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T up = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += up;
  }
  const T before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
  return x + (warp > 0 ? before : T{0});
}

// Of up to 1,024 keys (one a thread): the m-th largest, bit by bit, by how many reach a candidate.
__device__ __forceinline__ uint32_t nth_key_by_bits(uint32_t key, bool in, int m, int &ties) {
  uint32_t prefix = 0;
  int above = 0;                           // keys of a higher prefix
#pragma unroll 1
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t want = prefix | 1u << bit;
    const int n = __syncthreads_count(in && (key >> bit) == (want >> bit));
    if (above + n >= m) prefix = want; else above += n;
  }
  ties = m - above;
  return prefix;
}

// The m-th largest key of the middle, and who is kept.  E = 1: one CTA has a key to a
// thread and finds it bit by bit.  Else by digits, the highest first: a histogram of the
// digit over the keys that agree with the digits found, and the digit where the
// count from above passes m.  A cluster holds one (sequence, KV head), each CTA a run of
// the middle; every CTA adds up all histograms through shared memory, those of the runs before its
// own also apart: they say where its rows go.  A CTA's keys are read once, E to a thread, all loads in
// flight, and stay in registers (longer runs: read again from L2 for each digit).
// Four digits of 8 bits: three of 11 take a round less, but a CTA then reads eight times the
// counts of every other (4 x 262,144 weights in clusters of 16: 23 us for the digits, with these 11).
template <int E>
__global__ void __launch_bounds__(kThreads, 1) evict_select_kernel(const EvictParams p) {
  __shared__ int hist[E > 1 ? kDigits : 1][E > 1 ? kBins : 1];
  __shared__ unsigned long long scan_sums[kWarps];
  __shared__ int warp_sums[kWarps], warp_over[kWarps];
  __shared__ int found[4];                 // the digit, how many of its keys are wanted; in the runs before: keys above, and of it
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, ranks = E > 1 ? cluster.num_blocks() : 1, rank = E > 1 ? cluster.block_rank() : 0;
  const int row = blockIdx.x / ranks, b = row / p.n_kv_heads;
  if constexpr (E > 1)
    for (int i = tid; i < kDigits * kBins; i += kThreads) hist[i / kBins][i % kBins] = 0;
  grid_dependency_wait();
  allow_dependent_launch();
  const Share s = share_of(p, b);
  if (s.bad && row % p.n_kv_heads == 0 && rank == 0 && tid == 0) flag_error(p.status, MEMRA_DEVERR_BAD_SEQ_LEN);
  const float *w = p.weights + static_cast<int64_t>(row) * p.weight_stride;
  const int middle = s.T - s.sink - s.recent, m = s.n - s.sink - s.recent;
  const int run = (middle + ranks - 1) / ranks, lo = s.sink + min(rank * run, middle),
            hi = s.sink + min((rank + 1) * run, middle);
  // A warp's keys lie behind one another, E * 32 of them.
  const int lane = tid & 31, warp = tid >> 5;
  auto index = [&](int i0, int e) { return i0 + (warp * E + e) * 32 + lane; };
  uint32_t key[E];
  // this thread's keys of a round
  auto mine = [&](int i0) { return (max(hi - index(i0, 0), 0) + 31) / 32; };
  auto load = [&](int i0) {
    const int n = mine(i0);
    const float *at = w + index(i0, 0);
    float x[E];
    if (n >= E) {                          // (without conditions, so that all are in flight together)
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = at[e * 32];
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = e < n ? at[e * 32] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) key[e] = key_of(x[e]);
  };
  // f(key) for this thread's keys
  auto each = [&](auto f) {
    for (int i0 = lo; i0 < hi; i0 += E * kThreads) {
      if (hi - lo > E * kThreads) load(i0);
      const int n = mine(i0);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e < n) f(key[e]);
    }
  };
  load(lo);
  __syncthreads();

  // every key above `last` is taken, and the first `ties` equal to it; and how many of either the runs before hold
  uint32_t last = 0;
  int ties = middle, over_before = lo - s.sink, equal_before = 0;
  if (m == 0) {
    last = 0xFFFFFFFFu, ties = 0;
  } else if (m < middle) {                 // (the same for the whole cluster)
    over_before = 0;
    if constexpr (E == 1) {
      last = nth_key_by_bits(key[0], lo + tid < hi, m, ties);
    } else {
      ties = m;
#pragma unroll
      for (int digit = 0; digit < kDigits; ++digit) {
        const int shift = 32 - kBits * (digit + 1);
        each([&](uint32_t k) {
          if (digit == 0 || (k ^ last) >> shift < kBins) atomicAdd(&hist[digit][(k >> shift) & (kBins - 1)], 1);
        });
        cluster.sync();
        // a bin of each of the first threads, from the highest down: of all runs, and of those before (low half)
        const int bin = kBins - 1 - tid;
        unsigned long long count = 0;
        if (bin >= 0) {
#pragma unroll
          for (int r = 0; r < kClusterMax; ++r) {
            if (r >= ranks) break;
            count += cluster.map_shared_rank(&hist[digit][0], r)[bin] * ((1ull << 32) + (r < rank));
          }
        }
        const unsigned long long above = block_scan(count, scan_sums) - count;
        const int over = static_cast<int>(above >> 32);
        if (ties > over && ties <= over + static_cast<int>(count >> 32)) {
          found[0] = bin;
          found[1] = ties - over;
          found[2] = static_cast<int>(above);
          found[3] = static_cast<int>(count);
        }
        __syncthreads();
        last |= static_cast<uint32_t>(found[0]) << shift;
        ties = found[1];
        over_before += found[2];
        equal_before = found[3];
      }
      if (ranks > 1) cluster.barrier_arrive();         // (waited for at the end: no CTA leaves while another reads its shared memory)
    }
  }

  int32_t *kept = p.kept + static_cast<int64_t>(row) * p.max_budget;
  if (rank == 0) {
    for (int i = tid; i < s.sink; i += kThreads) kept[i] = i;
    for (int i = tid; i < s.recent; i += kThreads) kept[s.n - s.recent + i] = s.T - s.recent + i;
    for (int i = s.n + tid; i < p.max_budget; i += kThreads) kept[i] = -1;
  }
  for (int i0 = lo; i0 < hi; i0 += E * kThreads) {
    if (hi - lo > E * kThreads) load(i0);
    // counts of the warp (above `last`; equal), of the warps before it, then of the keys before each
    const int n = mine(i0);
    int over = 0, equal = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      over += e < n && key[e] > last;
      equal += e < n && key[e] == last;
    }
    over = __reduce_add_sync(0xffffffffu, over);
    equal = __reduce_add_sync(0xffffffffu, equal);
    __syncthreads();                       // (the counts of the round before have been read)
    if (lane == 0) warp_over[warp] = over, warp_sums[warp] = equal;
    __syncthreads();
    const int o = warp_over[lane], q = warp_sums[lane];
    int overs = over_before + __reduce_add_sync(0xffffffffu, lane < warp ? o : 0);
    int equals = equal_before + __reduce_add_sync(0xffffffffu, lane < warp ? q : 0);
    over_before += __reduce_add_sync(0xffffffffu, o);
    equal_before += __reduce_add_sync(0xffffffffu, q);
    const unsigned below = (1u << lane) - 1u;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool above = e < n && key[e] > last, same = e < n && key[e] == last;
      if (!__any_sync(0xffffffffu, above || same)) continue;
      const unsigned ma = __ballot_sync(0xffffffffu, above), ms = __ballot_sync(0xffffffffu, same);
      const int before = equals + __popc(ms & below);
      if (above || (same && before < ties)) kept[s.sink + overs + __popc(ma & below) + min(before, ties)] = index(i0, e);
      overs += __popc(ma);
      equals += __popc(ms);
    }
  }
  if (E > 1 && ranks > 1 && m > 0 && m < middle) cluster.barrier_wait();
}

// The kept rows to their new pages, byte for byte, and their weights.  A thread makes one unit of the new
// segment, at most 16 bytes: a K unit of one token is a copy, the others hold bytes of
// two tokens (NVFP4 K) or of four (V), which it picks from the units that lie at the
// same place of their old pages, all loads in flight.  (A thread that moved single
// bytes of the page's 16 rows made seven times the loads: 81 us for 28,000 rows of 4 heads.)  Bytes
// bound it, those of other tokens too: a V unit is read from sectors that hold eight tokens' (65,536 rows
// that lie apart: 15 MB of them, 135 MB of sectors, 87 MB from memory in 19 us).  Where a row
// does not move, a unit is read from the new page and left unused: loads with conditions go one after the other.

__device__ __forceinline__ uint32_t word_of(const uint4 &x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }

// Where a token of a page lies among those that share units.
struct Spot {
  const uint8_t *seg;           // its old segment; null: its row does not move
  int t;
  __device__ __forceinline__ int c() const { return (t & 7) >> 1; }
  __device__ __forceinline__ int f() const { return t & 1; }
  __device__ __forceinline__ int p() const { return t >> 3; }
};

// Of four tokens' words: byte at[i] of each to byte i (tokens in the order of the bytes they have in the new word).
__device__ __forceinline__ uint32_t pick4(const uint32_t (&x)[4], const int (&at)[4]) {
  const uint32_t a = __byte_perm(x[0], x[1], at[0] | (4 + at[1]) << 4), b = __byte_perm(x[2], x[3], at[2] | (4 + at[3]) << 4);
  return __byte_perm(a, b, 0x5410);
}

// The new word keeps its old bytes where a token does not move.
__device__ __forceinline__ uint32_t merge_bytes(uint32_t fresh, uint32_t old, uint32_t mask) { return (fresh & mask) | (old & ~mask); }

template <int D, int KF>
struct KUnits {
  static constexpr int kCodes = KF == MEMRA_KV_NVFP4 ? 8 * D / 16 : 16 * D / 16;
  static constexpr int kScaleBytes = KF == MEMRA_KV_Q8_0 ? D / 16 : KF == MEMRA_KV_NVFP4 ? D / 16 : 0;      // of a token
  static constexpr int kAll = kCodes + (kScaleBytes ? kPage : 0);
  template <class SpotOf>
  static __device__ __forceinline__ void move(int u, uint8_t *to, SpotOf spot) {
    if (u >= kCodes) {                     // a token's block scales
      const int t = u - kCodes;
      const Spot s = spot(t);
      constexpr int at = KF == MEMRA_KV_NVFP4 ? 8 * D : 16 * D;
      if (!s.seg) return;
      if constexpr (kScaleBytes == 8)
        *reinterpret_cast<uint2 *>(to + at + 8 * t) = *reinterpret_cast<const uint2 *>(s.seg + at + 8 * s.t);
      else if constexpr (kScaleBytes == 16)
        *reinterpret_cast<uint4 *>(to + at + 16 * t) = *reinterpret_cast<const uint4 *>(s.seg + at + 16 * s.t);
    } else if constexpr (KF == MEMRA_KV_NVFP4) {
      // unit (word group, 4 tg + c): tokens tg and tg + 8, bytes tp + 2 e of each word
      const int w4 = u / 32, lane = u % 32, tg = lane >> 2;
      Spot s[2];
      uint4 x[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[i] = spot(tg + 8 * i);
        x[i] = *reinterpret_cast<const uint4 *>((s[i].seg ? s[i].seg : to) + (w4 * 32 + 4 * (s[i].t & 7) + (lane & 3)) * 16);
      }
      uint4 *dst = reinterpret_cast<uint4 *>(to + u * 16);
      const uint32_t mask = (s[0].seg ? 0x00FF00FFu : 0u) | (s[1].seg ? 0xFF00FF00u : 0u);
      if (!mask) return;
      const uint4 old = mask != 0xFFFFFFFFu ? *dst : make_uint4(0, 0, 0, 0);
      const int a = s[0].p(), c = 4 + s[1].p();
      const int sel = a | c << 4 | (a + 2) << 8 | (c + 2) << 12;
      *dst = make_uint4(merge_bytes(__byte_perm(x[0].x, x[1].x, sel), old.x, mask),
                        merge_bytes(__byte_perm(x[0].y, x[1].y, sel), old.y, mask),
                        merge_bytes(__byte_perm(x[0].z, x[1].z, sel), old.z, mask),
                        merge_bytes(__byte_perm(x[0].w, x[1].w, sel), old.w, mask));
    } else {
      // unit (token half, 64-dim block, 4 tg + kc): one token's
      constexpr int B2 = D / 64;
      const int lane = u % 32, b2 = u / 32 % B2, tp = u / (32 * B2);
      const Spot s = spot(8 * tp + (lane >> 2));
      if (s.seg)
        *reinterpret_cast<uint4 *>(to + u * 16) =
            *reinterpret_cast<const uint4 *>(s.seg + ((s.p() * B2 + b2) * 32 + 4 * (s.t & 7) + (lane & 3)) * 16);
    }
  }
};

template <int D, int VF>
struct VUnits {
  static constexpr int NB = D / 32;
  static constexpr int kCodes = (VF == MEMRA_KV_FP8_E4M3 ? 16 : 8) * D / 16;
  static constexpr int kFifths = VF == MEMRA_KV_Q5_1 ? 32 : 0;                   // a lane's words, 2 NB bytes
  static constexpr int kHalves = VF == MEMRA_KV_Q5_1 ? 2 * 4 * NB : VF == MEMRA_KV_Q4_0 ? 4 * NB : 0;   // 8 bytes of four tokens
  static constexpr int kBytes = VF == MEMRA_KV_NVFP4 ? D / 16 : 0;               // 16 bytes of scales: four blocks of one c
  static constexpr int kAll = kCodes + kFifths + kHalves + kBytes;
  // Token of a word's byte (q5_1, q4_0: byte 2 f + p; nvfp4: f + 2 p), and the byte of a token.
  static __device__ __forceinline__ int token(int c, int byte) {
    return VF == MEMRA_KV_NVFP4 ? 2 * c + (byte & 1) + 8 * (byte >> 1) : 2 * c + (byte >> 1) + 8 * (byte & 1);
  }
  static __device__ __forceinline__ int byte_of(const Spot &s) {
    return VF == MEMRA_KV_NVFP4 ? s.f() + 2 * s.p() : 2 * s.f() + s.p();
  }
  // N words at `at` (for the token's c: at + step * c), each with one byte of four tokens
  template <int N, class SpotOf>
  static __device__ __forceinline__ void words(uint8_t *to, int c, int at, int step, SpotOf spot) {
    Spot s[4];
    uint32_t x[4][N], mask = 0;
    int byte[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = spot(token(c, i));
      byte[i] = byte_of(s[i]);
      if (s[i].seg) mask |= 0xFFu << (8 * i);
      const uint8_t *src = (s[i].seg ? s[i].seg : to) + at + step * s[i].c();
      if constexpr (N == 4) {
        const uint4 y = *reinterpret_cast<const uint4 *>(src);
        x[i][0] = y.x, x[i][1] = y.y, x[i][2] = y.z, x[i][3] = y.w;
      } else {
        const uint2 y = *reinterpret_cast<const uint2 *>(src);
        x[i][0] = y.x, x[i][1] = y.y;
      }
    }
    if (!mask) return;
    uint32_t y[N];
    uint32_t *dst = reinterpret_cast<uint32_t *>(to + at + step * c);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t w[4] = {x[0][n], x[1][n], x[2][n], x[3][n]};
      y[n] = pick4(w, byte);
      if (mask != 0xFFFFFFFFu) y[n] = merge_bytes(y[n], dst[n], mask);
    }
    if constexpr (N == 4)
      *reinterpret_cast<uint4 *>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
    else
      *reinterpret_cast<uint2 *>(dst) = make_uint2(y[0], y[1]);
  }
  template <class SpotOf>
  static __device__ __forceinline__ void move(int u, uint8_t *to, SpotOf spot) {
    if (u < kCodes) {
      const int lane = u % 32, c = lane & 3, run = u / 32;
      const int at = (run * 32 + (lane & ~3)) * 16;
      if constexpr (VF == MEMRA_KV_FP8_E4M3) {
        // words 2 h + p hold the tokens f = 0, 1 in bytes f and f + 2
        uint32_t y[4] = {0, 0, 0, 0}, mask[2] = {0, 0};
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const Spot s = spot(2 * c + f + 8 * p);
            const uint4 x = *reinterpret_cast<const uint4 *>((s.seg ? s.seg : to) + at + 16 * s.c());
            if (s.seg) mask[p] |= 0x00FF00FFu << (8 * f);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t w = s.p() ? word_of(x, 2 * h + 1) : word_of(x, 2 * h);
              y[2 * h + p] |= (s.f() ? w >> 8 & 0x00FF00FFu : w & 0x00FF00FFu) << (8 * f);
            }
          }
        if (!(mask[0] | mask[1])) return;
        uint4 *dst = reinterpret_cast<uint4 *>(to + at + 16 * c);
        if ((mask[0] & mask[1]) != 0xFFFFFFFFu) {
          const uint4 old = *dst;
          y[0] = merge_bytes(y[0], old.x, mask[0]), y[1] = merge_bytes(y[1], old.y, mask[1]);
          y[2] = merge_bytes(y[2], old.z, mask[0]), y[3] = merge_bytes(y[3], old.w, mask[1]);
        }
        *dst = make_uint4(y[0], y[1], y[2], y[3]);
      } else {
        words<4>(to, c, at, 16, spot);
      }
    } else if (u < kCodes + kFifths) {
      const int lane = u - kCodes;
      words<NB / 2>(to, lane & 3, 8 * D + (lane & ~3) * 2 * NB, 2 * NB, spot);
    } else if (u < kCodes + kFifths + kHalves) {
      // scales, and D bytes on the minima of q5_1: block b of the tokens of one c, halves 2 p + f
      const int i = u - kCodes - kFifths, side = i / (4 * NB), c = i % (4 * NB) / NB, b = i % NB;
      const int at = (VF == MEMRA_KV_Q5_1 ? 10 : 8) * D + side * D + b * 8;
      Spot s[4];
      uint16_t x[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        s[h] = spot(2 * c + (h & 1) + 8 * (h >> 1));
        x[h] = *reinterpret_cast<const uint16_t *>((s[h].seg ? s[h].seg : to) + at + s[h].c() * NB * 8 +
                                                   2 * (2 * s[h].p() + s[h].f()));
      }
#pragma unroll
      for (int h = 0; h < 4; ++h)
        if (s[h].seg) *reinterpret_cast<uint16_t *>(to + at + c * NB * 8 + 2 * h) = x[h];
    } else {
      const int i = u - kCodes - kFifths - kHalves, c = i / (D / 64), b4 = i % (D / 64);
      words<4>(to, c, 8 * D + b4 * 16, D / 4, spot);
    }
  }
};

constexpr int kMovePages = 8;              // pages of a CTA at most (16 x 8,192 tokens: 24 us, with 2 28, with 1 36)

template <int D, int KF, int VF>
struct MoveCfg {
  static constexpr int kK = KUnits<D, KF>::kAll, kV = VUnits<D, VF>::kAll;
  // K's and V's units of a page by warps of their own
  static constexpr int kKThreads = (kK + 31) / 32 * 32, kThreads = kKThreads + (kV + 31) / 32 * 32;
  static_assert(kThreads <= 1024 && kThreads >= kMovePages * kPage, "a unit to a thread");
};

template <int D, int KF, int VF>
__global__ void __launch_bounds__(MoveCfg<D, KF, VF>::kThreads, 1536 / MoveCfg<D, KF, VF>::kThreads) evict_move_kernel(const EvictParams p, int pages) {
  using C = MoveCfg<D, KF, VF>;
  __shared__ int s_page[kMovePages][kPage], s_token[kMovePages][kPage], s_to[kMovePages];
  grid_dependency_wait();
  allow_dependent_launch();
  const int tid = threadIdx.x, page0 = blockIdx.x * pages, h = blockIdx.y % p.n_kv_heads, b = blockIdx.y / p.n_kv_heads;
  if (tid < pages * kPage) {
    // (the row's index is read beside the lengths; what lies behind the last is -1)
    const int j = page0 * kPage + tid;
    const int64_t row = blockIdx.y;
    const int i = j < p.max_budget ? p.kept[row * p.max_budget + j] : -1;
    const int to = j < p.max_budget ? p.dst_table[static_cast<int64_t>(b) * p.dst_pages + j / kPage] : -1;
    int from = -1;
    if (i >= 0) {
      if (p.new_weights) p.new_weights[row * p.new_stride + j] = p.weights[row * p.weight_stride + i];
      from = p.page_table[static_cast<int64_t>(b) * p.max_pages + i / kPage];
      if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages) {
        from = -1;
        flag_error(p.status, MEMRA_DEVERR_BAD_PAGE);
      }
    }
    // How many stay: stored here, because new_lens may be seq_lens or budgets, and every CTA of the selection reads those.
    if (p.new_lens && h == 0) {
      const int after = j + 1 < p.max_budget ? p.kept[row * p.max_budget + j + 1] : -1;
      if (i >= 0 ? after < 0 : j == 0) p.new_lens[b] = i >= 0 ? j + 1 : 0;
    }
    s_page[tid / kPage][tid % kPage] = from;
    s_token[tid / kPage][tid % kPage] = i & (kPage - 1);
    if (tid % kPage == 0) s_to[tid / kPage] = to >= 0 && to < p.num_pages && i >= 0 ? to : -1;
  }
  __syncthreads();
  const bool v = tid >= C::kKThreads;
  const int u = v ? tid - C::kKThreads : tid;
  if (u >= (v ? C::kV : C::kK)) return;
  uint8_t *const pool = (v ? p.v_pool : p.k_pool) + static_cast<size_t>(h) * (v ? v_seg_bytes(VF, D) : k_seg_bytes(KF, D));
  const size_t stride = static_cast<size_t>(p.n_kv_heads) * (v ? v_seg_bytes(VF, D) : k_seg_bytes(KF, D));
#pragma unroll 1
  for (int g = 0; g < pages; ++g) {
    if (s_to[g] < 0) continue;             // (a page's first row has none: nor have the others)
    auto spot = [&](int t) {
      const int from = s_page[g][t];
      return Spot{from >= 0 ? pool + from * stride : nullptr, s_token[g][t]};
    };
    uint8_t *to = pool + s_to[g] * stride;
    if (v) VUnits<D, VF>::move(u, to, spot); else KUnits<D, KF>::move(u, to, spot);
  }
}

template <int D, int KF, int VF>
cudaError_t launch_move(const EvictParams &p, int sms, cudaStream_t st) {
  // As many pages to a CTA as still leave six CTAs to each SM.
  const int64_t rows = static_cast<int64_t>(p.batch) * p.n_kv_heads, all = (p.max_budget + kPage - 1) / kPage;
  const int pages = static_cast<int>(std::min<int64_t>(std::max<int64_t>(all * rows / (6 * sms), 1), kMovePages));
  const dim3 grid(static_cast<unsigned>((all + pages - 1) / pages), static_cast<unsigned>(rows));
  return launch_pdl(evict_move_kernel<D, KF, VF>, grid, dim3(MoveCfg<D, KF, VF>::kThreads), 0, st, p, pages);
}

template <int D, int KF>
cudaError_t launch_move_v(const EvictParams &p, int sms, cudaStream_t st) {
  switch (p.v_fmt) {
    case MEMRA_KV_Q5_1: return launch_move<D, KF, MEMRA_KV_Q5_1>(p, sms, st);
    case MEMRA_KV_Q4_0: return launch_move<D, KF, MEMRA_KV_Q4_0>(p, sms, st);
    case MEMRA_KV_FP8_E4M3: return launch_move<D, KF, MEMRA_KV_FP8_E4M3>(p, sms, st);
    case MEMRA_KV_NVFP4: return launch_move<D, KF, MEMRA_KV_NVFP4>(p, sms, st);
    default: return cudaErrorInvalidValue;
  }
}

template <int D>
cudaError_t launch_move_k(const EvictParams &p, int sms, cudaStream_t st) {
  switch (p.k_fmt) {
    case MEMRA_KV_Q8_0: return launch_move_v<D, MEMRA_KV_Q8_0>(p, sms, st);
    case MEMRA_KV_FP8_E4M3: return launch_move_v<D, MEMRA_KV_FP8_E4M3>(p, sms, st);
    case MEMRA_KV_NVFP4: return launch_move_v<D, MEMRA_KV_NVFP4>(p, sms, st);
    default: return cudaErrorInvalidValue;
  }
}

template <int E>
cudaError_t launch_select(const EvictParams &p, int64_t rows, int ranks, cudaStream_t st) {
  if (ranks > 8) {
    static bool ready[64] = {};            // the larger cluster, allowed once per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
      e = cudaFuncSetAttribute(evict_select_kernel<E>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      ready[dev] = true;
    }
  }
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
  cfg.numAttrs = E > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<E>, p);
}

}  // namespace

cudaError_t launch_evict_select(const EvictParams &p, int sms, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(p.batch) * p.n_kv_heads;
  if (p.max_seq_len <= kThreads) return launch_select<1>(p, rows, 1, st);
  // CTAs for the weights of one row: 4,096 of them each, as long as there are SMs (16 x 8,192 weights of 4 heads 36 us so, 40
  // with 16,384 to a CTA; one of 262,144 50 us in clusters of 16, 91 of 8; one of 512, by digits too, 12 us, by bits 8)
  int ranks = 1;
  while (ranks < kClusterMax && 4096ll * ranks < p.max_seq_len && 2 * ranks * rows <= 2 * sms) ranks *= 2;
  if (rows * ranks > INT32_MAX) return cudaErrorInvalidValue;
  return p.max_seq_len <= 4ll * kThreads * ranks ? launch_select<4>(p, rows, ranks, st) : launch_select<16>(p, rows, ranks, st);
}

cudaError_t launch_evict_move(int D, const EvictParams &p, int sms, cudaStream_t st) {
  return D == 128 ? launch_move_k<128>(p, sms, st) : launch_move_k<256>(p, sms, st);
}

}  // namespace memra
