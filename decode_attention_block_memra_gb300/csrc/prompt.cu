// Prompt attention: causal attention of whole prompts, packed one behind the
// other, with grouped heads and an optional sliding window.
//
//   o[t, h] = sum_u p_u v[u, h / G] / sum_u p_u,  p_u = 2^(s_u - m),
//   s_u = q[t, h] . k[u, h / G] * scale * log2(e),  u = max(first, t - W + 1) .. t
//
// One pass over the keys with a running reference maximum m and sum.  The two
// products are dense contractions, so they run on the fifth-generation tensor
// cores with their accumulators in tensor memory, and the kernel is built so
// that they never wait for the softmax:
//   * A tile is 128 query rows of one KV head: 128 / G consecutive tokens times
//     the G heads of the group, so a short prompt of grouped heads still fills
//     the M = 128 side and a tile's rows share one diagonal.
//   * head_dim 128: a CTA holds two tiles (256 rows) and takes 128 keys a step.
//     The tiles share one score buffer, free again as soon as the softmax warps
//     hold the scores in registers, and P has columns of its own, so each softmax
//     has a whole step's MMAs (2,048 clocks) to finish in.
//   * head_dim 256: one tile, 64 keys a step, Q in tensor memory (an A operand
//     in shared memory would need more than its bandwidth at N = 64), two score
//     buffers that P overwrites; the scores run two steps ahead.
//   * Q, K and V arrive by TMA tensor copies in the 128-byte-swizzled layout
//     (K V ring of 32 KB stages); V is read by the MMA as it lies, keys along
//     rows (MN-major B), so nothing is transposed.
//   * P goes to tensor memory in fp16 and is the A operand of O += P V: no
//     shared-memory round trip.
// Warps: four softmax warps per tile (thread = row), one that issues the score
// MMAs, one that issues the products, one that loads.  The reference maximum
// moves only when a tile's maximum passes it by more than kLazy (log2 units), so
// O in tensor memory is rescaled rarely; P then stays <= 2^kLazy.  Scores, maxima,
// sums and O are float32; P is rounded to fp16 (relative 2^-11 a weight), the
// operand type of the tensor cores.
// The tensor cores cut an accumulator's last bits at every step (half of 2^-21 of
// it on average, always towards zero: a mean over 524,288 keys in one sum was off
// by 2.8e-3), so no more than kSumKeys keys go into one sum.  Then each element's
// fp16 part moves to the row's place in `out`, over a power of two that keeps it
// in range, and what is left of it, exact in float32, stays in O as the start of
// the next sum: no bit is lost and no scratch is needed.  On 16,384 tokens this takes
// 0.5 to 1% of the time (1,459 to 1,467 .. 1,474 us; as a branch inside the step loop,
// where its registers spill the loop's, 1,640).
// What bounds it: the tensor cores.  16,384 tokens, 32/4 heads, D 128: 1.47 ms a
// call in a loop (1,500 TFLOP/s, the power cap on), 1.28 ms for a single one, the
// tensor pipe active 78% of the time; 8 ragged prompts of up to 4,860 tokens 490 to
// 519 us (1,263 to 1,337 TFLOP/s, 67%); 9,713 tokens, 16/2 heads, D 256, window 1,024:
// 149 us (935 TFLOP/s, 44%, 17 steps a CTA); 256 tokens, 8/2 heads: 9.1 us, all latency.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "prompt.cuh"
#include "kv_stage.cuh"
#include "softmax_tile.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace memra {
namespace {

constexpr int kTileRows = 128;
constexpr float kLazy = 8.f;
constexpr int kSumKeys = 8192;             // most keys of one float32 sum in the tensor cores

template <int D>
struct PromptCfg {
  static constexpr int kTiles = D == 128 ? 2 : 1;       // query tiles of a CTA
  static constexpr int kKeys = D == 128 ? 128 : 64;     // keys of a step
  static constexpr bool kQSmem = D == 128;              // where Q lies
  static constexpr int kStages = D == 128 ? 5 : 7;
  static constexpr int kBlocks = D / 64;                // 64-element column blocks of a row
  static constexpr uint32_t kQBytes = kTileRows * D * 2;
  static constexpr uint32_t kKvBytes = kKeys * D * 2;
  static constexpr uint32_t kOffKv = kQSmem ? kTiles * kQBytes : 0;
  // head_dim 256: Q passes through the ring's last stages on its way to tensor memory
  static constexpr int kQStage = kStages - static_cast<int>(kQBytes / kKvBytes);
  static constexpr uint32_t kOffQ = kQSmem ? 0 : kOffKv + kQStage * kKvBytes;
  static constexpr uint32_t kOffBar = kOffKv + kStages * kKvBytes;
  // The barriers, 8 bytes each
  enum Bar { kKvFull = 0, kKvEmpty = kStages, kQFull = 2 * kStages, kSFull = kQFull + 2, kPFull = kSFull + 4,
             kPvDone = kPFull + 4, kVZeroed = kPvDone + 2, kSRead, kDrained, kSFree = kDrained + 2,
             kQLanded = kSFree + 2, kBars };
  static constexpr uint32_t kBarBytes = (8 * kBars + 15) / 16 * 16;
  static constexpr uint32_t kSmem = kOffBar + kBarBytes + 1024;    // 1024: aligning the base
  static constexpr int kThreads = 128 * kTiles + 96;
  // tensor-memory columns: D 128 scores 0, P 128 + 64 i, O 256 + 128 i; D 256 scores 64 b, Q 128, O 256
  static constexpr uint32_t kQCol = 128, kOCol = 256;
  static_assert(kSmem <= 232448, "shared memory");
};

// The sequence and the tile pair of this CTA, found from the packed lengths.
struct Work {
  int first, len;       // first row and rows of the sequence
  int t0;               // first token of the CTA's first tile, within the sequence
};

// A sequence's rows as the kernel uses them: within 0 .. total, not before they start.
__device__ __forceinline__ Work clamp_rows(const PromptParams &p, int b, bool report) {
  Work w{0, 0, -1};
  if (b < p.batch) {
    const int cs = p.cu_seqlens[b], ce = p.cu_seqlens[b + 1];
    w.first = min(max(cs, 0), p.total);
    w.len = min(max(ce, w.first), p.total) - w.first;
    if (report && (w.first != cs || w.first + w.len != ce)) flag_error(p.status, MEMRA_DEVERR_BAD_SEQ_LEN);
  }
  return w;
}

__device__ __forceinline__ Work broadcast(const Work &w, int src) {
  return Work{__shfl_sync(0xffffffffu, w.first, src), __shfl_sync(0xffffffffu, w.len, src),
              __shfl_sync(0xffffffffu, w.t0, src)};
}

// The `rank`-th piece of `tpc` tokens of the call, by a whole warp; t0 < 0: there
// is none.  Pieces are numbered sequence by sequence, a sequence's last (its
// longest) first.  (Ordering the pieces of all sequences by length instead gained
// nothing: 516 against 512 us on 8 ragged prompts of up to 4,860 tokens, 32/4
// heads, D 128.)  CTA 0 checks every length.
__device__ __forceinline__ Work find_work(const PromptParams &p, int rank, int tpc, int lane) {
  const bool report = blockIdx.x == 0;
  Work found{0, 0, -1};
  int start = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    Work w = clamp_rows(p, b0 + lane, report);
    const int pieces = (w.len + tpc - 1) / tpc;
    int incl = pieces;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += up;
    }
    const int nth = rank - start - (incl - pieces);
    if (nth >= 0 && nth < pieces) w.t0 = (pieces - 1 - nth) * tpc;
    const unsigned who = __ballot_sync(0xffffffffu, w.t0 >= 0);
    if (who) found = broadcast(w, __ffs(who) - 1);
    if (who && !report) break;
    start += __shfl_sync(0xffffffffu, incl, 31);
  }
  return found;
}

// Steps [lo, hi) of kKeys keys that a tile of tokens t .. t + tpt - 1 takes; empty when the tile is.
template <int D>
__device__ __forceinline__ void tile_steps(const PromptParams &p, const Work &w, int t, int &lo, int &hi) {
  constexpr int KT = PromptCfg<D>::kKeys;
  lo = hi = 0;
  if (t >= w.len) return;
  const int last = min(w.len, t + p.tpt) - 1;
  hi = last / KT + 1;
  if (p.window > 0) lo = max(0, t - p.window + 1) / KT;
}

template <int D>
__global__ void __launch_bounds__(PromptCfg<D>::kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const PromptParams p) {
  using C = PromptCfg<D>;
  constexpr int NT = C::kTiles, KT = C::kKeys, ST = C::kStages;
  constexpr int NBUF = NT == 2 ? 1 : 2;             // uses of a tile's barriers that alternate: the score buffers
  constexpr int kScoreWarp = 4 * NT, kOutWarp = kScoreWarp + 1, kLoadWarp = kScoreWarp + 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Work s_work;
  __shared__ uint32_t tmem_slot;
  const uint32_t sb = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bars = sb + C::kOffBar;
  auto kv_full = [&](int s) { return bars + 8 * (C::kKvFull + s); };
  auto kv_empty = [&](int s) { return bars + 8 * (C::kKvEmpty + s); };
  auto q_full = [&](int i) { return bars + 8 * (C::kQFull + i); };
  auto s_full = [&](int i, int b) { return bars + 8 * (C::kSFull + 2 * i + b); };
  auto p_full = [&](int i, int b) { return bars + 8 * (C::kPFull + 2 * i + b); };
  auto pv_done = [&](int i) { return bars + 8 * (C::kPvDone + i); };
  const uint32_t v_zeroed = bars + 8 * C::kVZeroed, s_read = bars + 8 * C::kSRead;
  auto drained = [&](int which) { return bars + 8 * (C::kDrained + which); };
  auto s_free = [&](int b) { return bars + 8 * (C::kSFree + b); };
  // Q in shared memory; where it goes on to tensor memory, q_full follows when it is there
  auto q_landed = [&](int i) { return C::kQSmem ? q_full(i) : bars + 8 * C::kQLanded; };
  // columns of tile i's scores and P (score buffer b)
  auto s_col_of = [&](int b) { return static_cast<uint32_t>(NT == 2 ? 0 : b * KT); };
  auto p_col_of = [&](int i, int b) { return static_cast<uint32_t>(NT == 2 ? 128 + 64 * i : b * KT); };

  grid_dependency_wait();
  allow_dependent_launch();

  const int kvh = blockIdx.x % p.n_kv_heads, rank = blockIdx.x / p.n_kv_heads;
  if (warp == 0) {
    const Work w = find_work(p, rank, NT * p.tpt, lane);
    if (lane == 0) s_work = w;
  }
  if (tid == 32) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full(i), C::kQSmem ? 1 : 4);
      mbar_init(pv_done(i), 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(s_full(i, b), 1);
        mbar_init(p_full(i, b), 4);
      }
    }
    mbar_init(v_zeroed, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(drained(b), 1);
      mbar_init(s_free(b), 1);
      if (!C::kQSmem && b == 0) mbar_init(q_landed(0), 1);
    }
    mbar_init(s_read, 4);
    fence_barrier_init();
  }
  __syncthreads();
  const Work w = s_work;
  if (w.t0 < 0) return;                             // fewer tiles than the grid's bound
  if (warp == kScoreWarp) {
    tc::tmem_alloc(smem_addr(&tmem_slot), 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;

  int lo[NT], hi[NT], jlo = 0, jhi = 0;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    tile_steps<D>(p, w, w.t0 + i * p.tpt, lo[i], hi[i]);
    jhi = max(jhi, hi[i]);
  }
  jlo = lo[0];                                      // the first tile's keys start first, and it is never empty
  const bool tail = jhi * KT > w.len;               // the last step's V holds rows behind the sequence
  bool ok = true;

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------------ loads --
    const int slots = 2 * (jhi - jlo);
    int issued = 0;
    const bool leader = tc::elect_one();
    if (leader) {
      auto load_q = [&](int i) {
        if (lo[i] == hi[i]) return;
        mbar_arrive_expect_tx(q_landed(i), static_cast<uint32_t>(p.group * p.tpt) * 128 * C::kBlocks);
#pragma unroll
        for (int c = 0; c < C::kBlocks; ++c)
          tma_load_3d(sb + C::kOffQ + i * C::kQBytes + c * kTileRows * 128, &qmap, 64 * c, kvh * p.group,
                      w.first + w.t0 + i * p.tpt, q_landed(i));
      };
      load_q(0);
      for (int n = 0; n < slots; ++n) {             // K and V of a step by turns
        const int s = n % ST;
        if (!C::kQSmem && n == C::kQStage) ok = mbar_wait_suspended(q_full(0), 0, p.status);   // Q has left the ring
        if (ok && n >= ST) ok = mbar_wait_suspended(kv_empty(s), (n / ST - 1) & 1, p.status);
        if (!ok) break;
        mbar_arrive_expect_tx(kv_full(s), C::kKvBytes + (n == 0 && blockIdx.x == 0 ? p.test_extra_tx : 0));
#pragma unroll
        for (int c = 0; c < C::kBlocks; ++c)
          tma_load_3d(sb + C::kOffKv + s * C::kKvBytes + c * KT * 128, n & 1 ? &vmap : &kmap, 64 * c, kvh,
                      w.first + (jlo + n / 2) * KT, kv_full(s));
        issued = n + 1;
        if (NT > 1 && n == 0) load_q(NT - 1);
      }
    }
    __syncwarp();
    ok = __all_sync(0xffffffffu, ok);
    if (ok && tail) {
      // rows behind the sequence may hold anything, and 0 * inf is not 0: they become zeros
      const int n = slots - 1, s = n % ST;
      ok = mbar_wait_suspended(kv_full(s), (n / ST) & 1, p.status);
      const int from = w.len - (jhi - 1) * KT;
      const uint32_t v = sb + C::kOffKv + s * C::kKvBytes;
      for (int i = lane; ok && i < (KT - from) * 8 * C::kBlocks; i += 32) {
        const int u = i & 7, c = (i >> 3) % C::kBlocks, row = from + (i >> 3) / C::kBlocks;
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v + c * KT * 128 + row * 128 + 16 * u), "r"(0)
                     : "memory");
      }
      fence_proxy_async();
      __syncwarp();
      if (leader && ok) mbar_arrive(v_zeroed);
    }
    // every copy has landed before the CTA can leave
    if (leader)
      for (int n = max(0, issued - ST); n < issued; ++n) mbar_wait_suspended(kv_full(n % ST), (n / ST) & 1, p.status);
  } else if (warp == kScoreWarp) {
    // ----------------------------------------------------------------- scores --
    // S_i(j) = Q_i K(j)^T, step by step, the tiles in turn
    if (tc::elect_one()) {
      constexpr uint32_t idesc_s = tc::idesc_f16_f32(kTileRows, KT);
      int issued = 0;
      for (int j = jlo; j < jhi && ok; ++j) {
        const int n = 2 * (j - jlo), stage = n % ST;
        ok = mbar_wait_suspended(kv_full(stage), (n / ST) & 1, p.status);
        const uint64_t kd = tc::smem_desc_sw128(sb + C::kOffKv + stage * C::kKvBytes, 16, 1024);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          if (!ok || j < lo[i] || j >= hi[i]) continue;
          const int u = j - lo[i], b = NBUF > 1 ? u & 1 : 0;
          if (u == 0) ok = mbar_wait_suspended(q_full(i), 0, p.status);
          if (NT == 2) {                            // one buffer: the scores before these are in registers
            if (ok && issued > 0) ok = mbar_wait_suspended(s_read, (issued - 1) & 1, p.status);
          } else {                                  // two: the product that read this one's P is done
            if (ok && u >= 2) ok = mbar_wait_suspended(s_free(b), ((u >> 1) - 1) & 1, p.status);
          }
          if (!ok) continue;
          ++issued;
          tc::fence_after_sync();
          const uint32_t d = tmem + s_col_of(b);
          const uint64_t qd = tc::smem_desc_sw128(sb + i * C::kQBytes, 16, 1024);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t bd = tc::desc_at(kd, (ks / 4) * KT * 128 + (ks % 4) * 32);
            if constexpr (C::kQSmem)
              tc::mma_f16(d, tc::desc_at(qd, (ks / 4) * kTileRows * 128 + (ks % 4) * 32), bd, idesc_s, ks > 0);
            else
              tc::mma_f16_ta(d, tmem + C::kQCol + 8 * ks, bd, idesc_s, ks > 0);
          }
          tc::commit(s_full(i, b));
        }
        if (ok) tc::commit(kv_empty(stage));
      }
      tc::commit(drained(0));                       // what was issued has completed before the CTA can leave
      mbar_wait_suspended(drained(0), 0, p.status);
    }
    __syncwarp();
  } else if (warp == kOutWarp) {
    // --------------------------------------------------------------- products --
    // O_i += P_i(j) V(j), from a thread of its own: neither kind of MMA waits for the other's operands
    if (tc::elect_one()) {
      constexpr uint32_t idesc_o = tc::idesc_f16_f32_bmn(kTileRows, D);
      for (int j = jlo; j < jhi && ok; ++j) {
        const int n = 2 * (j - jlo) + 1, stage = n % ST;
        ok = mbar_wait_suspended(kv_full(stage), (n / ST) & 1, p.status);
        if (ok && tail && j == jhi - 1) ok = mbar_wait_suspended(v_zeroed, 0, p.status);
        const uint64_t vd = tc::smem_desc_sw128(sb + C::kOffKv + stage * C::kKvBytes, KT * 128, 1024);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          if (!ok || j < lo[i] || j >= hi[i]) continue;
          const int u = j - lo[i], b = NBUF > 1 ? u & 1 : 0;
          ok = mbar_wait_suspended(p_full(i, b), (u / NBUF) & 1, p.status);
          if (!ok) continue;
          tc::fence_after_sync();
#pragma unroll
          for (int ks = 0; ks < KT / 16; ++ks)
            tc::mma_f16_ta(tmem + C::kOCol + i * D, tmem + p_col_of(i, b) + 8 * ks, tc::desc_at(vd, ks * 2048), idesc_o,
                           u > 0 || ks > 0);
          if (NT == 1) tc::commit(s_free(b));
          tc::commit(pv_done(i));
        }
        if (ok) tc::commit(kv_empty(stage));
      }
      tc::commit(drained(1));
      mbar_wait_suspended(drained(1), 0, p.status);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax --
    const int i = NT == 1 ? 0 : warp >> 2;
    const int rl = tid & 127;
    const uint32_t tlane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int tl = rl / p.group, t = w.t0 + i * p.tpt + tl;       // the row's token within the sequence
    const bool live = tl < p.tpt && t < w.len;
    const int tile_first = w.t0 + i * p.tpt, tile_last = min(w.len, tile_first + p.tpt) - 1;
    const int n_steps = hi[i] - lo[i];
    float m = -INFINITY;
    uint64_t l = 0;                                 // two sums, of the even and the odd keys
    // What earlier sums left in the row of `out`: fp16 parts, times `far`; and their weights' sum
    constexpr int kSumSteps = kSumKeys / KT;
    float far = 0.f, l_far = 0.f;
    const uint32_t o_col = tmem + tlane + C::kOCol + i * D;
    auto row_at = [&] { return (static_cast<int64_t>(w.first + t) * p.n_heads + kvh * p.group + rl % p.group) * D; };
    // O plus what the row of `out` holds (`held`): the whole to O, or its fp16 part, over `up`, to the row and
    // the rest to O.  (An infinity stays in O: what goes to the row is cut to fp16's range.)
    auto join = [&](bool held, bool split, float up) {
      const uint64_t far2 = pack_f2(far, far), down2 = pack_f2(1.f / up, 1.f / up), minus_up2 = pack_f2(-up, -up);
      uint4 *const row = reinterpret_cast<uint4 *>(p.out + (live ? row_at() : 0));
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 128) {
        uint4 x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = held && live ? row[c0 / 8 + e] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          uint32_t o[32];
          tc::ld_32x32b_x32(o_col + c0 + c, o);
          tc::wait_ld_all();
          tc::hold<32>(o);
          uint32_t *y = &x[c / 8].x;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 old = __half22float2(bits_h2(y[e]));
            uint64_t s = fma_f2(pack_f2(old.x, old.y), far2,
                                pack_f2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])));
            if (split) {
              float s0, s1;
              unpack_f2(mul_f2(s, down2), s0, s1);
              y[e] = pack_half2_sat(s0, s1);
              const float2 hi = __half22float2(bits_h2(y[e]));
              s = fma_f2(pack_f2(hi.x, hi.y), minus_up2, s);
            }
            float s0, s1;
            unpack_f2(s, s0, s1);
            o[2 * e] = __float_as_uint(s0), o[2 * e + 1] = __float_as_uint(s1);
          }
          tc::st_32x32b_x32(o_col + c0 + c, o);
        }
        if (split && live)
#pragma unroll
          for (int e = 0; e < 16; ++e) row[c0 / 8 + e] = x[e];
        __syncwarp();
      }
      tc::wait_st();
    };
    if constexpr (!C::kQSmem) {
      // the row of Q, fp16 pairs as they lie (row by row from memory this took 7,000 clocks)
      ok = mbar_wait_suspended(q_landed(0), 0, p.status);
      ok = __all_sync(0xffffffffu, ok);
#pragma unroll
      for (int c = 0; c < D / 2; c += 32) {
        uint32_t x[32];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint4 y = lds128(sb + C::kOffQ + c / 32 * kTileRows * 128 + rl * 128 + ((e ^ (rl & 7)) * 16));
          x[4 * e] = y.x, x[4 * e + 1] = y.y, x[4 * e + 2] = y.z, x[4 * e + 3] = y.w;
        }
        tc::st_32x32b_x32(tmem + tlane + C::kQCol + c, x);
      }
      tc::wait_st();
      tc::fence_before_sync();
      fence_proxy_async();                          // the ring's stages are the copies' again
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(q_full(i));
    }
    int end = 0;                                    // the first step of the next sum
#pragma unroll 1
    for (int first = 0; first < n_steps && ok; first = end) {
      end = min(n_steps, first + kSumSteps);
#pragma unroll 1
      for (int u = first; u < end && ok; ++u) {
        const int j = lo[i] + u, b = NBUF > 1 ? u & 1 : 0;
        const uint32_t s_col = tmem + tlane + s_col_of(b), p_col = tmem + tlane + p_col_of(i, b);
        ok = mbar_wait_suspended(s_full(i, b), (u / NBUF) & 1, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc::fence_after_sync();
        uint32_t s[KT];
#pragma unroll
        for (int c = 0; c < KT; c += 32) tc::ld_32x32b_x32(s_col + c, s + c);
        tc::wait_ld_all();
        tc::hold<KT>(s);
        if (NT == 2) {                                // the score buffer is the other tile's turn
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_read);
        }
        const int last = t - j * KT;                  // the row's own key, in this step's columns
        if (j * KT + KT - 1 > tile_first) {           // keys behind the row's token
#pragma unroll
          for (int c = 0; c < KT; ++c)
            if (c > last) s[c] = 0xff800000u;         // -inf
        }
        if (p.window > 0 && j * KT < tile_last - p.window + 1) {    // keys before its window
#pragma unroll
          for (int c = 0; c < KT; ++c)
            if (c < last - p.window + 1) s[c] = 0xff800000u;
        }
        const float top = row_max(s) * p.scale_log2;
        float alpha = 1.f;
        if (live && top > m + kLazy) {                // also the first step with a key (m = -inf)
          if (m != -INFINITY) alpha = fast_exp2(m - top);
          m = top;
        }
        const bool moved = u > 0 && __any_sync(0xffffffffu, alpha != 1.f);
        if (u > 0 && (NT == 2 || moved || u == end - 1)) {
          // The product before has completed: it has read P's columns (their own, head_dim 128), and O is
          // still.  At the last step in any case: the wait behind the loop names the last product by its
          // parity, which the product two before has too.
          ok = mbar_wait_suspended(pv_done(i), (u - 1) & 1, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc::fence_after_sync();
        }
        if (moved) {                                  // O's rows of this warp times alpha
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tc::ld_32x32b_x32(o_col + c, o);
            tc::wait_ld_all();
            tc::hold<32>(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc::st_32x32b_x32(o_col + c, o);
          }
          l = fma_f2(l, pack_f2(alpha, alpha), 0);
          far *= alpha, l_far *= alpha;
        }
        const float mu = m == -INFINITY ? 0.f : m;
        uint64_t sum = 0;                             // (a step's own, so that no long sum takes single weights)
#pragma unroll
        for (int c = 0; c < KT; c += 32) {
          uint32_t w2[16];
          row_weights<16>(s + c, p.scale_log2, mu, w2, sum);
          tc::st_32x32b_x16(p_col + c / 2, w2);
        }
        l = add_f2(l, sum);
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(i, b));
      }
      if (ok) ok = mbar_wait_suspended(pv_done(i), (end - 1) & 1, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (ok && end < n_steps) {
        tc::fence_after_sync();
        float l0, l1;
        unpack_f2(l, l0, l1);
        l_far += l0 + l1;
        l = 0;
        // |O| <= the largest |V| times the weights' sum: a power of two above that brings O into fp16's range
        const float up = l_far < 1e30f ? __uint_as_float(((__float_as_uint(l_far) >> 23) + 2u) << 23) : 1.f;
        join(first > 0, true, up);
        far = up;
      }
    }
    if (__all_sync(0xffffffffu, n_steps > 0 && ok)) {
      tc::fence_after_sync();
      float l0, l1;
      unpack_f2(l, l0, l1);
      l0 += l1 + l_far;
      const float inv = l0 > 0.f ? 1.f / l0 : 0.f;
      if (n_steps > kSumSteps) join(true, false, 1.f);
      // The row into shared memory (the tile's Q, or at head_dim 256 the ring: both read for the last
      // time), 16-byte units XORed with the row so that eight rows' stores fall on different banks ...
      constexpr uint32_t kRow = D * 2;
      const uint32_t rows = sb + (C::kQSmem ? i * C::kQBytes : C::kOffKv) + (warp & 3) * 32 * kRow;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tc::ld_32x32b_x32(o_col + c, o);
        tc::wait_ld_all();
        tc::hold<32>(o);
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint32_t x[4];
#pragma unroll
          for (int h = 0; h < 4; ++h)
            x[h] = pack_half2(__uint_as_float(o[e + 2 * h]) * inv, __uint_as_float(o[e + 2 * h + 1]) * inv);
          sts128(rows + lane * kRow + ((((c + e) / 8) ^ (lane & 7)) * 16), make_uint4(x[0], x[1], x[2], x[3]));
        }
      }
      // ... and from there to memory, the heads of a token side by side.
      const int64_t to = live ? row_at() : -1;
      __syncwarp();
      constexpr int U = D / 8, PER = 32 / U;        // 16-byte units of a row, rows at a time
#pragma unroll 8
      for (int e = 0; e < 32; e += PER) {
        const int row = e + lane / U, u = lane % U;
        const uint4 x = lds128(rows + row * kRow + (u ^ (row & 7)) * 16);
        const int64_t at = __shfl_sync(0xffffffffu, to, row);
        if (at >= 0) *reinterpret_cast<uint4 *>(p.out + at + 8 * u) = x;
      }
    } else if (n_steps > 0 && live) {               // a wait gave up: NaN, and no part of a sum
      uint4 *row = reinterpret_cast<uint4 *>(p.out + row_at());
#pragma unroll 1
      for (int u = 0; u < D / 8; ++u) row[u] = make_uint4(kNanPair, kNanPair, kNanPair, kNanPair);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kScoreWarp) tc::tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch_one(const PromptParams &p, cudaStream_t st) {
  using C = PromptCfg<D>;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  CUtensorMap qm, km, vm;
  if (!encode_rows(&qm, p.q, D, p.n_heads, p.total, p.q_stride, p.group, p.tpt) ||
      !encode_rows(&km, p.k, D, p.n_kv_heads, p.total, p.k_stride, 1, C::kKeys) ||
      !encode_rows(&vm, p.v, D, p.n_kv_heads, p.total, p.v_stride, 1, C::kKeys))
    return cudaErrorInvalidValue;
  // at most this many CTAs' worth of tokens, whatever the lengths: one partial each sequence
  const int64_t tiles = static_cast<int64_t>(p.total) / (C::kTiles * p.tpt) + p.batch;
  const int64_t grid = tiles * p.n_kv_heads;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(prompt_kernel<D>, dim3(static_cast<unsigned>(grid)), dim3(C::kThreads), C::kSmem, st, qm, km, vm,
                    p);
}

}  // namespace

cudaError_t launch_prompt(int D, const PromptParams &p, cudaStream_t st) {
  return D == 128 ? launch_one<128>(p, st) : launch_one<256>(p, st);
}

}  // namespace memra
