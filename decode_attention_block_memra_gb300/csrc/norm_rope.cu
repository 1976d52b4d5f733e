// Query and key rows made ready for attention in one pass: each head's row is
// normalized, its first dims are turned by the token's position, and the keys
// (with the values) are stored in the paged cache where the call has one.
//
//   y = x / sqrt(mean(x^2) + eps) * w
//   (a, b) -> (a cos - b sin, b cos + a sin),  angle = position * inv_freq[j],
//   (a, b) = (y_j, y_{j + R/2})  or, interleaved,  (y_{2j}, y_{2j+1})
//
// Everything is float32 until the one rounding to fp16; the stored bytes are those
// that kv_append makes of the rounded row.
//
// Angles.  position * inv_freq reaches 10^5 and more radians, where float32 has no
// digits left behind the point.  So a frequency is kept in turns (inv_freq / 2 pi)
// as a 64-bit binary fraction, rounded once, and the position multiplies it modulo
// 2^64: whole turns fall away exactly, and the angle of position 2^20 is off by
// less than 2^-27 turns.  Its sine and cosine are taken once a token, not once a head: the
// CTA's threads put them into shared memory for all rows of their tokens.
//
// A row is D / 8 lanes of 8 consecutive dims (one 16-byte load); a warp takes 32 / (D / 8)
// heads of one token at a time, of one kind (K, V or Q), so that it never diverges
// in the quantizer, and has the next rows' loads in flight meanwhile.
#include <algorithm>

#include "kv_stage.cuh"
#include "norm_rope.cuh"

namespace memra {
namespace {

constexpr int kWarps = 8;
constexpr int kTileMax = 8;                // tokens of a CTA at most

template <int D>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_kernel(const NormRopeParams p) {
  constexpr int L = D / 8, ROWS = 32 / L;  // lanes of a row, rows of a warp
  __shared__ unsigned long long s_turns[D / 2];
  __shared__ __align__(16) float s_cos[kTileMax][D / 2], s_sin[kTileMax][D / 2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, l = lane % L, sub = lane / L;
  const int t0 = blockIdx.x * p.tile, tokens = min(p.tile, p.tokens - t0);
  const int first = blockIdx.y * p.passes, count = min(p.passes, p.k_passes + p.v_passes + p.q_passes - first);
  grid_dependency_wait();
  allow_dependent_launch();

  // Row group `at` of this CTA: its token, kind and head.
  enum { kK, kV, kQ };
  struct Rows {
    int token, kind, head;
    bool live;
    uint4 x;
    int slot;
  };
  auto fetch = [&](int at) {
    Rows r{t0, kK, 0, false, make_uint4(0, 0, 0, 0), -1};
    if (at >= tokens * count) return r;
    int pass = first + at % count;
    r.token = t0 + at / count;
    const __half *src = p.k;
    int64_t stride = p.k_stride;
    int heads = p.n_kv_heads;
    if (pass >= p.k_passes + p.v_passes) {
      pass -= p.k_passes + p.v_passes;
      r.kind = kQ, src = p.q, stride = p.q_stride, heads = p.n_heads;
    } else if (pass >= p.k_passes) {
      pass -= p.k_passes;
      r.kind = kV, src = p.v, stride = p.v_stride;
    }
    r.head = pass * ROWS + sub;
    r.live = r.head < heads;
    if (r.live) r.x = *reinterpret_cast<const uint4 *>(src + r.token * stride + static_cast<int64_t>(r.head) * D + 8 * l);
    if (r.kind != kQ && p.slots) r.slot = p.slots[r.token];
    return r;
  };
  Rows next = fetch(warp);

  if (p.half) {
    for (int j = tid; j < p.half; j += 32 * kWarps) {
      const double turns = static_cast<double>(p.inv_freq[j]) * 0.15915494309189533577;      // 1 / (2 pi)
      s_turns[j] = __double2ull_rz((turns - floor(turns)) * 18446744073709551616.0);
    }
    __syncthreads();
    for (int i = tid; i < tokens * p.half; i += 32 * kWarps) {
      const int t = i / p.half, j = i % p.half;
      const unsigned long long turn =
          s_turns[j] * static_cast<unsigned long long>(static_cast<long long>(p.positions[t0 + t]));
      // The nearest quarter turn and what is left of the angle, an eighth of a turn at most: as a float that is
      // off by less than 2^-28 turns.
      const unsigned quarter = static_cast<unsigned>((turn + (1ull << 61)) >> 62);
      const long long rest = static_cast<long long>(turn << 2) >> 2;     // (modulo a quarter)
      float s, c;
      sincospif(__ll2float_rn(rest) * 1.084202172485504434e-19f, &s, &c);        // 2^-63: in units of pi
      s_sin[t][j] = quarter & 1 ? (quarter & 2 ? -c : c) : (quarter & 2 ? -s : s);
      s_cos[t][j] = quarter & 1 ? (quarter & 2 ? s : -s) : (quarter & 2 ? -c : c);
    }
    __syncthreads();
  }

  float qw[8], kw[8];                      // the norm's weights of this lane's dims
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    qw[i] = p.q_weight ? p.q_weight[8 * l + i] : 1.f;
    kw[i] = p.k_weight && p.k ? p.k_weight[8 * l + i] : 1.f;
  }
  // Dims of this lane in the rotation: pair j + i (half-split), or the lane's own four pairs.
  const bool turned = 8 * l < 2 * p.half, second = 8 * l >= p.half;
  const int j0 = p.interleaved ? 4 * l : second ? 8 * l - p.half : 8 * l;
  const int partner = turned && !p.interleaved ? (second ? l - p.half / 8 : l + p.half / 8) : l;

#pragma unroll 1
  for (int at = warp; at < tokens * count; at += kWarps) {
    const Rows r = next;
    next = fetch(at + kWarps);
    uint4 y = r.x;
    if (r.kind != kV) {
      float x[8];
      const uint32_t in[4] = {r.x.x, r.x.y, r.x.z, r.x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(bits_h2(in[i]));
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
      }
      if (r.kind == kQ ? p.q_weight != nullptr : p.k_weight != nullptr) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
        for (int d = 1; d < L; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const float scale = 1.f / sqrtf(fmaf(sum, 1.f / D, p.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= scale * (r.kind == kQ ? qw[i] : kw[i]);
      }
      if (p.half) {
        const float *cs = s_cos[r.token - t0] + j0, *sn = s_sin[r.token - t0] + j0;
        if (p.interleaved) {
          if (turned) {
            const float4 c = *reinterpret_cast<const float4 *>(cs), s = *reinterpret_cast<const float4 *>(sn);
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = x[2 * i], b = x[2 * i + 1];
              x[2 * i] = fmaf(a, cc[i], -b * ss[i]);
              x[2 * i + 1] = fmaf(b, cc[i], a * ss[i]);
            }
          }
        } else {
          float other[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) other[i] = __shfl_sync(0xffffffffu, x[i], partner, L);
          if (turned) {
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
              const float4 c = *reinterpret_cast<const float4 *>(cs + i), s = *reinterpret_cast<const float4 *>(sn + i);
              const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                x[i + e] = fmaf(x[i + e], cc[e], second ? other[i + e] * ss[e] : -other[i + e] * ss[e]);
            }
          }
        }
      }
      y = make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
      if (r.live && r.kind == kQ)
        *reinterpret_cast<uint4 *>(p.q_out + r.token * p.q_out_stride + static_cast<int64_t>(r.head) * D + 8 * l) = y;
      if (r.live && r.kind == kK && p.k_out)
        *reinterpret_cast<uint4 *>(p.k_out + r.token * p.k_out_stride + static_cast<int64_t>(r.head) * D + 8 * l) = y;
    }
    if (r.kind != kQ && p.slots) {
      int slot = r.slot;
      if (slot >= 0 && slot / kPage >= p.num_pages) {
        if (r.kind == kK && lane == 0) flag_error(p.status, MEMRA_DEVERR_BAD_SLOT);
        slot = -1;
      }
      const bool act = r.live && slot >= 0;
      quantize_store_row<D>(p.cache, act, act ? slot / kPage : 0, act ? slot % kPage : 0, act ? r.head : 0, l, y, y,
                            r.kind == kK, r.kind == kV);
    }
  }
}

template <int D>
cudaError_t launch(NormRopeParams p, int sms, cudaStream_t st) {
  constexpr int kRows = 32 / (D / 8);
  auto groups = [](int heads) { return (heads + kRows - 1) / kRows; };
  p.k_passes = p.k ? groups(p.n_kv_heads) : 0;
  p.v_passes = p.slots ? groups(p.n_kv_heads) : 0;
  p.q_passes = groups(p.n_heads);
  const int all = p.k_passes + p.v_passes + p.q_passes;
  // As many tokens to a CTA as still leave four CTAs to each SM; with few tokens, the row groups of one are
  // spread over CTAs too, one to each warp.
  p.tile = static_cast<int>(std::min<int64_t>(std::max<int64_t>(p.tokens / (4ll * sms), 1), kTileMax));
  p.passes = p.tokens >= 4 * sms ? all : kWarps;
  const dim3 grid((p.tokens + p.tile - 1) / p.tile, (all + p.passes - 1) / p.passes);
  if (grid.y > 65535) return cudaErrorInvalidValue;
  return launch_pdl(norm_rope_kernel<D>, grid, dim3(32 * kWarps), 0, st, p);
}

}  // namespace

cudaError_t launch_norm_rope(int D, NormRopeParams p, int sms, cudaStream_t st) {
  return D == 128 ? launch<128>(p, sms, st) : launch<256>(p, sms, st);
}

}  // namespace memra
