// qk_norm_rope.cu -- RMSNorm of each query and key head, rotary positions, and
// the new rows of the KV cache, held in fp16 or in 4 bits.
//
// Source: DAMASCUS project overview, "[04] one decode step" (RoPE between the
// QKV projections and the attention over the KV cache); the norms of the heads
// and the 4-bit cache are this library's.
//
// A head's row of D values x becomes, where its gamma is given,
//   x / sqrt(mean x^2 + eps) * gamma,
// its first n_rot dimensions turn as in qk_rope.cu, and q (fp16) and the cache
// rows are written.  A 4-bit row holds groups of 32 values as v = d q + m:
//   m = fp16(min x),  d = fp16(max(max x - m, 0) / 15),
//   q = (x - m) / d rounded to the nearest of 0 .. 15 (0 where d = 0),
// d one step lower where 15 d + m would not be a finite fp16 number.
//
// A CTA has a few tokens and computes their sines and cosines together, while its
// first rows are on their way; a row is a head of a token, 8 dimensions a lane, and two
// rows load while one is computed.  The sum of squares and a group's extremes
// meet by shuffles.  Where a whole head of the half layout turns, a lane has two runs of
// four dimensions, each other's mates; otherwise a run of eight, and the half layout's
// mates, which other lanes hold, pass through shared memory (2047 tokens of 32 + 4 + 4
// heads of 128 in the half layout: 15.3 us with mates in a lane, a third more through shared
// memory; the interleaved layout 16.3).  A value's level comes from a reciprocal, and from
// a division where that is near a border between two levels: a division for each took
// twice as long.
//
// Every input is read once: 4095 tokens of 24 + 8 + 8 heads of 128 into 4 bits move 115
// MB (17 us at a copy's rate) in 28.9 us, bound by instructions (159 for a row and warp,
// issue slots 77 % busy; 178 with clamps and looks for borders value by value, 3 us more);
// into fp16 126 MB in 25.8 us.  Four CTAs an SM: three took 18.7 us where four
// took 15.9 (2047 tokens into fp16).  One token 2.1 us, latency.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "qk_device.cuh"
#include "qk_internal.h"
#include "qk_packed.cuh"
#include "qk_rope.cuh"

namespace qk {

namespace {

constexpr int kNrThreads = 256;
constexpr int kNrMaxD = 512;
constexpr int kNrTokens = 4;  // of a CTA at most

__device__ __forceinline__ uint32_t pack2h(float a, float b) {
  const __half2 x = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}

// max(a, b), NaN where one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// kN of the 32 values of a group, which 32 / kN lanes hold: their nibbles in order,
// and (d, m) as two fp16.  Every lane of the warp takes part.
template <int kN>
__device__ __forceinline__ uint32_t quantize(const float* y, uint32_t& dm) {
  float lo = y[0], hi = y[0];
#pragma unroll
  for (int e = 1; e < kN; ++e) {
    lo = fminf(lo, y[e]);
    hi = max_nan(hi, y[e]);
  }
#pragma unroll
  for (int o = 1; o < 32 / kN; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float m = __half2float(__float2half_rn(lo));
  __half dh = __float2half_rn(max_nan(hi - m, 0.f) / 15.f);
  // a value that is not finite or rounds to an infinite fp16 number, or a 15 d that does,
  // makes the group NaN (hi is NaN where a value is)
  const bool fine = lo > -65520.f && hi < 65520.f && __half2float(dh) <= 4366.f;
  // where d was rounded up so far that level 15 would be infinite as fp16, the number below d:
  // that is less than (hi - m) / 15, and level 15 less than hi
  if (fmaf(15.f, __half2float(dh), m) >= 65520.f) dh = __ushort_as_half((unsigned short)(__half_as_ushort(dh) - 1u));
  const float d = __half2float(dh);
  uint32_t q = 0;
  if (d > 0.f) {
    // (y - m) / (15 d) by the reciprocal, clamped to 0 .. 1, is within 2^-21 of the
    // quotient, and 15 times it within 2^-17 of the level; where one is nearer to a
    // border than that, the lane divides.  The levels add up in q with the bits of
    // kMagic, which come off in the end.
    constexpr float kMagic = 12582912.f;  // 1.5 2^23: adding it rounds to an integer in the low bits
    constexpr uint32_t kBits = 0x4B400000u, kSum = kN == 4 ? kBits * 0x1111u : kBits * 0x11111111u;
    const float r = __fdividef(1.0f / 15.0f, d);
    float n[kN], far = 0.f;
#pragma unroll
    for (int e = kN - 1; e >= 0; --e) {
      n[e] = y[e] - m;
      const float t = __saturatef(n[e] * r), k = fmaf(t, 15.f, kMagic);
      far = fmaxf(far, fabsf(fmaf(t, 15.f, -__fsub_rn(k, kMagic))));
      q = (q << 4) + __float_as_uint(k);
    }
    q -= kSum;
    if (far > 0.4999f) {
      q = 0;
#pragma unroll
      for (int e = kN - 1; e >= 0; --e)
        q = (q << 4) + __float_as_uint(__fadd_rn(fminf(fmaxf(n[e] / d, 0.f), 15.f), kMagic)) - kBits;
    }
  }
  dm = fine ? pack2h(d, m) : 0x7FFF7FFFu;
  return fine ? q : 0u;
}

// The rows of a CTA: heads first .. first + count - 1 of its tokens, token by token.
// A slot of 2^lph_log2 lanes takes every slots-th row.  kPer: 8s of dimensions of a
// row that one lane holds (2 where D > 256).  kMates: they are two runs of 4, half a
// head apart (half layout, all of a head turns, D <= 256 a multiple of 64).
template <bool kQ4, int kPer, bool kMates>
__global__ void __launch_bounds__(kNrThreads, kPer == 1 ? 4 : 2)
    norm_rope_kernel(const __grid_constant__ NormRopeArgs N, int lph_log2, int tokens, int per_cta) {
  __shared__ __align__(16) float cosines[kNrTokens][kNrMaxD / 2], sines[kNrTokens][kNrMaxD / 2];
  __shared__ __align__(16) float rows[kNrThreads / 32][kNrMaxD];
  const RopeArgs& A = N.rope;
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int nt = (int)min((int64_t)tokens, A.M - t0);
  const int lph = 1 << lph_log2, slots = kNrThreads >> lph_log2;
  const int c = threadIdx.x & (lph - 1), slot = threadIdx.x >> lph_log2;
  const int heads = A.H + 2 * A.Hkv, first = blockIdx.y * per_cta, count = min(per_cta, heads - first);
  float* row = &rows[threadIdx.x >> 5][((threadIdx.x & 31) >> lph_log2) * A.D];
  const int h2 = A.n_rot / 2;
  const float per_d = 1.0f / (float)A.D;
  const bool vec = A.half ? h2 % 8 == 0 : true;  // this lane's turns lie together
  dependent_wait();

  // This CTA's part of each tensor; offsets within it fit 32 bits.
  const float *q_in = A.q + t0 * A.H * A.D, *k_in = A.k + t0 * A.Hkv * A.D, *v_in = A.v + t0 * A.Hkv * A.D;
  uint16_t* q_to = A.q_out + t0 * A.H * A.D;
  struct Row {  // a head of a token (tok >= nt: none), on its way
    int tok, hd;
    uint4 v[kPer][2];
  };
  const int tok_step = slots / count, hd_step = slots - tok_step * count;
  int tok_next = slot / count, hd_next = first + slot - tok_next * count;
  const bool whole = 8 * lph * kPer == A.D;  // every lane has dimensions
  auto load = [&](Row& x) {  // past the last row: the last token's again
    x.tok = tok_next;
    x.hd = hd_next;
    const bool is_q = x.hd < A.H, is_k = x.hd < A.H + A.Hkv;
    const float* base = is_q ? q_in : is_k ? k_in : v_in;
    const int h = x.hd - (is_q ? 0 : is_k ? A.H : A.H + A.Hkv);
    const float* in = base + (min(x.tok, nt - 1) * (is_q ? A.H : A.Hkv) + h) * A.D;
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      const int d0 = 8 * (c + r * lph), d = whole || d0 < A.D ? (kMates ? d0 / 2 : d0) : 0;
      x.v[r][0] = ldg_stream16(in + d);
      x.v[r][1] = ldg_stream16(in + d + (kMates ? h2 : 4));
    }
    tok_next += tok_step;
    hd_next += hd_step;
    if (hd_next >= first + count) hd_next -= count, ++tok_next;
  };
  Row x0, x1;  // two rows on their way
  load(x0);
  load(x1);
  for (int j = threadIdx.x; j < nt * h2; j += kNrThreads) {
    const int t = j / h2, i = j - t * h2;
    const float2 cs = turn(A, A.pos0 + t0 + t, i);
    cosines[t][i] = cs.x;
    sines[t][i] = cs.y;
  }
  uint4 gq[kPer], gk[kPer];
#pragma unroll
  for (int r = 0; r < kPer; ++r) {
    const int d0 = 8 * (c + r * lph);
    gq[r] = gk[r] = make_uint4(0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u);  // ones
    if (d0 < A.D) {
      auto gamma = [&](const uint16_t* from) {
        if (!kMates) return *reinterpret_cast<const uint4*>(from + d0);
        const uint2 a = *reinterpret_cast<const uint2*>(from + d0 / 2);
        const uint2 b = *reinterpret_cast<const uint2*>(from + d0 / 2 + h2);
        return make_uint4(a.x, a.y, b.x, b.y);
      };
      if (N.q_gamma) gq[r] = gamma(N.q_gamma);
      if (N.k_gamma) gk[r] = gamma(N.k_gamma);
    }
  }
  __syncthreads();

  auto compute = [&](Row& x) {
    const int tok = x.tok, hd = x.hd;
    float y[kPer][8];
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      const uint4 lo = x.v[r][0], hi = x.v[r][1];
      const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) y[r][e] = __uint_as_float(w[e]);
      if (!whole && 8 * (c + r * lph) >= A.D)
#pragma unroll
        for (int e = 0; e < 8; ++e) y[r][e] = 0.f;
    }
    load(x);
    const bool on = tok < nt, is_q = hd < A.H, turns = hd < A.H + A.Hkv;
    // every lane takes the same path through the shuffles: a head without a norm (v,
    // or no gamma) only drops the result
    if (N.q_gamma || N.k_gamma) {
      Two sums(0.f);
#pragma unroll
      for (int r = 0; r < kPer; ++r)
#pragma unroll
        for (int e = 0; e < 8; e += 2) sums = fma2(Two(y[r][e], y[r][e + 1]), Two(y[r][e], y[r][e + 1]), sums);
      float ss, odd;
      sums.get(ss, odd);
      ss += odd;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1)
        if (o < lph) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (is_q ? N.q_gamma != nullptr : turns && N.k_gamma != nullptr) {
        const float inv = rsqrtf(fmaf(ss, per_d, N.eps));
#pragma unroll
        for (int r = 0; r < kPer; ++r) {
          const uint4 g4 = is_q ? gq[r] : gk[r];
          const uint32_t g[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 gg = __half22float2(*reinterpret_cast<const __half2*>(&g[e]));
            mul2(mul2(Two(y[r][2 * e], y[r][2 * e + 1]), Two(inv)), Two(gg.x, gg.y)).get(y[r][2 * e], y[r][2 * e + 1]);
          }
        }
      }
    }
    if (kMates) {
      if (turns && on && 8 * c < A.D) {
        const float4 cc = *reinterpret_cast<const float4*>(cosines[tok] + 4 * c);
        const float4 ss = *reinterpret_cast<const float4*>(sines[tok] + 4 * c);
        const Two tc[2] = {Two(cc.x, cc.y), Two(cc.z, cc.w)}, ts[2] = {Two(ss.x, ss.y), Two(ss.z, ss.w)};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const Two a(y[0][2 * e], y[0][2 * e + 1]), b(y[0][4 + 2 * e], y[0][5 + 2 * e]);
          fma2(a, tc[e], mul2(mul2(b, ts[e]), Two(-1.f))).get(y[0][2 * e], y[0][2 * e + 1]);
          fma2(b, tc[e], mul2(a, ts[e])).get(y[0][4 + 2 * e], y[0][5 + 2 * e]);
        }
      }
    } else if (h2 > 0 && __any_sync(0xffffffffu, turns && on)) {
      if (A.half) {  // the mates are other lanes'
        __syncwarp();
#pragma unroll
        for (int r = 0; r < kPer; ++r) {
          const int d0 = 8 * (c + r * lph);
          if (d0 < A.D) {
            *reinterpret_cast<float4*>(row + d0) = make_float4(y[r][0], y[r][1], y[r][2], y[r][3]);
            *reinterpret_cast<float4*>(row + d0 + 4) = make_float4(y[r][4], y[r][5], y[r][6], y[r][7]);
          }
        }
        __syncwarp();
      }
      if (turns && on) {
        const float *cosine = cosines[tok], *sine = sines[tok];
#pragma unroll
        for (int r = 0; r < kPer; ++r) {
          const int d0 = 8 * (c + r * lph);
          if (d0 >= A.n_rot) continue;
          if (!A.half) {
            const float4 cc = *reinterpret_cast<const float4*>(cosine + d0 / 2);
            const float4 ss = *reinterpret_cast<const float4*>(sine + d0 / 2);
            const float tc[4] = {cc.x, cc.y, cc.z, cc.w}, ts[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (d0 + 2 * e < A.n_rot) {
                const float a = y[r][2 * e], b = y[r][2 * e + 1];
                y[r][2 * e] = a * tc[e] - b * ts[e];
                y[r][2 * e + 1] = b * tc[e] + a * ts[e];
              }
          } else if (vec) {  // all 8 dimensions turn, on the same side of their mates
            const bool second = d0 >= h2;
            const int p0 = second ? d0 - h2 : d0, m0 = second ? p0 : d0 + h2;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float4 cc = *reinterpret_cast<const float4*>(cosine + p0 + 4 * q);
              const float4 ss = *reinterpret_cast<const float4*>(sine + p0 + 4 * q);
              const float4 mm = *reinterpret_cast<const float4*>(row + m0 + 4 * q);
              const float tc[4] = {cc.x, cc.y, cc.z, cc.w}, ts[4] = {ss.x, ss.y, ss.z, ss.w};
              const float mate[4] = {mm.x, mm.y, mm.z, mm.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                y[r][4 * q + e] = y[r][4 * q + e] * tc[e] + mate[e] * (second ? ts[e] : -ts[e]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int d = d0 + e;
              if (d >= A.n_rot) continue;
              const bool second = d >= h2;
              const int p = second ? d - h2 : d;
              y[r][e] = y[r][e] * cosine[p] + row[second ? p : d + h2] * (second ? sine[p] : -sine[p]);
            }
          }
        }
      }
    }
    const int g = hd - A.H - (turns ? 0 : A.Hkv);  // key/value head
    const int64_t at = (int64_t)g * A.Lmax + A.pos0 + t0 + tok;  // its row of the cache
    const bool packs = kQ4 && __any_sync(0xffffffffu, on && !is_q);
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      const int d0 = 8 * (c + r * lph);
      uint32_t q = 0, dm = 0, dm2 = 0;
      if (packs && !kMates) q = quantize<8>(y[r], dm);
      if (packs && kMates) {
        // lanes of a pair: the even one gets 8 dimensions of the first run, the odd one of the second
        const uint32_t a = quantize<4>(y[r], dm), b = quantize<4>(y[r] + 4, dm2);
        const uint32_t other = __shfl_xor_sync(0xffffffffu, c & 1 ? a : b, 1);
        q = c & 1 ? other | (b << 16) : a | (other << 16);
      }
      if (!on || d0 >= A.D) continue;
      if (!kQ4 || is_q) {
        uint16_t* out = is_q ? q_to + (tok * A.H + hd) * A.D : (turns ? A.k_cache : A.v_cache) + at * A.D;
        const uint4 h = make_uint4(pack2h(y[r][0], y[r][1]), pack2h(y[r][2], y[r][3]), pack2h(y[r][4], y[r][5]),
                                   pack2h(y[r][6], y[r][7]));
        if (!kMates) {
          *reinterpret_cast<uint4*>(out + d0) = h;
        } else {
          *reinterpret_cast<uint2*>(out + d0 / 2) = make_uint2(h.x, h.y);
          *reinterpret_cast<uint2*>(out + d0 / 2 + h2) = make_uint2(h.z, h.w);
        }
      } else {
        uint32_t* q_row = (turns ? N.k_q4 : N.v_q4) + at * (A.D / 8);
        uint32_t* dm_row = (turns ? N.k_dm : N.v_dm) + at * (A.D / 32);
        if (!kMates) {
          q_row[d0 / 8] = q;
          if ((c & 3) == 0) dm_row[d0 / 32] = dm;
        } else {
          q_row[(c & 1 ? h2 / 8 : 0) + c / 2] = q;
          if ((c & 7) == 0) dm_row[c / 8] = dm;
          if ((c & 7) == 1) dm_row[h2 / 32 + c / 8] = dm2;
        }
      }
    }
  };
  const int total = (nt * count + slots - 1) / slots;  // rows of the longest slot
#pragma unroll 1
  for (int step = 0; step < total; step += 2) {
    compute(x0);
    if (step + 1 < total) compute(x1);
  }
}

template <bool kQ4>
cudaError_t launch(const NormRopeArgs& a, cudaStream_t s) {
  const RopeArgs& r = a.rope;
  const bool two = r.D > 256;
  int lph_log2 = 0;
  while (lph_log2 < 5 && (8 << lph_log2) < r.D) ++lph_log2;
  const int slots = kNrThreads >> lph_log2, heads = r.H + 2 * r.Hkv;
  // Few tokens: one a CTA, its heads over several CTAs.  us with 1, 2, 4 tokens a CTA,
  // 24 + 8 + 8 heads of 128 into fp16: 152 tokens 3.7, 4.3, 6.6; 304: 5.2, 4.3, 6.7; 1216:
  // 17.2, 8.4, 8.8; 2047: 27.7, 13.8, 15.0; 4095: 54.2, 26.2, 25.3; 8190: 106, 49.9, 47.5.
  const int64_t sms = device_sms();
  const int tokens = 2 * r.M <= 3 * sms ? 1 : r.M <= 16 * sms ? 2 : kNrTokens;
  const int per_cta = tokens == 1 ? std::min(slots, heads) : heads;
  const dim3 grid((unsigned)((r.M + tokens - 1) / tokens), (unsigned)((heads + per_cta - 1) / per_cta));
  const bool mates = r.half && r.n_rot == r.D && !two && r.D % 64 == 0;
  return launch_dependent(two     ? norm_rope_kernel<kQ4, 2, false>
                          : mates ? norm_rope_kernel<kQ4, 1, true>
                                  : norm_rope_kernel<kQ4, 1, false>,
                          grid, kNrThreads, 0, 1, s, a, lph_log2, tokens, per_cta);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t s) {
  return a.k_q4 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace qk
