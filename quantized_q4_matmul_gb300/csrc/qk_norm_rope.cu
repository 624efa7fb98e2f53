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
//   q = (x - m) / d rounded to the nearest of 0 .. 15 (0 where d = 0).
//
// HBM-bound for a prompt: each input is read once.  A CTA has one token and
// computes its n_rot / 2 sines and cosines once, while its first rows are on
// their way.  A head is 8 dimensions a lane: the sum of squares and a group's
// extremes meet by shuffles, and every lane keeps gamma and the turns of its
// dimensions in registers for all of its heads; the half layout's mates, which
// other lanes hold, pass through shared memory.  Few tokens: their heads are
// spread over several CTAs.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qk_device.cuh"
#include "qk_internal.h"
#include "qk_rope.cuh"

namespace qk {

namespace {

constexpr int kNrThreads = 256;
constexpr int kNrMaxD = 512;

__device__ __forceinline__ uint32_t pack2h(float a, float b) {
  const __half2 x = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}

// 8 values of a group of 32 that four lanes hold: their nibbles in order, and
// (d, m) as two fp16.  Every lane of the warp takes part.
__device__ __forceinline__ uint32_t quantize8(const float (&y)[8], uint32_t& dm) {
  float lo = y[0], hi = y[0];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lo = fminf(lo, y[e]);
    hi = fmaxf(hi, y[e]);
    bad |= !(fabsf(y[e]) < INFINITY);
  }
  if (bad) hi = INFINITY;
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float m = __half2float(__float2half_rn(lo));
  const float d = __half2float(__float2half_rn(fmaxf(hi - m, 0.f) / 15.f));
  // a value that is not finite, or m or 15 d past fp16, makes the group NaN (d is
  // infinite then, or NaN where m is: infinity less infinity)
  const bool fine = fabsf(m) < INFINITY && d <= 4366.f;
  uint32_t q = 0;
  if (d > 0.f)
#pragma unroll
    for (int e = 0; e < 8; ++e) q |= (uint32_t)fminf(fmaxf(rintf((y[e] - m) / d), 0.f), 15.f) << (4 * e);
  dm = fine ? pack2h(d, m) : 0x7FFF7FFFu;
  return fine ? q : 0u;
}

// A CTA: one token, heads blockIdx.y, blockIdx.y + gridDim.y ... of its H + 2 Hkv
// in turns of slots; a slot is 2^lph_log2 lanes.  kPer: runs of 8 dimensions of a
// head that one lane holds (2 where D > 256).
template <bool kQ4, int kPer>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs N, int lph_log2) {
  constexpr int kBatch = kPer == 1 ? 3 : 1;  // heads of a slot in flight: 48 of 128 at once
  __shared__ float2 cs[kNrMaxD / 2];
  __shared__ __align__(16) float rows[kNrThreads / 32][kNrMaxD];
  const RopeArgs& A = N.rope;
  const int64_t i = blockIdx.x, p = A.pos0 + i;
  const int lph = 1 << lph_log2, slots = kNrThreads >> lph_log2;
  const int c = threadIdx.x & (lph - 1), slot = threadIdx.x >> lph_log2;
  const int heads = A.H + 2 * A.Hkv, step = gridDim.y * slots;
  float* row = &rows[threadIdx.x >> 5][((threadIdx.x & 31) >> lph_log2) * A.D];
  const int h2 = A.n_rot / 2;
  float tc[kPer][8], ts[kPer][8];  // y = x tc + mate ts
  uint4 gq[kPer], gk[kPer];
  bool ready = false;
  dependent_wait();
  for (int h0 = blockIdx.y * slots; h0 < heads; h0 += kBatch * step) {
    uint4 x[kBatch][kPer][2];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int hd = h0 + b * step + slot;
      const float* in = hd < A.H           ? A.q + (i * A.H + hd) * A.D
                        : hd < A.H + A.Hkv ? A.k + (i * A.Hkv + hd - A.H) * A.D
                                           : A.v + (i * A.Hkv + hd - A.H - A.Hkv) * A.D;
#pragma unroll
      for (int r = 0; r < kPer; ++r) {
        const int d0 = 8 * (c + r * lph);
        x[b][r][0] = x[b][r][1] = make_uint4(0u, 0u, 0u, 0u);
        if (hd < heads && d0 < A.D) {
          x[b][r][0] = ldg_stream16(in + d0);
          x[b][r][1] = ldg_stream16(in + d0 + 4);
        }
      }
    }
    if (!ready) {
      fill_table(A, p, cs, kNrThreads);
      __syncthreads();
      ready = true;
#pragma unroll
      for (int r = 0; r < kPer; ++r) {
        const int d0 = 8 * (c + r * lph);
        gq[r] = gk[r] = make_uint4(0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u);  // ones
        if (d0 < A.D) {
          if (N.q_gamma) gq[r] = *reinterpret_cast<const uint4*>(N.q_gamma + d0);
          if (N.k_gamma) gk[r] = *reinterpret_cast<const uint4*>(N.k_gamma + d0);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = d0 + e;
          tc[r][e] = 1.f;
          ts[r][e] = 0.f;
          if (d < A.n_rot) {
            const bool second = A.half ? d >= h2 : (e & 1) != 0;
            const float2 t = cs[A.half ? (second ? d - h2 : d) : d >> 1];
            tc[r][e] = t.x;
            ts[r][e] = second ? t.y : -t.y;
          }
        }
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int hd = h0 + b * step + slot;
      const bool is_q = hd < A.H, turns = hd < A.H + A.Hkv;
      float y[kPer][8];
#pragma unroll
      for (int r = 0; r < kPer; ++r) {
        const uint32_t w[8] = {x[b][r][0].x, x[b][r][0].y, x[b][r][0].z, x[b][r][0].w,
                               x[b][r][1].x, x[b][r][1].y, x[b][r][1].z, x[b][r][1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) y[r][e] = __uint_as_float(w[e]);
      }
      // every lane takes the same path through the shuffles: a head without a
      // norm (v, or no gamma) only drops the result
      if (N.q_gamma || N.k_gamma) {
        float ss = 0.f;
#pragma unroll
        for (int r = 0; r < kPer; ++r)
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(y[r][e], y[r][e], ss);
        for (int o = 1; o < lph; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (is_q ? N.q_gamma != nullptr : turns && N.k_gamma != nullptr) {
          const float inv = 1.0f / sqrtf(ss / (float)A.D + N.eps);
#pragma unroll
          for (int r = 0; r < kPer; ++r) {
            const uint4 g4 = is_q ? gq[r] : gk[r];
            const uint32_t g[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 gg = __half22float2(*reinterpret_cast<const __half2*>(&g[e]));
              y[r][2 * e] = y[r][2 * e] * inv * gg.x;
              y[r][2 * e + 1] = y[r][2 * e + 1] * inv * gg.y;
            }
          }
        }
      }
      if (A.half && A.n_rot > 0) {  // the mates are other lanes'
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
      if (turns) {
#pragma unroll
        for (int r = 0; r < kPer; ++r) {
          const int d0 = 8 * (c + r * lph);
          float mate[8];
          if (A.half) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int d = d0 + e;
              mate[e] = d < A.n_rot ? row[d < h2 ? d + h2 : d - h2] : 0.f;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) mate[e] = y[r][e ^ 1];
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (d0 + e < A.n_rot) y[r][e] = y[r][e] * tc[r][e] + mate[e] * ts[r][e];
        }
      }
      const int g = hd - A.H - (turns ? 0 : A.Hkv);  // key/value head
#pragma unroll
      for (int r = 0; r < kPer; ++r) {
        const int d0 = 8 * (c + r * lph);
        uint32_t q = 0, dm = 0;
        if (kQ4) q = quantize8(y[r], dm);
        if (hd >= heads || d0 >= A.D) continue;
        if (!kQ4 || is_q) {
          uint16_t* out = is_q ? A.q_out + (i * A.H + hd) * A.D
                               : (turns ? A.k_cache : A.v_cache) + ((int64_t)g * A.Lmax + p) * A.D;
          *reinterpret_cast<uint4*>(out + d0) =
              make_uint4(pack2h(y[r][0], y[r][1]), pack2h(y[r][2], y[r][3]), pack2h(y[r][4], y[r][5]),
                         pack2h(y[r][6], y[r][7]));
        } else {
          const int64_t at = ((int64_t)g * A.Lmax + p) * (A.D / 8) + d0 / 8;
          (turns ? N.k_q4 : N.v_q4)[at] = q;
          if ((c & 3) == 0) (turns ? N.k_dm : N.v_dm)[at >> 2] = dm;
        }
      }
    }
  }
}

template <bool kQ4>
cudaError_t launch(const NormRopeArgs& a, cudaStream_t s) {
  const RopeArgs& r = a.rope;
  const bool two = r.D > 256;
  int lph_log2 = 0;
  while (lph_log2 < 5 && (8 << lph_log2) < r.D) ++lph_log2;
  const int slots = kNrThreads >> lph_log2;
  const int split = r.M <= 2 * (int64_t)device_sms() ? (r.H + 2 * r.Hkv + slots - 1) / slots : 1;
  const dim3 grid((unsigned)r.M, (unsigned)split);
  return launch_dependent(two ? norm_rope_kernel<kQ4, 2> : norm_rope_kernel<kQ4, 1>, grid, kNrThreads, 0, 1, s, a,
                          lph_log2);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t s) {
  return a.k_q4 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace qk
