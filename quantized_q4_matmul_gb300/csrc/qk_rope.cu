// qk_rope.cu -- rotary positions on the QKV projections' outputs, and the new
// rows of the KV cache.
//
// Source: DAMASCUS project overview, "[04] one decode step" (RoPE between the
// QKV projections and the attention over the KV cache), "[06] the target"
// (theta = 500000).
//
// For token i at position p = pos0 + i, pair j of the first n_rot dimensions of
// every q and k head turns by the angle p * inv_freq[j]:
//   (a, b) -> magnitude * (a cos - b sin, b cos + a sin).
// The angle's fraction of a turn is taken in fp64 (p * f / 2 pi minus its
// nearest integer: at p = 10^5 an fp32 angle would be off by 2^-8 rad), its
// sine and cosine in fp32.
//
// HBM-bound for a prompt: one CTA per token computes the token's n_rot / 2
// sines and cosines once, in shared memory, while its first inputs are on their
// way, and turns every head with them; each input is read once (2048 tokens, 32
// + 8 + 8 heads of 128, 96 dimensions turning: 14.3 us or 5.3 TB/s).  A decode
// step has one token: its heads are spread over several CTAs, each with its own
// table (1.8 us between calls of a graph, all latency).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qk_device.cuh"
#include "qk_internal.h"

namespace qk {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 256;  // D <= 512

// Sine and cosine of every pair of the token at position p, times the magnitude.
__device__ __forceinline__ void fill_table(const RopeArgs& A, int64_t p, float2* cs) {
  for (int j = threadIdx.x; j < A.n_rot / 2; j += kRopeThreads) {
    const double t = (double)p * A.inv_freq[j] * 0.15915494309189533577;  // turns
    float s, c;
    sincospif(2.0f * (float)(t - rint(t)), &s, &c);
    cs[j] = make_float2(c * A.magnitude, s * A.magnitude);
  }
}

// Where head `hd` of the q heads, k heads and v heads of token i (position p)
// comes from and goes to; the return value says whether it turns.
__device__ __forceinline__ bool head_of(const RopeArgs& A, int64_t i, int64_t p, int hd, const float*& in,
                                        uint16_t*& out) {
  if (hd < A.H) {
    in = A.q + (i * A.H + hd) * A.D;
    out = A.q_out + (i * A.H + hd) * A.D;
    return true;
  }
  const bool k = hd < A.H + A.Hkv;
  const int g = hd - A.H - (k ? 0 : A.Hkv);
  in = (k ? A.k : A.v) + (i * A.Hkv + g) * A.D;
  out = (k ? A.k_cache : A.v_cache) + ((int64_t)g * A.Lmax + p) * A.D;
  return k;
}

__device__ __forceinline__ uint2 half4(float a, float b, float c, float d) {
  const __half2 x = __floats2half2_rn(a, b), y = __floats2half2_rn(c, d);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

// n_rot a multiple of 8: an item is 8 dimensions of a head, two 16-byte loads.
// Of the turning dimensions it has four pairs (two runs of four dimensions
// n_rot / 2 apart, or one run of eight), of the others a run of eight.
constexpr int kRopeItems = 3;  // items of a thread in flight: 48 heads of 128 at once

__global__ void __launch_bounds__(kRopeThreads) rope_kv_kernel(const __grid_constant__ RopeArgs A) {
  __shared__ float2 cs[kRopeMaxPairs];
  const int64_t i = blockIdx.x, p = A.pos0 + i;
  const int per_head = A.D / 8, items = (A.H + 2 * A.Hkv) * per_head, step = gridDim.y * kRopeThreads;
  const int apart = A.half ? A.n_rot / 2 : 4;  // from a turning item's first run to its second
  bool ready = false;
  dependent_wait();
  for (int w0 = blockIdx.y * kRopeThreads + threadIdx.x; w0 - (int)threadIdx.x < items; w0 += kRopeItems * step) {
    uint4 x[kRopeItems], y[kRopeItems];
#pragma unroll
    for (int b = 0; b < kRopeItems; ++b) {
      const int w = w0 + b * step;
      if (w < items) {
        const int hd = w / per_head, c = w - hd * per_head;
        const float* in;
        uint16_t* out;
        const bool turns = head_of(A, i, p, hd, in, out) && c < A.n_rot / 8;
        const float* src = in + (turns && A.half ? 4 * c : 8 * c);
        x[b] = ldg_stream16(src);
        y[b] = ldg_stream16(src + (turns ? apart : 4));
      }
    }
    if (!ready) {
      fill_table(A, p, cs);
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int b = 0; b < kRopeItems; ++b) {
      const int w = w0 + b * step;
      if (w >= items) continue;
      const int hd = w / per_head, c = w - hd * per_head;
      const float* in;
      uint16_t* out;
      const bool turns = head_of(A, i, p, hd, in, out) && c < A.n_rot / 8;
      const float f[8] = {__uint_as_float(x[b].x), __uint_as_float(x[b].y), __uint_as_float(x[b].z),
                          __uint_as_float(x[b].w), __uint_as_float(y[b].x), __uint_as_float(y[b].y),
                          __uint_as_float(y[b].z), __uint_as_float(y[b].w)};
      float g[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = f[e];
      if (turns) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 t = cs[4 * c + e];
          const float a = A.half ? f[e] : f[2 * e], b2 = A.half ? f[4 + e] : f[2 * e + 1];
          const float ra = a * t.x - b2 * t.y, rb = b2 * t.x + a * t.y;
          if (A.half) {
            g[e] = ra;
            g[4 + e] = rb;
          } else {
            g[2 * e] = ra;
            g[2 * e + 1] = rb;
          }
        }
      }
      const uint2 lo = half4(g[0], g[1], g[2], g[3]), hi = half4(g[4], g[5], g[6], g[7]);
      if (turns && A.half) {
        *reinterpret_cast<uint2*>(out + 4 * c) = lo;
        *reinterpret_cast<uint2*>(out + 4 * c + apart) = hi;
      } else {
        *reinterpret_cast<uint4*>(out + 8 * c) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  }
}

// Any even n_rot: an item is 4 dimensions of a head, a turning one reads its
// mate beside it (the runs of pairs do not fall on 16-byte boundaries).
__global__ void __launch_bounds__(kRopeThreads) rope_kv_any_kernel(const __grid_constant__ RopeArgs A) {
  __shared__ float2 cs[kRopeMaxPairs];
  const int64_t i = blockIdx.x, p = A.pos0 + i;
  dependent_wait();
  fill_table(A, p, cs);
  __syncthreads();
  const int n4 = A.D / 4, items = (A.H + 2 * A.Hkv) * n4, h = A.n_rot / 2;
  for (int w = blockIdx.y * kRopeThreads + threadIdx.x; w < items; w += gridDim.y * kRopeThreads) {
    const int hd = w / n4, d0 = 4 * (w - hd * n4);
    const float* in;
    uint16_t* out;
    const bool turns = head_of(A, i, p, hd, in, out);
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = d0 + e;
      const float x = in[d];
      if (turns && d < A.n_rot) {
        const bool second = A.half ? d >= h : (d & 1) != 0;
        const int pair = A.half ? (second ? d - h : d) : d >> 1;
        const float mate = in[A.half ? (second ? d - h : d + h) : d ^ 1];
        y[e] = second ? x * cs[pair].x + mate * cs[pair].y : x * cs[pair].x - mate * cs[pair].y;
      } else {
        y[e] = x;
      }
    }
    *reinterpret_cast<uint2*>(out + d0) = half4(y[0], y[1], y[2], y[3]);
  }
}

}  // namespace

cudaError_t launch_rope_kv(const RopeArgs& a, cudaStream_t s) {
  const bool vec = a.n_rot % 8 == 0;
  const int items = (a.H + 2 * a.Hkv) * (a.D / (vec ? 8 : 4));
  // Few tokens: a CTA per 256 items, so that the heads' loads are all in flight.
  // 24 + 8 + 8 heads of 128, us so and with a CTA per token: 1 token 1.9, 2.7; 100
  // tokens 2.9, 3.0; 300 4.0, 4.4; 2048 14.4, 10.8.
  const int split = a.M <= 2 * (int64_t)device_sms() ? (items + kRopeThreads - 1) / kRopeThreads : 1;
  const dim3 grid((unsigned)a.M, (unsigned)split);
  return launch_dependent(vec ? rope_kv_kernel : rope_kv_any_kernel, grid, kRopeThreads, 0, 1, s, a);
}

}  // namespace qk
