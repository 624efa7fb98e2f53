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
// sines and cosines once, in shared memory, and turns every head with them;
// each input is read once.  A decode step has one token: its heads are spread
// over several CTAs, each with its own table.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qk_device.cuh"
#include "qk_internal.h"

namespace qk {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 256;  // D <= 512

// The output of dimension d of one head: in[0 .. D) with the turn applied.
__device__ __forceinline__ float turned(const RopeArgs& A, const float* in, int d, const float2* cs) {
  const float x = in[d];
  if (d >= A.n_rot) return x;
  int pair, mate;
  bool second;
  if (A.half) {
    const int h = A.n_rot / 2;
    second = d >= h;
    pair = second ? d - h : d;
    mate = second ? d - h : d + h;
  } else {
    second = d & 1;
    pair = d >> 1;
    mate = d ^ 1;
  }
  const float y = in[mate];
  return second ? x * cs[pair].x + y * cs[pair].y : x * cs[pair].x - y * cs[pair].y;
}

__global__ void __launch_bounds__(kRopeThreads) rope_kv_kernel(const __grid_constant__ RopeArgs A) {
  __shared__ float2 cs[kRopeMaxPairs];
  const int64_t i = blockIdx.x;
  const int64_t p = A.pos0 + i;
  for (int j = threadIdx.x; j < A.n_rot / 2; j += kRopeThreads) {
    const double t = (double)p * A.inv_freq[j] * 0.15915494309189533577;  // turns
    float s, c;
    sincospif(2.0f * (float)(t - rint(t)), &s, &c);
    cs[j] = make_float2(c * A.magnitude, s * A.magnitude);
  }
  __syncthreads();
  const int D = A.D, n4 = D / 4, heads = A.H + 2 * A.Hkv;
  for (int w = blockIdx.y * kRopeThreads + threadIdx.x; w < heads * n4; w += gridDim.y * kRopeThreads) {
    const int hd = w / n4, d = 4 * (w % n4);
    const float* in;
    uint16_t* out;
    bool turn = true;
    if (hd < A.H) {
      in = A.q + (i * A.H + hd) * D;
      out = A.q_out + (i * A.H + hd) * D;
    } else if (hd < A.H + A.Hkv) {
      const int g = hd - A.H;
      in = A.k + (i * A.Hkv + g) * D;
      out = A.k_cache + ((int64_t)g * A.Lmax + p) * D;
    } else {
      const int g = hd - A.H - A.Hkv;
      in = A.v + (i * A.Hkv + g) * D;
      out = A.v_cache + ((int64_t)g * A.Lmax + p) * D;
      turn = false;
    }
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = turn ? turned(A, in, d + e, cs) : in[d + e];
    const __half2 a = __floats2half2_rn(y[0], y[1]), b = __floats2half2_rn(y[2], y[3]);
    *reinterpret_cast<uint2*>(out + d) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

}  // namespace

cudaError_t launch_rope_kv(const RopeArgs& a, cudaStream_t s) {
  const int items = (a.H + 2 * a.Hkv) * (a.D / 4);
  const int split = a.M < 64 ? (items + kRopeThreads - 1) / kRopeThreads : 1;
  const dim3 grid((unsigned)a.M, (unsigned)split);
  rope_kv_kernel<<<grid, kRopeThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace qk
