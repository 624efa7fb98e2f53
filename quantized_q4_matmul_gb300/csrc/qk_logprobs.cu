// qk_logprobs.cu -- log probabilities of given tokens, entropy and the top
// alternatives from the LM head's logits.
//
// Source: DAMASCUS project overview, "[02] the pipeline" (the tied LM head's
// logits go to the sampler; greedy and top-k are choices among them).
//
// With m the row's maximum and z = x - m:
//   S = sum e^z, T = sum e^z z, lse = m + log S,
//   logprob(t) = z_t - log S,  entropy = log S - T / S,
// all relative to m, so that nothing large cancels.  One pass keeps a running
// (m, S, T) per thread, rescaled when its maximum moves.
//
// The order of the alternatives is that of a 64-bit key, the logit's bits in
// sortable form above the complement of the token: larger logits first, equal
// ones by the lower token.
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>

#include "qk_device.cuh"
#include "qk_internal.h"

namespace qk {

namespace {

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Sortable bits: larger floats have larger bits, NaN the smallest of all.
__device__ __forceinline__ uint32_t order_bits(float x) {
  if (x != x) return 0u;
  if (x == 0.f) x = 0.f;  // -0 equals +0
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint64_t key_of(float x, int token) {
  return ((uint64_t)order_bits(x) << 32) | (uint32_t)~token;
}

// (m, S, T) of a set of logits; the empty set is (-FLT_MAX, 0, 0).
struct Stat {
  float m, S, T;
};

__device__ __forceinline__ void rescale(Stat& a, float m) {  // to a reference m >= a.m
  const float d = fmaxf(a.m - m, -1e30f), f = ex2(d * kLog2e);
  a.T = f * (a.T + d * a.S);
  a.S *= f;
  a.m = m;
}

__device__ __forceinline__ void add(Stat& a, float x) {
  if (x > a.m) rescale(a, x);
  const float z = x - a.m, e = ex2(z * kLog2e);
  a.S += e;
  a.T = fmaf(e, fmaxf(z, -1e30f), a.T);  // -inf: 0 * -1e30
}

__device__ __forceinline__ Stat join(Stat a, Stat b) {
  const float m = fmaxf(a.m, b.m);
  rescale(a, m);
  rescale(b, m);
  return Stat{m, a.S + b.S, a.T + b.T};
}

// Insert key k (the same in every lane) into the warp's descending list, one
// key per lane.
__device__ __forceinline__ void insert(uint64_t& mine, uint64_t k, int lane) {
  const uint32_t above = __ballot_sync(0xffffffffu, mine > k);  // a prefix of the lanes
  const uint64_t left = __shfl_up_sync(0xffffffffu, mine, 1);
  const int at = __popc(above);
  if (lane == at) mine = k;
  else if (lane > at) mine = left;
}

__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const __grid_constant__ LogprobArgs A) {
  __shared__ Stat wstat[kLpWarps];
  __shared__ uint64_t wtop[kLpWarps][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x;
  const float* x = A.logits + row * A.V;
  const int V = A.V, n = A.top_n;
  Stat st{-FLT_MAX, 0.f, 0.f};
  uint64_t top = 0, last = 0;  // this lane's key of the warp's list; its n-th key
  for (int base = warp * 32; base < V; base += kLpThreads) {
    const int v = base + lane;
    const bool on = v < V;
    const float f = on ? x[v] : 0.f;
    if (on) add(st, f);
    if (n > 0) {
      const uint64_t k = on ? key_of(f, v) : 0;
      uint32_t cand = __ballot_sync(0xffffffffu, k > last);
      while (cand) {
        const int src = __ffs(cand) - 1;
        cand &= cand - 1;
        const uint64_t kk = __shfl_sync(0xffffffffu, k, src);
        if (kk > last) {
          insert(top, kk, lane);
          last = __shfl_sync(0xffffffffu, top, n - 1);
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Stat b{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.S, o),
                 __shfl_xor_sync(0xffffffffu, st.T, o)};
    st = join(st, b);
  }
  if (lane == 0) wstat[warp] = st;
  wtop[warp][lane] = top;
  __syncthreads();
  if (warp != 0) return;
  st = wstat[0];
  for (int w = 1; w < kLpWarps; ++w) st = join(st, wstat[w]);
  const float log_s = st.S > 0.f ? logf(st.S) : NAN;
  if (lane == 0) {
    if (A.entropy) A.entropy[row] = log_s - st.T / st.S;
    if (A.logprob) {
      const int t = A.tokens[row];
      A.logprob[row] = t >= 0 && t < V ? x[t] - st.m - log_s : NAN;
    }
  }
  if (n > 0) {
    for (int w = 1; w < kLpWarps; ++w)
      for (int i = 0; i < n; ++i) {
        const uint64_t k = wtop[w][i];
        if (k <= last) break;
        insert(top, k, lane);
        last = __shfl_sync(0xffffffffu, top, n - 1);
      }
    if (lane < n) {
      const int t = (int)~(uint32_t)top;
      A.top_ids[row * n + lane] = t;
      A.top_logprobs[row * n + lane] = x[t] - st.m - log_s;
    }
  }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t s) {
  logprobs_kernel<<<(unsigned)a.M, kLpThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace qk
