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
// (m, S, T) per thread, rescaled when a batch's maximum passes it.
//
// HBM-bound for many rows: the row is read once, 8 independent 16-byte loads
// per thread and batch.  The alternatives cost almost nothing on the way: a
// thread notes the maximum of every batch of 32 logits (a segment) that it
// needs for the rescaling anyway.  Afterwards t0, the n-th largest of the 512
// threads' maxima, is a lower bound of the n-th largest logit, so the
// alternatives lie in the few segments whose maximum reaches it; only those
// (about n of 4008) are read again.
//
// The order of the alternatives is that of a 64-bit key, the logit's bits in
// sortable form above the complement of the token: larger logits first, equal
// ones by the lower token.  All keys differ, so the result does not depend on
// the order in which candidates are found.
//
// Few rows: a cluster of up to 8 CTAs splits a row; each finds its own sums and
// top n, and rank 0 joins them (distributed shared memory, in rank order).
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>

#include "qk_device.cuh"
#include "qk_internal.h"

namespace qk {

namespace {

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpVecs = 8;                           // 16-byte loads per thread and batch
constexpr int kLpBatch = kLpThreads * kLpVecs;       // vectors per batch
constexpr int kLpSegs = 8;                           // segments per thread (of one batch each up to 131072 logits)
constexpr int kLpTop = 32;                           // largest top_n
constexpr int kLpTies = 64;                          // segments whose maximum is t0 itself, at most, before the scan
constexpr int kLpList = kLpTop * kLpSegs + kLpTies;  // segments read again
constexpr int kLpCand = 1024;                        // candidate keys: 512 kept, 512 of a round
constexpr int kLpMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max(x, lo) that keeps NaN.
__device__ __forceinline__ float max_nan(float x, float lo) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(lo));
  return y;
}

// Sortable bits: larger floats have larger bits, -0 those of +0, NaN 0.
__device__ __forceinline__ uint32_t order_bits(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float from_order_bits(uint32_t b) {
  if (b == 0u) return NAN;
  return __uint_as_float(b & 0x80000000u ? b & 0x7FFFFFFFu : ~b);
}

__device__ __forceinline__ uint64_t key_of(uint32_t bits, int token) { return ((uint64_t)bits << 32) | (uint32_t)~token; }

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

__device__ __forceinline__ Stat join(Stat a, Stat b) {
  const float m = fmaxf(a.m, b.m);
  rescale(a, m);
  rescale(b, m);
  return Stat{m, a.S + b.S, a.T + b.T};
}

__device__ __forceinline__ Stat shfl_xor(const Stat& a, int o) {
  return Stat{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.S, o),
              __shfl_xor_sync(0xffffffffu, a.T, o)};
}

struct LpShared {
  float seg[kLpSegs][kLpThreads];  // each thread's segment maxima
  float top[kLpWarps][kLpTop];     // warps' sorted maxima
  uint64_t cand[kLpCand];
  uint64_t best[kLpTop];           // this CTA's top n, sorted
  uint64_t all[kLpMaxCluster * kLpTop];  // rank 0: every CTA's
  Stat wstat[kLpWarps];
  Stat cstat[kLpMaxCluster];       // rank 0: every CTA's
  int list[kLpList];               // segments to read again: 512 * segment + thread
  int n_above, n_equal, n_cand;
};

// One step of a bitonic sort across the warp: lanes o apart, the larger value
// to the lower lane where `down`.
__device__ __forceinline__ float exchange(float v, int o, bool down, int lane) {
  const float w = __shfl_xor_sync(0xffffffffu, v, o);
  const bool low = (lane & o) == 0;
  return (low == down) ? fmaxf(v, w) : fminf(v, w);
}

// The n-th largest (1-based) of one value per thread, to every thread.
__device__ float nth_of_threads(LpShared& S, float v, int n, int warp, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int o = k >> 1; o > 0; o >>= 1) v = exchange(v, o, (lane & k) == 0 || k == 32, lane);
  S.top[warp][lane] = v;
  // the 32 largest of two descending lists a, b are max(a_i, b_(31 - i)), a bitonic sequence
  for (int half = kLpWarps / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (warp < half) {
      v = fmaxf(v, S.top[warp + half][31 - lane]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v = exchange(v, o, true, lane);
    }
    __syncthreads();
    if (warp < half) S.top[warp][lane] = v;
  }
  __syncthreads();
  return S.top[0][n - 1];
}

// Keep the n largest of cand[0 .. count): sorted into best[], the rest of
// best[0 .. n) zero.  A key's place is the number of larger keys.
__device__ void select_n(uint64_t* best, const uint64_t* cand, int count, int n, int tid) {
  if (tid < n) best[tid] = 0;
  __syncthreads();
  for (int i = tid; i < count; i += kLpThreads) {
    const uint64_t k = cand[i];
    int place = 0;
    for (int j = 0; j < count; ++j) place += cand[j] > k;
    if (place < n && k != 0) best[place] = k;
  }
  __syncthreads();
}

// Append the keys of lanes with `on` to the candidates.
__device__ __forceinline__ void append(LpShared& S, uint64_t key, bool on, int lane) {
  const uint32_t b = __ballot_sync(0xffffffffu, on);
  if (b == 0) return;
  int at = 0;
  if (lane == 0) at = atomicAdd(&S.n_cand, __popc(b));
  at = __shfl_sync(0xffffffffu, at, 0);
  if (on) S.cand[at + __popc(b & ((1u << lane) - 1u))] = key;
}

// After a round of at most 512 appended keys: keep n if there is no room for another.
__device__ __forceinline__ void make_room(LpShared& S, int n, int tid) {
  __syncthreads();
  const int count = S.n_cand;
  __syncthreads();  // read by every thread before the next round adds to it
  if (count <= kLpCand - kLpThreads) return;
  select_n(S.best, S.cand, count, n, tid);
  if (tid < n) S.cand[tid] = S.best[tid];
  if (tid == 0) S.n_cand = n;
  __syncthreads();
}

template <int C>
__global__ void __launch_bounds__(kLpThreads, 2) logprobs_kernel(const __grid_constant__ LogprobArgs A) {
  __shared__ LpShared S;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = C > 1 ? (int)(blockIdx.x % C) : 0;
  const int64_t row = blockIdx.x / C;
  const int V = A.V, n = A.top_n;
  const float* x = A.logits + row * (int64_t)V;
  // Vector j of the row holds logits 4 j - shift .. 4 j - shift + 3 (the row may
  // start off a 16-byte boundary); this CTA takes vectors v0 .. v1 - 1.
  const int shift = (int)((reinterpret_cast<uintptr_t>(x) >> 2) & 3);
  const int64_t nv = ((int64_t)V + shift + 3) / 4;
  const int64_t v0 = nv * rank / C, v1 = nv * (rank + 1) / C;
  const int batches = (int)((v1 - v0 + kLpBatch - 1) / kLpBatch);
  const int per_seg = (batches + kLpSegs - 1) / kLpSegs;  // batches per segment (1 up to 131072 logits)
  dependent_wait();
  float given = NAN;
  if (rank == 0 && tid == 0 && A.logprob) {
    const int t = A.tokens[row];
    if (t >= 0 && t < V) given = x[t];
  }
  if (tid == 0) S.n_above = S.n_equal = S.n_cand = 0;

  // ------------------------------------------------------------ the one pass
  Stat st{-FLT_MAX, 0.f, 0.f};
  float most = -INFINITY;  // this thread's maximum
  for (int s = 0, b = 0; b < batches; ++s) {
    float smax = -INFINITY;
    for (int e = min(b + per_seg, batches); b < e; ++b) {
      const int64_t first = v0 + (int64_t)b * kLpBatch + tid;
      float4 f[kLpVecs];
#pragma unroll
      for (int j = 0; j < kLpVecs; ++j) {
        const int64_t v = first + j * kLpThreads;
        const int64_t at = 4 * v - shift;
        f[j] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);  // past the slice: weight 0
        if (v < v1) {
          if (at >= 0 && at + 4 <= V) {
            const uint4 u = ldg_stream16(x + at);
            f[j] = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
          } else {
            if (at >= 0 && at < V) f[j].x = x[at];
            if (at + 1 >= 0 && at + 1 < V) f[j].y = x[at + 1];
            if (at + 2 >= 0 && at + 2 < V) f[j].z = x[at + 2];
            if (at + 3 >= 0 && at + 3 < V) f[j].w = x[at + 3];
          }
        }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < kLpVecs; ++j) mx = fmaxf(mx, fmaxf(fmaxf(f[j].x, f[j].y), fmaxf(f[j].z, f[j].w)));
      smax = fmaxf(smax, mx);
      if (mx > st.m) rescale(st, mx);
      // four partial sums keep the chains short; -200 has weight 0 (2^-288) and a finite product with it
      float ps[4] = {0.f, 0.f, 0.f, 0.f}, pt[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kLpVecs; ++j) {
        const float v[4] = {f[j].x, f[j].y, f[j].z, f[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float z = max_nan(v[i] - st.m, -200.f), w = ex2(z * kLog2e);
          ps[i] += w;
          pt[i] = fmaf(w, z, pt[i]);
        }
      }
      st.S += (ps[0] + ps[1]) + (ps[2] + ps[3]);
      st.T += (pt[0] + pt[1]) + (pt[2] + pt[3]);
    }
    if (n > 0) S.seg[s][tid] = smax;
    most = fmaxf(most, smax);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) st = join(st, shfl_xor(st, o));
  if (lane == 0) S.wstat[warp] = st;

  // -------------------------------------------------------- the alternatives
  if (n > 0) {
    const float t0 = nth_of_threads(S, most, n, warp, lane);
    const uint32_t b0 = order_bits(t0);
    const int segs = batches > 0 ? (batches + per_seg - 1) / per_seg : 0;
    for (int s = 0; s < segs; ++s) {
      const bool filled = v0 + (int64_t)s * per_seg * kLpBatch + tid < v1;
      const float smax = S.seg[s][tid];
      if (filled && smax > t0) S.list[atomicAdd(&S.n_above, 1)] = s * kLpThreads + tid;  // at most n - 1 threads
    }
    __syncthreads();
    const int above = S.n_above;
    for (int s = 0; s < segs; ++s) {
      const bool filled = v0 + (int64_t)s * per_seg * kLpBatch + tid < v1;
      if (filled && !(S.seg[s][tid] > t0) && S.seg[s][tid] >= t0) {
        const int i = atomicAdd(&S.n_equal, 1);
        if (i < kLpTies) S.list[above + i] = s * kLpThreads + tid;
      }
    }
    __syncthreads();
    const bool scan = S.n_equal > kLpTies;  // many logits equal to t0: found by the scan below instead
    const int units = (above + (scan ? 0 : S.n_equal)) * per_seg;
    for (int u0 = 0; u0 < units; u0 += kLpWarps) {
      const int u = u0 + warp;
      bool on = false;
      uint64_t key = 0;
      if (u < units) {
        const int seg = S.list[u / per_seg], b = (seg / kLpThreads) * per_seg + u % per_seg;
        const int64_t v = v0 + (int64_t)b * kLpBatch + (lane >> 2) * kLpThreads + seg % kLpThreads;
        const int64_t at = 4 * v - shift + (lane & 3);
        if (v < v1 && at >= 0 && at < V) {
          const uint32_t bits = order_bits(x[at]);
          on = scan ? bits > b0 : bits >= b0;
          key = key_of(bits, (int)at);
        }
      }
      append(S, key, on, lane);
      make_room(S, n, tid);
    }
    // Ties at t0, and, where logits are NaN, those: in token order until n are found.
    if (scan || S.n_cand < n) {
      const int64_t lo = max((int64_t)0, 4 * v0 - shift), hi = min((int64_t)V, 4 * v1 - shift);
      for (int pass = scan ? 0 : 1; pass < 2; ++pass) {
        const uint32_t want = pass == 0 ? b0 : 0u;
        for (int64_t c = lo; c < hi; c += kLpThreads) {
          __syncthreads();
          if (S.n_cand >= n) break;  // the same in every thread
          __syncthreads();
          const int64_t at = c + tid;
          const bool on = at < hi && order_bits(x[at]) == want;
          append(S, key_of(want, (int)at), on, lane);
          make_room(S, n, tid);
        }
      }
    }
    __syncthreads();
    select_n(S.best, S.cand, S.n_cand, n, tid);
  } else {
    __syncthreads();
  }

  // ---------------------------------------------------------------- the join
  if (warp == 0) {
    st = S.wstat[lane % kLpWarps];
#pragma unroll
    for (int o = kLpWarps / 2; o > 0; o >>= 1) st = join(st, shfl_xor(st, o));
  }
  const uint64_t* best = S.best;
  if (C > 1) {
    cluster_sync_all();  // every CTA of the cluster is running
    if (warp == 0) {
      const uint32_t to = mapa_shared(smem_u32(&S.cstat[rank]), 0);
      const float part[3] = {st.m, st.S, st.T};
      if (lane < 3)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4u * (uint32_t)lane), "f"(part[lane]) : "memory");
      if (lane < n)
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(
                         mapa_shared(smem_u32(&S.all[rank * n + lane]), 0)),
                     "l"(S.best[lane])
                     : "memory");
    }
    cluster_sync_all();
    if (rank != 0) return;
    if (n > 0) select_n(S.best, S.all, C * n, n, tid);
    if (warp == 0) {
      st = S.cstat[0];
      for (int r = 1; r < C; ++r) st = join(st, S.cstat[r]);
    }
  }
  if (warp != 0) return;
  const float log_s = st.S > 0.f ? logf(st.S) : NAN;
  if (lane == 0) {
    if (A.entropy) A.entropy[row] = log_s - st.T / st.S;
    if (A.logprob) A.logprob[row] = given - st.m - log_s;
  }
  if (lane < n) {
    const uint64_t k = best[lane];
    A.top_ids[row * n + lane] = (int)~(uint32_t)k;
    A.top_logprobs[row * n + lane] = from_order_bits((uint32_t)(k >> 32)) - st.m - log_s;
  }
}

template <int C>
cudaError_t launch(const LogprobArgs& a, cudaStream_t s) {
  return launch_dependent(logprobs_kernel<C>, dim3((unsigned)(a.M * C)), kLpThreads, 0, C, s, a);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t s) {
  // A cluster per row while the rows alone leave SMs idle and a CTA's share
  // stays a quarter of a batch at least.
  int C = 1;
  while (C < kLpMaxCluster && a.M * C * 2 <= device_sms() && a.V / (2 * C) >= kLpBatch) C *= 2;
  switch (C) {
    case 1: return launch<1>(a, s);
    case 2: return launch<2>(a, s);
    case 4: return launch<4>(a, s);
    default: return launch<8>(a, s);
  }
}

}  // namespace qk
