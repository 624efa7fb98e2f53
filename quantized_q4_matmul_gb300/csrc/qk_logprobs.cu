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
// per thread and batch.  1024 rows of 128256: 80 us without alternatives (6.5
// TB/s), 95.3 us with 20 (5.5 TB/s): while one of an SM's two CTAs finds them,
// the other's loads alone do not fill the memory's latency.  The alternatives
// cost almost nothing on the way: a thread notes the maximum of every batch of
// 32 logits (a segment) that it needs for the rescaling anyway.  Afterwards t0, the n-th largest of the maxima
// of 64 groups of threads, is a lower bound of the n-th largest logit, so the
// alternatives lie in the few segments whose maximum reaches it; only those
// (about 1.2 n of 4008) are read again.
//
// The order of the alternatives is that of a 64-bit key, the logit's bits in
// sortable form above the complement of the token: larger logits first, equal
// ones by the lower token.  All keys differ, so the result does not depend on
// the order in which candidates are found.
//
// Few rows: a cluster of up to 8 CTAs splits a row; each finds its own sums and
// top n, and rank 0 joins them (distributed shared memory, in rank order).  One
// row of 128256: 5.5 us between calls of a graph, latency from end to end.
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
constexpr int kLpGroups = 64;                        // groups of up to 8 threads
constexpr int kLpTies = 64;                          // segments whose maximum is t0 itself, at most, before the scan
// Segments above t0: those of the threads of at most top_n - 1 groups.
constexpr int kLpList = (kLpTop - 1) * (kLpThreads / kLpGroups) * kLpSegs + kLpTies;
constexpr int kLpUnits = 3;                          // segments of a warp and round
constexpr int kLpRound = kLpUnits * kLpThreads;      // candidate keys of a round, at most
constexpr int kLpKeep = 512;                         // and between rounds
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

// The lanes' sets in one, in every lane.
__device__ __forceinline__ void warp_join(Stat& a) {
  float m = a.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  rescale(a, m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a.S += __shfl_xor_sync(0xffffffffu, a.S, o);
    a.T += __shfl_xor_sync(0xffffffffu, a.T, o);
  }
}

struct LpShared {
  float seg[kLpSegs][kLpThreads];  // each thread's segment maxima
  float top[kLpGroups];            // the groups' maxima
  uint64_t cand[kLpKeep + kLpRound];
  uint64_t best[kLpTop];           // this CTA's top n, sorted
  uint64_t all[kLpMaxCluster * kLpTop];  // rank 0: every CTA's
  Stat wstat[kLpWarps];
  Stat cstat[kLpMaxCluster];       // rank 0: every CTA's
  uint16_t list[kLpList];          // segments to read again: 512 * segment + thread
  int n_above, n_equal, n_cand;
};
static_assert(sizeof(LpShared) <= 48 * 1024 && kLpSegs * kLpThreads <= 65536, "static shared memory; segment numbers");

// One step of a bitonic sort of 64 values, two per lane (a: 0 .. 31, b: 32 ..
// 63): values o apart, the larger to the lower place where `down`.
__device__ __forceinline__ float exchange(float v, int o, bool down, int lane) {
  const float w = __shfl_xor_sync(0xffffffffu, v, o);
  const bool low = (lane & o) == 0;
  return (low == down) ? fmaxf(v, w) : fminf(v, w);
}

// A lower bound of the n-th largest of one value per thread that n of them
// reach: the n-th largest (1-based) of the groups' maxima.  Every warp sorts
// the 64 maxima for itself.  A group is 8 threads, or as few as give 64 groups
// of the threads that have any of the `nv` vectors (20000 rows of 511 logits,
// top 20: 1619 us with 8 always, whose 16 maxima exclude nothing).
__device__ __forceinline__ float bound_of_threads(LpShared& S, float v, int n, int64_t nv, int warp, int lane) {
  int lg = 3;  // a group is 2^lg threads
  static_assert(kLpThreads == kLpGroups << 3, "groups of 8 take every thread");
  while (lg > 0 && nv <= kLpGroups << (lg - 1)) --lg;
#pragma unroll
  for (int o = 1; o < kLpThreads / kLpGroups; o <<= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    if (o < 1 << lg) v = fmaxf(v, w);
  }
  const int t = 32 * warp + lane;
  if ((t & ((1 << lg) - 1)) == 0 && t >> lg < kLpGroups) S.top[t >> lg] = v;
  __syncthreads();
  float a = S.top[lane], b = S.top[lane + 32];
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int o = k >> 1; o > 0; o >>= 1) {
      const bool down = (lane & k) == 0 || k == 32;
      a = exchange(a, o, down, lane);
      b = exchange(b, o, k == 32 ? false : down, lane);  // ascending in the end: a, b bitonic
    }
  const float hi = fmaxf(a, b), lo = fminf(a, b);
  a = hi;
  b = lo;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = exchange(a, o, true, lane);
  return __shfl_sync(0xffffffffu, a, n - 1);  // n <= 32: among the upper half
}

// Keep the n largest of cand[0 .. count): sorted into best[], the rest of
// best[0 .. n) zero.  A key's place is the number of larger keys, which eight
// threads count together.
__device__ void select_n(uint64_t* best, const uint64_t* cand, int count, int n, int tid) {
  if (tid < n) best[tid] = 0;
  __syncthreads();
  for (int i0 = 0; i0 < count; i0 += kLpThreads / 8) {
    const int i = i0 + tid / 8;
    const uint64_t k = i < count ? cand[i] : 0;
    int place = 0;
#pragma unroll 4
    for (int j = tid % 8; j < count; j += 8) place += cand[j] > k;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
    if (tid % 8 == 0 && place < n && k != 0) best[place] = k;
  }
  __syncthreads();
}

// The same for `lists` (at most 8) lists of n keys, each in order: one thread
// for each list finds by halving how many of its keys are larger.
__device__ void select_n_sorted(uint64_t* best, const uint64_t* keys, int lists, int n, int tid) {
  if (tid < n) best[tid] = 0;
  __syncthreads();
  for (int i0 = 0; i0 < lists * n; i0 += kLpThreads / 8) {
    const int i = i0 + tid / 8, q = tid % 8;
    const uint64_t k = i < lists * n ? keys[i] : 0;
    int place = 0;
    if (q < lists) {
      int hi = n;
      while (place < hi) {
        const int mid = (place + hi) / 2;
        if (keys[q * n + mid] > k)
          place = mid + 1;
        else
          hi = mid;
      }
    }
    __syncwarp();
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
    if (q == 0 && place < n && k != 0) best[place] = k;
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

// After a round of at most kLpRound appended keys: keep n if there is no room for another.
__device__ __forceinline__ void make_room(LpShared& S, int n, int tid) {
  __syncthreads();
  const int count = S.n_cand;
  __syncthreads();  // read by every thread before the next round adds to it
  if (count <= kLpKeep) return;
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
  if (C > 1) {
    __syncwarp();  // each warp arrives converged (the cluster barrier is .aligned)
    cluster_arrive();
  }
  dependent_wait();
  const int token = rank == 0 && tid == 0 && A.logprob ? A.tokens[row] : -1;
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
  const float given = token >= 0 && token < V ? x[token] : NAN;
  warp_join(st);
  if (lane == 0) S.wstat[warp] = st;

  // -------------------------------------------------------- the alternatives
  if (n > 0) {
    const float t0 = bound_of_threads(S, most, n, v1 - v0, warp, lane);
    const uint32_t b0 = order_bits(t0);
    const int segs = batches > 0 ? (batches + per_seg - 1) / per_seg : 0;
    if (most >= t0) {
      for (int s = 0; s < segs; ++s) {
        if (v0 + (int64_t)s * per_seg * kLpBatch + tid >= v1) break;  // nothing of the slice is in it
        const float smax = S.seg[s][tid];
        if (smax > t0) {
          S.list[atomicAdd(&S.n_above, 1)] = (uint16_t)(s * kLpThreads + tid);
        } else if (smax >= t0) {  // from the list's end
          const int i = atomicAdd(&S.n_equal, 1);
          if (i < kLpTies) S.list[kLpList - 1 - i] = (uint16_t)(s * kLpThreads + tid);
        }
      }
    }
    __syncthreads();
    const int above = S.n_above;
    const bool scan = S.n_equal > kLpTies;  // many logits equal to t0: found by the scan below instead
    const int units = (above + (scan ? 0 : S.n_equal)) * per_seg;
    for (int u0 = 0; u0 < units; u0 += kLpUnits * kLpWarps) {
      float f[kLpUnits];
      int token[kLpUnits];
#pragma unroll
      for (int i = 0; i < kLpUnits; ++i) {
        const int u = u0 + i * kLpWarps + warp;
        token[i] = -1;
        if (u < units) {
          const int q = u / per_seg, seg = S.list[q < above ? q : kLpList - 1 - (q - above)];
          const int b = (seg / kLpThreads) * per_seg + u % per_seg;
          const int64_t v = v0 + (int64_t)b * kLpBatch + (lane >> 2) * kLpThreads + seg % kLpThreads;
          const int64_t at = 4 * v - shift + (lane & 3);
          if (v < v1 && at >= 0 && at < V) {
            token[i] = (int)at;
            f[i] = x[at];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kLpUnits; ++i) {
        const uint32_t bits = token[i] >= 0 ? order_bits(f[i]) : 0u;
        append(S, key_of(bits, token[i]), token[i] >= 0 && (scan ? bits > b0 : bits >= b0), lane);
      }
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
    st = lane < kLpWarps ? S.wstat[lane] : Stat{-FLT_MAX, 0.f, 0.f};
    warp_join(st);
  }
  const uint64_t* best = S.best;
  if (C > 1) {
    __syncwarp();
    cluster_wait();  // every CTA of the cluster is running
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
    __syncwarp();
    cluster_sync_all();
    if (rank != 0) return;
    if (n > 0) select_n_sorted(S.best, S.all, C, n, tid);
    if (warp == 0) {
      st = lane < C ? S.cstat[lane] : Stat{-FLT_MAX, 0.f, 0.f};
      warp_join(st);
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
  // stays a quarter of a batch at least.  Rows of 128256, top 5, us with 1, 2, 4,
  // 8 CTAs: 1 row 13.9, 9.9, 7.2, 5.8; 19 rows 14.1, 10.0, 9.0, 7.9; 38 rows 14.2,
  // 10.1, 10.1, 12.7; 152 rows 15.3, 15.1, 24.4, 34.8.
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
