// qk_sample.cu -- a token from each row of logits and a given random number:
// temperature, top-k, top-p, min-p.
//
// Source: DAMASCUS project overview, "[02] the pipeline", compartment 07 (the LM
// head's logits go to the sampler); the pages print no formula.
//
// With the tokens in descending order of their logits (equal ones by the lower
// token; -inf never counts), w_v = exp((x_v - max) / T) and C(n) the sum of the
// first n weights: n_k = top_k, n_p the least n with C(n) >= top_p C(n_k), n_m the
// number of w_v >= min_p; n is the least of them, and the token the first whose
// C exceeds u C(n).
//
// Every decision compares sums of up to 2^19 weights with a border, and a row of
// 10^5 tokens has 10^5 borders: sums in fp32 would choose another token in some
// percent of the rows.  Weights are therefore computed in pairs of fp32 to about
// 2^-42 (a difference without error, a table of 2^(-i / 256) and a polynomial of
// degree 4) and summed in pairs within a thread and in 64-bit integers, multiples
// of 2^-44 of the largest weight, between threads: no order changes a result.
//
// A cluster of C CTAs has a row and goes over it three times (it stays in L2):
//   1. its maximum, minimum, and whether it can be sampled from;
//   2. a histogram over (max - x) of counts and mean positions within a bin, from
//      which the bins that hold the three borders and the token follow, the sums
//      being known to 1e-5;
//   3. the exact sums of what lies before, between and behind those bins, and a
//      list of the tokens in them (candidates).
// Rank 0 sorts the candidates, adds their weights up and answers the questions in
// turn, checking for each that the border lies where it was expected.  Where it
// does not, or the candidates are too many (equal logits), it searches the order
// bit by bit instead, with an exact sum over the row at each step.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "qk_device.cuh"
#include "qk_internal.h"

namespace qk {

namespace {

constexpr int kSaThreads = 512;
constexpr int kSaWarps = kSaThreads / 32;
constexpr int kSaMaxCluster = 16;
constexpr int kBins = 4096;
constexpr int kBinsPer = kBins / kSaThreads;
constexpr int kCap = 2048;  // candidates
constexpr int kCapPer = kCap / kSaThreads;
constexpr int kWhole = 1024;  // a kept set of at most so many is listed whole
constexpr int kSegs = 5;
constexpr float kOne = 17592186044416.f;  // 2^44: the largest weight
constexpr float kSlack = 4e-5f;           // of the histogram's sums, relative

struct SaTable {
  float2 t[256];  // 2^(-i / 256) as a pair
};

struct SaArgs {
  SampleArgs a;
  float ch, cl;  // 256 log2(e) / T as a pair
  int C;
  SaTable table;
};

struct SaStat {
  unsigned long long first;  // order of the best token
  float mn;                  // least finite logit
  uint32_t finite;           // finite logits
  uint32_t bad;              // NaN or +inf among them
  uint32_t pad;
};

struct SaShared {
  uint32_t cnt[kBins], frac[kBins];  // a bin's tokens, and their positions in it in 4096ths
  unsigned long long cand[kCap];     // the candidates' places in the order
  uint8_t cls[kBins];
  float2 table[256];
  SaStat stat[kSaMaxCluster];
  unsigned long long seg_sum[kSaMaxCluster][kSegs];
  uint32_t seg_cnt[kSaMaxCluster][kSegs];
  uint32_t ncand;
  unsigned long long red64[kSaWarps];
  uint32_t red32[kSaWarps];
  float redf[kSaWarps];
  int lo[4], hi[4];  // bins of the candidates: k, p, m, token
  int found[4];
  unsigned long long s_k, s_n, s_p;
  uint32_t n_p;
};

// Ascending in the order of the tokens: by the logit from the largest, then by the token.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return (b >> 31) ? b : ~(b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key >> 31) ? key : ~key & 0x7FFFFFFFu);
}

// A sum as a pair of fp32.
struct Pair {
  float h = 0.f, l = 0.f;
  __device__ __forceinline__ void add(float wh, float wl) {
    const float s = __fadd_rn(h, wh), b = __fsub_rn(s, h);
    const float e = __fadd_rn(__fsub_rn(h, __fsub_rn(s, b)), __fsub_rn(wh, b));
    h = s;
    l = __fadd_rn(l, __fadd_rn(e, wl));
  }
  __device__ __forceinline__ unsigned long long fixed() const {
    return (unsigned long long)(__float2ll_rn(h * kOne) + __float2ll_rn(l * kOne));
  }
};

// exp((x - mx) / T) as a pair, within 2^-42; x finite.
__device__ __forceinline__ float2 weight(float x, float mx, float ch, float cl, const float2* table) {
  // d = mx - x without error
  const float d = __fsub_rn(mx, x), b = __fsub_rn(d, mx);
  const float dl = __fsub_rn(__fsub_rn(mx, __fsub_rn(d, b)), __fadd_rn(x, b));
  // t = 256 log2(e) d / T
  const float th = __fmul_rn(d, ch);
  if (!(th < 45.f * 256.f)) return make_float2(0.f, 0.f);
  const float tl = __fmaf_rn(dl, ch, __fmaf_rn(d, cl, __fmaf_rn(d, ch, -th)));
  const float r = rintf(th), f = __fsub_rn(th, r);
  const int m = (int)r;
  // u = (f + tl) ln 2 / 256, at most 2^-9.5; exp(-u) = 1 - uh + s
  constexpr double kLn = 0.69314718055994530942 / 256;
  constexpr float L = (float)kLn, Ll = (float)(kLn - (double)L);
  const float uh = __fmul_rn(f, L);
  const float ul = __fmaf_rn(tl, L, __fmaf_rn(f, Ll, __fmaf_rn(f, L, -uh)));
  const float q = __fmul_rn(__fmul_rn(uh, uh), __fmaf_rn(-uh, __fmaf_rn(-uh, 1.f / 24.f, 1.f / 6.f), 0.5f));
  const float s = __fadd_rn(__fmaf_rn(uh, ul, q), -ul);
  // 2^(-i / 256) (1 - uh + s)
  const float2 t = table[m & 255];
  const float p = __fmul_rn(t.x, uh), pl = __fmaf_rn(t.y, uh, __fmaf_rn(t.x, uh, -p));
  const float h = __fsub_rn(t.x, p), e = __fsub_rn(__fsub_rn(t.x, h), p);
  const float l = __fadd_rn(e, __fadd_rn(t.y, __fmaf_rn(t.x, s, -pl)));
  const float scale = __uint_as_float((uint32_t)(127 - (m >> 8)) << 23);
  return make_float2(__fmul_rn(h, scale), __fmul_rn(l, scale));
}

__device__ __forceinline__ unsigned long long weight_fixed(float x, float mx, const SaArgs& A, const float2* table) {
  const float2 w = weight(x, mx, A.ch, A.cl, table);
  Pair p;
  p.h = w.x;
  p.l = w.y;
  return p.fixed();
}

// Whether a weight is at least min_p: the difference of two near numbers is exact.
__device__ __forceinline__ bool at_least(float2 w, float min_p) {
  return __fadd_rn(__fsub_rn(w.x, min_p), w.y) >= 0.f;
}

template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the CTA; every thread gets it.
template <typename T>
__device__ __forceinline__ T cta_sum(T v, T* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  T s = red[0];
#pragma unroll
  for (int w = 1; w < kSaWarps; ++w) s += red[w];
  return s;
}

// What lies before this thread's value, over the CTA.
template <typename T>
__device__ __forceinline__ T cta_before(T v, T* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) red[warp] = x;
  __syncthreads();
  T before = 0;
  for (int w = 0; w < warp; ++w) before += red[w];
  return before + (x - v);
}

// Calls f(logit, token) for every finite logit of chunks c0 .. c1 - 1 of a row; a
// chunk is 16 aligned bytes, the first has `pad` values before the row.
template <typename F>
__device__ __forceinline__ void each_logit(const float* row, int V, int pad, int c0, int c1, F f) {
  const int last = (V + pad + 3) / 4 - 1;
  constexpr int kFlight = 4;
  for (int c = c0 + (int)threadIdx.x; c < c1; c += kFlight * kSaThreads) {
    float4 x[kFlight];
#pragma unroll
    for (int b = 0; b < kFlight; ++b) {
      const int k = c + b * kSaThreads;
      x[b] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (k < c1) {
        if (k > 0 && k < last) {
          x[b] = __ldg(reinterpret_cast<const float4*>(row - pad) + k);
        } else {  // the row's ends
          const int v = 4 * k - pad;
          if (v >= 0 && v < V) x[b].x = __ldg(row + v);
          if (v + 1 >= 0 && v + 1 < V) x[b].y = __ldg(row + v + 1);
          if (v + 2 >= 0 && v + 2 < V) x[b].z = __ldg(row + v + 2);
          if (v + 3 >= 0 && v + 3 < V) x[b].w = __ldg(row + v + 3);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < kFlight; ++b) {
      const int v = 4 * (c + b * kSaThreads) - pad;
      const float y[4] = {x[b].x, x[b].y, x[b].z, x[b].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (y[e] != -INFINITY) f(__fadd_rn(y[e], 0.f), v + e);  // -0 is 0
    }
  }
}

struct Sums {
  unsigned long long w;
  uint32_t n;
};

// The exact sum over the tokens up to `order`, by one CTA.
__device__ __noinline__ Sums sums_upto(const SaArgs& A, SaShared& S, const float* row, int pad, float mx,
                                       unsigned long long order) {
  Pair sum;
  uint32_t n = 0;
  each_logit(row, A.a.V, pad, 0, (A.a.V + pad + 3) / 4, [&](float x, int v) {
    if ((((unsigned long long)key_of(x) << 32) | (uint32_t)v) <= order) {
      const float2 w = weight(x, mx, A.ch, A.cl, S.table);
      sum.add(w.x, w.y);
      ++n;
    }
  });
  Sums r;
  r.w = cta_sum(sum.fixed(), S.red64);
  r.n = cta_sum(n, S.red32);
  return r;
}

// The first token in the order at which done(sums up to it) holds; it holds for
// the last.  The key bit by bit, then the token.
template <typename F>
__device__ __forceinline__ unsigned long long first_where(const SaArgs& A, SaShared& S, const float* row, int pad,
                                                          float mx, Sums& at, F done) {
  uint32_t lo = 0u, hi = 0xFFFFFFFFu;
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (done(sums_upto(A, S, row, pad, mx, ((unsigned long long)mid << 32) | 0xFFFFFFFFull)))
      hi = mid;
    else
      lo = mid + 1;
  }
  const unsigned long long key = (unsigned long long)lo << 32;
  lo = 0u;
  hi = (uint32_t)A.a.V - 1u;
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (done(sums_upto(A, S, row, pad, mx, key | mid)))
      hi = mid;
    else
      lo = mid + 1;
  }
  at = sums_upto(A, S, row, pad, mx, key | lo);
  return key | lo;
}

// The whole answer by searches; one CTA.
__device__ __noinline__ void sample_slowly(const SaArgs& A, SaShared& S, const float* row, int pad, float mx,
                                           uint32_t finite, float u, int64_t m) {
  Sums all = sums_upto(A, S, row, pad, mx, ~0ull), at;
  uint32_t n = finite;
  unsigned long long s_n = all.w;
  if (A.a.top_k > 0 && (uint32_t)A.a.top_k < finite) {
    const uint32_t k = (uint32_t)A.a.top_k;
    first_where(A, S, row, pad, mx, at, [&](const Sums& s) { return s.n >= k; });
    n = at.n;
    s_n = at.w;
  }
  if (A.a.top_p < 1.f) {
    const double t = (double)A.a.top_p * (double)s_n;
    first_where(A, S, row, pad, mx, at, [&](const Sums& s) { return s.n > 0 && (double)s.w >= t; });
    if (at.n < n) {
      n = at.n;
      s_n = at.w;
    }
  }
  if (A.a.min_p > 0.f) {
    uint32_t c = 0;
    each_logit(row, A.a.V, pad, 0, (A.a.V + pad + 3) / 4,
               [&](float x, int) { c += at_least(weight(x, mx, A.ch, A.cl, S.table), A.a.min_p) ? 1u : 0u; });
    c = cta_sum(c, S.red32);
    if (c < n) {
      first_where(A, S, row, pad, mx, at, [&](const Sums& s) { return s.n >= c; });
      n = at.n;
      s_n = at.w;
    }
  }
  const double t = (double)u * (double)s_n;
  const unsigned long long order = first_where(A, S, row, pad, mx, at, [&](const Sums& s) { return (double)s.w > t; });
  if (threadIdx.x == 0) {
    const unsigned long long w = weight_fixed(value_of((uint32_t)(order >> 32)), mx, A, S.table);
    A.a.token[m] = (int32_t)(uint32_t)order;
    if (A.a.logprob) A.a.logprob[m] = (float)log((double)w / (double)s_n);
    if (A.a.kept) A.a.kept[m] = (int32_t)n;
  }
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t atom_cluster_add(uint32_t addr, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
  return old;
}
__device__ __forceinline__ uint32_t sa_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Every thread of every CTA of the cluster arrives, its warps converged.
__device__ __forceinline__ void cluster_meet(int C) {
  if (C > 1) {
    __syncwarp();
    cluster_sync_all();
  } else {
    __syncthreads();
  }
}

// A row for each cluster of A.C CTAs along x.
__global__ void __launch_bounds__(kSaThreads, 2) sample_kernel(const __grid_constant__ SaArgs A) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SaShared& S = *reinterpret_cast<SaShared*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = A.C, rank = C > 1 ? (int)sa_rank() : 0;
  const int64_t m = blockIdx.x / (unsigned)C;
  const int V = A.a.V;
  const float* row = A.a.logits + m * V;
  const int pad = (int)((reinterpret_cast<uintptr_t>(row) >> 2) & 3u);
  const int chunks = (V + pad + 3) / 4;
  const int c0 = (int)((int64_t)rank * chunks / C), c1 = (int)((int64_t)(rank + 1) * chunks / C);
  const float T = A.a.temperature;
  for (int i = tid; i < kBins; i += kSaThreads) S.cnt[i] = S.frac[i] = 0u;
  if (tid < 256) S.table[tid] = A.table.t[tid];
  if (tid == 0) S.ncand = 0u;
  if (tid < 4) S.lo[tid] = S.hi[tid] = kBins, S.found[tid] = 0;
  dependent_wait();

  // ---- 1. the best token, the least finite logit
  {
    unsigned long long first = ~0ull;
    float mx = -INFINITY, mn = INFINITY;
    int id = 0;
    uint32_t finite = 0, bad = 0;
    each_logit(row, V, pad, c0, c1, [&](float x, int v) {
      if (x > mx) mx = x, id = v;  // a thread's tokens ascend: the first of equal ones stays
      mn = fminf(mn, x);
      bad |= !(x < INFINITY) ? 1u : 0u;
      ++finite;
    });
    if (mx > -INFINITY) first = ((unsigned long long)key_of(mx) << 32) | (uint32_t)id;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      bad |= __shfl_xor_sync(0xffffffffu, bad, o);
    }
    finite = warp_sum(finite);
    if (lane == 0) {
      S.red64[warp] = first;
      S.redf[warp] = mn;
      S.red32[warp] = (bad << 31) | finite;
    }
    __syncthreads();  // also: the histogram is clear
    cluster_meet(C);  // every CTA of the cluster is running
    if (tid < C) {
      for (int w = 0; w < kSaWarps; ++w) {
        first = w ? min(first, S.red64[w]) : S.red64[0];
        mn = w ? fminf(mn, S.redf[w]) : S.redf[0];
      }
      finite = bad = 0;
      for (int w = 0; w < kSaWarps; ++w) {
        finite += S.red32[w] & 0x7FFFFFFFu;
        bad |= S.red32[w] >> 31;
      }
      const uint32_t to = mapa_shared(smem_u32(&S.stat[rank]), (uint32_t)tid);
      st_cluster_u64(to, first);
      st_cluster_u32(to + 8, __float_as_uint(mn));
      st_cluster_u32(to + 12, finite);
      st_cluster_u32(to + 16, bad);
    }
    cluster_meet(C);
  }
  unsigned long long first = ~0ull;
  float mn = INFINITY;
  uint32_t finite = 0, bad = 0;
  for (int r = 0; r < C; ++r) {
    first = min(first, S.stat[r].first);
    mn = fminf(mn, S.stat[r].mn);
    finite += S.stat[r].finite;
    bad |= S.stat[r].bad;
  }
  if (bad || finite == 0 || T == 0.f) {  // nothing to sample from, or the best token
    if (rank == 0 && tid == 0) {
      const bool none = bad || finite == 0;
      A.a.token[m] = none ? -1 : (int32_t)(uint32_t)first;
      if (A.a.logprob) A.a.logprob[m] = none ? NAN : 0.f;
      if (A.a.kept) A.a.kept[m] = none ? 0 : 1;
    }
    return;
  }
  const float mx = value_of((uint32_t)(first >> 32));
  float u = A.a.u[m];
  u = u > 0.f ? fminf(u, 0.99999994f) : 0.f;

  // ---- 2. the histogram.  Bins beyond 31 T below the maximum are one.
  const float span = fminf(mx - mn, 31.f * T);
  const float scale = span > 1e-30f ? (float)(kBins - 1) / span : 0.f;
  auto bin_of = [&](float x, float& at) {
    at = fminf((mx - x) * scale, (float)(kBins - 1));
    return (int)at;
  };
  each_logit(row, V, pad, c0, c1, [&](float x, int) {
    float at;
    const int b = bin_of(x, at);
    atomicAdd(&S.cnt[b], 1u);
    atomicAdd(&S.frac[b], (uint32_t)((at - (float)b) * 4096.f));
  });
  if (C > 1) {
    cluster_meet(C);
    // each rank adds up a run of bins of all CTAs and gives each CTA the sums
    uint32_t n[kBins / 2 / kSaThreads], fr[kBins / 2 / kSaThreads];
    const int mine = kBins / C;
#pragma unroll
    for (int i = 0; i < kBins / 2 / kSaThreads; ++i) {
      n[i] = fr[i] = 0u;
      const int b = rank * mine + tid + i * kSaThreads;
      if (tid + i * kSaThreads < mine)
        for (int r = 0; r < C; ++r) {
          n[i] += ld_cluster_u32(mapa_shared(smem_u32(&S.cnt[b]), (uint32_t)r));
          fr[i] += ld_cluster_u32(mapa_shared(smem_u32(&S.frac[b]), (uint32_t)r));
        }
    }
    // a bin is read by its own rank alone, so it may be overwritten at once
#pragma unroll
    for (int i = 0; i < kBins / 2 / kSaThreads; ++i) {
      const int b = rank * mine + tid + i * kSaThreads;
      if (tid + i * kSaThreads < mine)
        for (int r = 0; r < C; ++r) {
          st_cluster_u32(mapa_shared(smem_u32(&S.cnt[b]), (uint32_t)r), n[i]);
          st_cluster_u32(mapa_shared(smem_u32(&S.frac[b]), (uint32_t)r), fr[i]);
        }
    }
  }
  cluster_meet(C);

  // The bins where the borders are: this thread's are kBinsPer consecutive ones.
  const bool with_k = A.a.top_k > 0 && (uint32_t)A.a.top_k < finite;
  const bool with_p = A.a.top_p < 1.f, with_m = A.a.min_p > 0.f;
  const float per_bin = scale > 0.f ? 1.44269504f / (T * scale) : 0.f;  // octaves
  uint32_t n0[kBinsPer + 1];
  unsigned long long f0[kBinsPer + 1];  // counts and sums before each bin
  {
    uint32_t cn = 0;
    unsigned long long cf = 0;
#pragma unroll
    for (int i = 0; i < kBinsPer; ++i) {
      const int b = tid * kBinsPer + i;
      const uint32_t k = S.cnt[b];
      n0[i] = cn;
      f0[i] = cf;
      cn += k;
      if (k)
        cf += (unsigned long long)__float2ll_rn(kOne * (float)k *
                                                exp2f(-per_bin * ((float)b + (float)S.frac[b] / (4096.f * (float)k))));
    }
    const uint32_t bn = cta_before(cn, S.red32);
    const unsigned long long bf = cta_before(cf, S.red64);
#pragma unroll
    for (int i = 0; i < kBinsPer; ++i) n0[i] += bn, f0[i] += bf;
    n0[kBinsPer] = bn + cn;
    f0[kBinsPer] = bf + cf;
  }
  // Sum and count up to and with bin b, which its thread tells all others.
  auto sum_with = [&](int b, uint32_t& count) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kBinsPer; ++i)
      if (tid * kBinsPer + i == b) S.redf[0] = (float)f0[i + 1], S.red32[0] = n0[i + 1];
    __syncthreads();
    count = S.red32[0];
    return S.redf[0];
  };
  uint32_t count;
  const float total = sum_with(kBins - 1, count);
  // The first bin whose sums reach t (the last where none does).
  auto reach = [&](float t, int* out) {
    const unsigned long long target = t > 1.f ? (unsigned long long)t : 1ull;
#pragma unroll
    for (int i = 0; i < kBinsPer; ++i)
      if (f0[i] < target && f0[i + 1] >= target) *out = tid * kBinsPer + i;
    if (tid == kSaThreads - 1 && f0[kBinsPer] < target) *out = kBins - 1;
  };
  float s_lo = total, s_hi = total;  // the kept weights, within kSlack
  uint32_t n_hi = finite;            // tokens up to the last bin that may hold the last kept one
  int b_hi = kBins - 1;
  if (with_k) {
#pragma unroll
    for (int i = 0; i < kBinsPer; ++i)
      if (n0[i] < (uint32_t)A.a.top_k && n0[i + 1] >= (uint32_t)A.a.top_k) S.lo[0] = S.hi[0] = tid * kBinsPer + i;
    __syncthreads();
    b_hi = S.hi[0];
    s_hi = sum_with(b_hi, n_hi);
    s_lo = b_hi > 0 ? sum_with(b_hi - 1, count) : 0.f;
  }
  if (with_p) {
    const float slack = kSlack * s_hi;
    reach(A.a.top_p * s_lo - slack, &S.lo[1]);
    reach(A.a.top_p * s_hi + slack, &S.hi[1]);
    __syncthreads();
    const int b = S.hi[1];
    const float with = sum_with(b, count);
    s_lo *= A.a.top_p;
    if (b < b_hi) {
      b_hi = b;
      s_hi = with;
      n_hi = count;
    }
  }
  if (with_m) {
    const int b = (int)fminf(-logf(A.a.min_p) * T * scale, (float)(kBins - 1));
    const int b1 = min(kBins - 1, b + 1);
    if (tid == 0) S.lo[2] = max(0, b - 1), S.hi[2] = b1;
    s_lo = fminf(s_lo, b >= 2 ? sum_with(b - 2, count) : 0.f);
    const float with = sum_with(b1, count);
    if (b1 < b_hi) {
      b_hi = b1;
      s_hi = with;
      n_hi = count;
    }
  }
  if (n_hi <= kWhole) {
    if (tid == 0) S.lo[3] = 0, S.hi[3] = b_hi;
  } else {
    const float slack = kSlack * total;
    reach(u * s_lo - slack, &S.lo[3]);
    reach(u * s_hi + slack, &S.hi[3]);
  }
  __syncthreads();
  // Classes of the bins: 255 for the candidates', else how many of the ranges end before.
  uint32_t listed = 0;
#pragma unroll
  for (int i = 0; i < kBinsPer; ++i) {
    const int b = tid * kBinsPer + i;
    int seg = 0;
    bool in = false;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      in = in || (b >= S.lo[r] && b <= S.hi[r]);
      seg += S.hi[r] < b ? 1 : 0;
    }
    S.cls[b] = in ? 255 : (uint8_t)seg;
    if (in) listed += n0[i + 1] - n0[i];
  }
  listed = cta_sum(listed, S.red32);
  int last = 0;  // the last bin that matters
  const bool all = !with_k && (with_p || !with_m);
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (S.hi[r] < kBins) last = max(last, S.hi[r]);
  if (all) last = kBins - 1;
  const bool fits = listed <= kCap;

  // ---- 3. exact sums, candidates
  if (fits) {
    Pair sum[kSegs];
    uint32_t n[kSegs] = {0u, 0u, 0u, 0u, 0u};
    const uint32_t cand0 = mapa_shared(smem_u32(&S.cand[0]), 0), count0 = mapa_shared(smem_u32(&S.ncand), 0);
    each_logit(row, V, pad, c0, c1, [&](float x, int v) {
      float at;
      const int b = bin_of(x, at);
      if (b > last) return;
      const int cls = S.cls[b];
      if (cls == 255) {
        const uint32_t i = atom_cluster_add(count0, 1u);
        if (i < kCap) st_cluster_u64(cand0 + 8 * i, ((unsigned long long)key_of(x) << 32) | (uint32_t)v);
      } else {
        const float2 w = weight(x, mx, A.ch, A.cl, S.table);
#pragma unroll
        for (int s = 0; s < kSegs; ++s)
          if (cls == s) sum[s].add(w.x, w.y), ++n[s];
      }
    });
#pragma unroll
    for (int s = 0; s < kSegs; ++s) {
      const unsigned long long w = cta_sum(sum[s].fixed(), S.red64);
      const uint32_t k = cta_sum(n[s], S.red32);
      if (tid == 0) {
        st_cluster_u64(mapa_shared(smem_u32(&S.seg_sum[rank][s]), 0), w);
        st_cluster_u32(mapa_shared(smem_u32(&S.seg_cnt[rank][s]), 0), k);
      }
    }
  }
  cluster_meet(C);
  if (rank != 0) return;

  // ---- rank 0: the candidates in order, and the answers
  bool done = false;
  if (fits) {
    const int n = (int)listed;
    int size = 32;
    while (size < n) size *= 2;
    for (int i = n + tid; i < size; i += kSaThreads) S.cand[i] = ~0ull;
    __syncthreads();
    for (int k = 2; k <= size; k *= 2)
      for (int j = k / 2; j > 0; j /= 2) {
        for (int i = tid; i < size; i += kSaThreads) {
          const int o = i ^ j;
          if (o > i) {
            const unsigned long long a = S.cand[i], b = S.cand[o];
            if ((a > b) == ((i & k) == 0)) S.cand[i] = b, S.cand[o] = a;
          }
        }
        __syncthreads();
      }
    unsigned long long base_w[kSegs];
    uint32_t base_n[kSegs];
#pragma unroll
    for (int s = 0; s < kSegs; ++s) {
      base_w[s] = s ? base_w[s - 1] : 0ull;
      base_n[s] = s ? base_n[s - 1] : 0u;
      for (int r = 0; r < C; ++r) {
        base_w[s] += S.seg_sum[r][s];
        base_n[s] += S.seg_cnt[r][s];
      }
    }
    auto seg_of = [&](int b) {
      int seg = 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) seg += S.hi[r] < b ? 1 : 0;
      return seg;
    };
    // this thread's candidates: kCapPer consecutive ones
    unsigned long long w[kCapPer], upto[kCapPer];
    uint32_t place[kCapPer];
    unsigned long long own = 0;
#pragma unroll
    for (int i = 0; i < kCapPer; ++i) {
      const int j = tid * kCapPer + i;
      w[i] = j < n ? weight_fixed(value_of((uint32_t)(S.cand[j] >> 32)), mx, A, S.table) : 0ull;
      own += w[i];
      upto[i] = own;
    }
    const unsigned long long before = cta_before(own, S.red64);
    const unsigned long long listed_w = cta_sum(own, S.red64);
#pragma unroll
    for (int i = 0; i < kCapPer; ++i) {
      const int j = tid * kCapPer + i;
      place[i] = 0;
      if (j < n) {
        float at;
        const int seg = seg_of(bin_of(value_of((uint32_t)(S.cand[j] >> 32)), at));
        unsigned long long bw = 0;
        uint32_t bn = 0;
#pragma unroll
        for (int s = 0; s < kSegs; ++s)
          if (s == seg) bw = base_w[s], bn = base_n[s];
        upto[i] += before + bw;
        place[i] = bn + (uint32_t)j + 1u;
      }
    }
    uint32_t n_keep = finite;
    unsigned long long s_keep = base_w[kSegs - 1] + listed_w;  // of all, where `all`
    bool ok = true;
    if (with_k) {
#pragma unroll
      for (int i = 0; i < kCapPer; ++i)
        if (place[i] == (uint32_t)A.a.top_k) S.s_k = upto[i], S.found[0] = 1;
      __syncthreads();
      ok = S.found[0] != 0;
      n_keep = (uint32_t)A.a.top_k;
      s_keep = S.s_k;
    }
    if (with_p && ok) {
      const double t = (double)A.a.top_p * (double)s_keep;
#pragma unroll
      for (int i = 0; i < kCapPer; ++i)
        if (place[i] > 0 && (double)upto[i] >= t && (place[i] == 1 || (double)(upto[i] - w[i]) < t))
          S.n_p = place[i], S.s_p = upto[i], S.found[1] = 1;
      __syncthreads();
      ok = S.found[1] != 0;
      if (S.n_p < n_keep) n_keep = S.n_p, s_keep = S.s_p;
    }
    if (with_m && ok) {
      // those before the range in the bins are all large enough
      uint32_t c = 0;
      unsigned long long cw = 0;
#pragma unroll
      for (int i = 0; i < kCapPer; ++i)
        if (place[i] > 0 && at_least(weight(value_of((uint32_t)(S.cand[tid * kCapPer + i] >> 32)), mx, A.ch, A.cl, S.table),
                                     A.a.min_p))
          ++c, cw += w[i];
      c = cta_sum(c, S.red32);
      cw = cta_sum(cw, S.red64);
      const int seg = seg_of(S.lo[2]);
#pragma unroll
      for (int s = 0; s < kSegs; ++s)
        if (s == seg) c += base_n[s], cw += base_w[s];
      if (c < n_keep) n_keep = c, s_keep = cw;
    }
    if (ok) {
      const double t = (double)u * (double)s_keep;
#pragma unroll
      for (int i = 0; i < kCapPer; ++i)
        if (place[i] > 0 && place[i] <= n_keep && (double)upto[i] > t && (double)(upto[i] - w[i]) <= t) {
          A.a.token[m] = (int32_t)(uint32_t)S.cand[tid * kCapPer + i];
          if (A.a.logprob) A.a.logprob[m] = (float)log((double)w[i] / (double)s_keep);
          if (A.a.kept) A.a.kept[m] = (int32_t)n_keep;
          S.found[3] = 1;
        }
      __syncthreads();
      done = S.found[3] != 0;
    }
  }
  if (!done) sample_slowly(A, S, row, pad, mx, finite, u, m);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s) {
  static PerDeviceFlag attr_set;
  const int dev = current_device();
  if (!attr_set.done(dev)) {
    cudaError_t e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SaShared));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_set.mark(dev);
  }
  SaArgs A;
  A.a = a;
  const double c = a.temperature > 0.f ? 256.0 * 1.4426950408889634 / (double)a.temperature : 0.0;
  A.ch = (float)c;
  A.cl = (float)(c - (double)A.ch);
  static const SaTable table = [] {
    SaTable t;
    for (int i = 0; i < 256; ++i) {
      const double x = std::exp2(-i / 256.0);
      t.t[i].x = (float)x;
      t.t[i].y = (float)(x - (double)t.t[i].x);
    }
    return t;
  }();
  A.table = table;
  // CTAs for two on every SM at most, with a few thousand logits each at least.
  int C = 1;
  while (C < kSaMaxCluster && a.M * 2 * C <= 2 * (int64_t)device_sms() && a.V >= 2048 * 2 * C) C *= 2;
  A.C = C;
  return launch_dependent(sample_kernel, dim3((unsigned)(a.M * C)), kSaThreads, sizeof(SaShared), (unsigned)C, s, A);
}

}  // namespace qk
