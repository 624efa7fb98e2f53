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
// percent of the rows.  Weights are therefore computed in pairs of fp32 to 2^-36 of
// themselves (a difference without error, a table of 2^(-i / 2048) and two powers) and summed in pairs within a thread and in 64-bit integers, multiples
// of 2^-44 of the largest weight, between threads: no order changes a result.
//
// A cluster of C CTAs has a row and goes over it two or three times (it stays in L2;
// kept in shared memory it was no faster):
//   1. its maximum and minimum, and whether it can be sampled from;
//   2. where top_k (up to 512) or min_p alone bounds what is kept, a list of the tokens
//      above a cut: the least of the CTAs' top_k / C-th largest of their threads' (or
//      warps') maxima, so that top_k tokens lie above it, and few more, or min_p's
//      border with a margin.  They are the candidates, and nothing else is needed.
//      Otherwise, or where they are many, a histogram over (max - x) of counts and
//      mean positions within a bin, from which the bins that hold the borders and
//      the token follow, the sums being known to 1e-5;
//   3. with the histogram, the exact sums of what lies before, between and behind
//      those bins, and a list of the tokens in them (candidates).
// Rank 0 sorts the candidates, adds their weights up and answers the questions in
// turn, checking for each that the border lies where it was expected.  Where it
// does not, or the candidates are too many (equal logits), it searches the order
// bit by bit instead, with an exact sum over the row at each step.
//
// Bound by latency for one row (9.3 us for 128256 logits with top_k 40: two passes of
// 1 us, two cluster barriers, then a dozen short steps of one CTA whose code is
// fetched once), and by instructions where all weights count: 512 rows of 128256
// without bounds 294 us, HBM 27 % (the weights are 53 of them: 21 packed instructions for
// two, as the table of 2048 spares a polynomial in pairs; with one of 256 it took 33 more.
// Sums that lose nothing are 8 of them).  One row with top_p 0.9 20.4 us, one without bounds
// 18.1, the largest logit of one (temperature 0) 4.3 and of 512 rows 83.
//
// A row that is searched (equal logits by the thousand) takes up to 8 ms at 128256 logits and
// 34 at 524288: up to 32 + 20 passes by one CTA for each border.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstddef>

#include "qk_device.cuh"
#include "qk_internal.h"
#include "qk_packed.cuh"

namespace qk {

namespace {

constexpr int kSaThreads = 512;
constexpr int kSaWarps = kSaThreads / 32;
constexpr int kSaMaxCluster = 16;
constexpr int kBins = 4096;
constexpr int kBinsPer = kBins / kSaThreads;
constexpr int kCap = 2048;  // candidates
constexpr int kCapPer = kCap / kSaThreads;
constexpr int kWhole = kSaThreads;  // a kept set of at most so many is listed whole
constexpr int kSegs = 5;
constexpr int kNone = kSegs, kListed = kSegs + 1;  // classes of logits of no account, and of candidates
constexpr float kOne = 17592186044416.f;  // 2^44: the largest weight
constexpr float kMagic = 12582912.f;      // 1.5 2^23: adding it rounds to an integer in the low bits
constexpr float kSlack = 3e-5f;           // of the histogram's sums, relative: twice what they may be off
// The histogram ends this many T below the maximum, where weights are 2^-45 of the
// largest; with a top_k, whose last token may lie anywhere, where they are 0 in
// every sum (the bins are wider then: 2^-16 of a bin's weight is lost).
constexpr float kSpan = 31.f, kSpanK = 83.f;
// Bins further than this many T below the maximum go without mean positions: of
// tokens of weight w that hold the whole sum, an error of a bin's 12th root each
// leaves sqrt(w) of one, 1.5e-5 of the sum at 10 T, and at 14 T of the wider bins.
constexpr float kMeans = 10.f, kMeansK = 14.f;

constexpr int kTable = 2048;     // 2^(-i / kTable)
constexpr int kFine = 64;        // it is the product of 2^(-i / 32) and 2^(-j / kTable), j < kFine
struct SaFactors {
  float2 coarse[kTable / kFine], fine[kFine];  // as pairs
};
struct SaTable {
  float h[kTable], l[kTable];  // as a pair
};

struct SaArgs {
  SampleArgs a;
  float ch, cl;  // kTable log2(e) / T as a pair
  int C;
  SaFactors factors;
};

struct SaStat {
  float mx;         // largest logit; NaN where one is
  float mn;         // least finite logit
  float cut;        // the top_k / C-th largest of the threads' maxima
  uint32_t finite;  // logits but -inf
};

constexpr int kRing = 4;  // chunks of a thread in flight

// What takes turns in the same place.
union SaFirst {
  struct {  // histogram: a bin's tokens, and their positions in it in 4096ths; later what lies before it
    uint32_t cnt[kBins], frac[kBins];
  };
  float4 ring[kRing][kSaThreads];  // sums: the logits on their way
  struct {                         // answers: each candidate's weight and C
    unsigned long long w[kCap], upto[kCap];
  };
};
union SaSecond {
  float4 ring[kRing][kSaThreads];  // until the sums
  float maxima[kSaThreads];        // the threads'
  float2 acc[kSegs + 2][kSaThreads];  // sums of weights; those of kNone and kListed are not used
  struct {                         // answers: the candidates in order, their places; bit 31 is min_p's
    unsigned long long sorted[kCap];
    uint32_t place[kCap];
  };
};

struct alignas(16) SaShared {
  SaFirst first;
  SaSecond second;
  unsigned long long cand[kCap];  // the candidates' places in the order
  alignas(8) uint8_t cls[kBins];
  SaTable table;
  alignas(16) SaStat stat[kSaMaxCluster];
  unsigned long long seg_sum[kSaMaxCluster][kSegs];
  unsigned long long red64[kSegs][kSaWarps];
  unsigned long long base[kSegs];  // sums of the classes up to each
  unsigned long long s_k, s_p;
  uint32_t red32[kSaWarps];
  float redf[3][kSaWarps];
  uint32_t base_cnt[kSegs];  // tokens of the classes up to each
  int found[4];
  uint32_t ncand, n_p, best, included, total, listed;
  uint32_t listed_by[kSaMaxCluster];
};
static_assert(sizeof(SaShared) % 16 == 0 && kBinsPer == 8, "16-byte accesses");

// Ascending in the order of the tokens: by the logit from the largest, then by the token.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.f));  // -0 is 0
  return (b >> 31) ? b : ~(b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key >> 31) ? key : ~key & 0x7FFFFFFFu);
}
__device__ __forceinline__ float value_of(unsigned long long order) { return value_of((uint32_t)(order >> 32)); }

// A pair of fp32 in multiples of 1 / kOne.
__device__ __forceinline__ unsigned long long fixed(float h, float l) {
  return (unsigned long long)(__float2ll_rn(h * kOne) + __float2ll_rn(l * kOne));
}

// A sum of weights as a pair of fp32, and 1: as no weight is larger than that, what an
// addition rounds off is the weight less what was added.  What h has rounded off so far
// goes in with the next weight, so that l stays within 2^-23 h, however many equal weights
// round the same way; an addition loses 3 2^-48 h at most.  (With l added up beside h its
// own roundings grow with it: 2^-25 of the sum for 128256 equal weights of 2^-24.6.)
struct Sum {
  float h = 1.f, l = 0.f;
  __device__ __forceinline__ void add(float2 w) {
    const float y = __fadd_rn(l, w.y), x = __fadd_rn(w.x, y), r = __fsub_rn(y, __fsub_rn(x, w.x));
    const float s = __fadd_rn(h, x), e = __fsub_rn(x, __fsub_rn(s, h));
    h = s;
    l = __fadd_rn(e, r);
  }
  __device__ __forceinline__ unsigned long long value() const { return fixed(h, l) - (1ull << 44); }
};

constexpr double kPerOctave = kTable * 1.44269504088896340736;  // kTable log2(e)
constexpr float kPerOctaveH = (float)kPerOctave, kPerOctaveL = (float)(kPerOctave - (double)kPerOctaveH);
constexpr float kFar = 87.f;  // exp(-87) is 2^-125.5, of the octaves that the exponent holds

// What the weights of a row need.
struct Weigh {
  float mx, least;  // logits below `least`, whose weight is 0 in every sum, count as it
  float ch, cl;     // kTable log2(e) / T as a pair
  const SaTable* table;
};

// exp((x - mx) / T) of two finite logits, as pairs, within 2^-36.
// The table is so fine that only u's first power matters beyond fp32.
__device__ __forceinline__ void weights(const Weigh& W, float x0, float x1, float2& w0, float2& w1) {
  constexpr float kLn = (float)(0.69314718055994530942 / kTable);
  const Two minus(-1.f), mx(W.mx), ch(W.ch), x(fmaxf(x0, W.least), fmaxf(x1, W.least));
  // d + dl = mx - x without error
  const Two d = fma2(x, minus, mx);
  const Two b = fma2(mx, minus, d);
  const Two dl = fma2(add2(x, b), minus, fma2(fma2(b, minus, d), minus, mx));
  // th + tl = kTable log2(e) (mx - x) / T, th = m + f with an integer m; tl is 2^-6 at most
  const Two th = mul2(d, ch);
  const Two tl = fma2(dl, ch, fma2(d, Two(W.cl), fma2(d, ch, mul2(d, Two(-W.ch)))));
  const Two mag = add2(th, Two(kMagic));
  const Two f = add2(fma2(add2(mag, Two(-kMagic)), minus, th), tl);
  // u = (f + tl) ln 2 / kTable, at most 2^-12.4; exp(-u) - 1 = u (u / 2 - 1), u^3 / 6 is 2^-40
  const Two u = mul2(f, Two(kLn));
  const Two r = mul2(u, fma2(u, Two(0.5f), minus));
  // 2^(-i / kTable) (1 + r), i = m modulo kTable, times 2^-(m / kTable)
  float m0, m1;
  mag.get(m0, m1);
  const uint32_t b0 = __float_as_uint(m0), b1 = __float_as_uint(m1);  // m in the low bits
  const uint32_t i0 = b0 & (kTable - 1u), i1 = b1 & (kTable - 1u);
  const Two h(W.table->h[i0], W.table->h[i1]), l(W.table->l[i0], W.table->l[i1]);
  constexpr uint32_t kOctaves = 127u * kTable;
  const Two scale(__uint_as_float((127u << 23) - ((b0 & kOctaves) * ((1u << 23) / kTable))),
                  __uint_as_float((127u << 23) - ((b1 & kOctaves) * ((1u << 23) / kTable))));
  const Two low = fma2(h, r, l), sum = add2(h, low);
  mul2(sum, scale).get(w0.x, w1.x);
  mul2(fma2(fma2(h, minus, sum), minus, low), scale).get(w0.y, w1.y);
}
__device__ __forceinline__ float2 weight(const Weigh& W, float x) {
  float2 a, b;
  weights(W, x, x, a, b);
  return a;
}

// Whether a weight is at least min_p: the difference of two near numbers is exact.
__device__ __forceinline__ bool at_least(float2 w, float min_p) {
  return __fadd_rn(__fsub_rn(w.x, min_p), w.y) >= 0.f;
}

// f S rounded down to an integer, 0 <= f <= 1; `rest`: whether something was lost.
__device__ __forceinline__ unsigned long long times(unsigned long long S, float f, bool& rest) {
  const uint32_t bits = __float_as_uint(f), ex = bits >> 23;
  const uint32_t man = ex ? (bits & 0x7FFFFFu) | 0x800000u : bits & 0x7FFFFFu;
  const int sh = 150 - (int)(ex ? ex : 1u);  // f = man 2^-sh, sh 23 .. 149
  const unsigned long long lo = S * man, hi = __umul64hi(S, man);
  if (sh < 64) {
    rest = (lo << (64 - sh)) != 0;
    return (lo >> sh) | (hi << (64 - sh));
  }
  const int k = sh - 64;
  const unsigned long long r = k < 64 ? hi >> k : 0ull;
  rest = lo != 0 || (k < 64 ? (r << k) != hi : hi != 0);
  return r;
}

// (x - mx) / T less the logarithm of the kept sum, which is 1 at least: no cancellation.
__device__ __forceinline__ float share_log(float x, float mx, float T, unsigned long long sum) {
  return (x - mx) / T - log1pf((float)(sum - (1ull << 44)) * (1.f / kOne));
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

// Sum over this and the lanes before.
template <typename T>
__device__ __forceinline__ T warp_upto(T x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

// Calls f(four logits, chunk) for this thread's chunks c0 + threadIdx.x, ... below c1
// of a row.  A chunk is 16 aligned bytes; the first has `pad` values before the row.
// Where there is no logit it has -inf.  Chunks come through the thread's
// places in `ring`, kRing - 1 of them on their way.  Past its last one a thread's
// logits are -inf.
template <typename F>
__device__ __forceinline__ void each_chunk(const float* row, int V, int pad, int c0, int c1,
                                           float4 (*ring)[kSaThreads], F f) {
  const int tid = threadIdx.x;
  const int whole = (V + pad) / 4;  // chunks 1 .. whole - 1 lie within the row
  const float* at = row - pad + 4 * (int64_t)(c0 + tid);
  const uint32_t to = smem_u32(&ring[0][tid]);
  int k = c0 + tid;  // the next chunk to fetch
  auto fetch = [&](int slot) {
    if (k < c1) {
      if ((unsigned)(k - 1) < (unsigned)(whole - 1)) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + (uint32_t)(slot * kSaThreads * 16)), "l"(at)
                     : "memory");
      } else {  // the row's ends
        const int v = 4 * k - pad;
        float4 x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (v >= 0 && v < V) x.x = __ldg(row + v);
        if (v + 1 >= 0 && v + 1 < V) x.y = __ldg(row + v + 1);
        if (v + 2 >= 0 && v + 2 < V) x.z = __ldg(row + v + 2);
        if (v + 3 >= 0 && v + 3 < V) x.w = __ldg(row + v + 3);
        ring[slot][tid] = x;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    k += kSaThreads;
    at += 4 * kSaThreads;
  };
  int c = c0 + tid;
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) fetch(i);
  int slot = 0;
#pragma unroll 1
  for (; c - (tid & 31) < c1; c += kSaThreads) {  // as often for all lanes
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
    float4 x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (c < c1) x = ring[slot][tid];
    fetch((slot + kRing - 1) & (kRing - 1));
    slot = (slot + 1) & (kRing - 1);
    const float y[4] = {x.x, x.y, x.z, x.w};
    f(y, c);
    __syncwarp();  // lanes that f parted go on together
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ---------------------------------------------------------------------------
// The search, for rows whose borders the histogram does not separate
// ---------------------------------------------------------------------------
struct Sums {
  unsigned long long w;
  uint32_t n;
};

// One CTA's view of a row.
struct Row {
  const float* x;
  int V, pad;
  float mn;  // least finite logit
  Weigh weigh;
};

// The exact sum over the tokens up to `order`.
__device__ __noinline__ Sums sums_upto(SaShared& S, const Row& R, unsigned long long order) {
  Sum sum;
  uint32_t n = 0;
  each_chunk(R.x, R.V, R.pad, 0, (R.V + R.pad + 3) / 4, S.first.ring, [&](const float(&y)[4], int k) {
    const int v = 4 * k - R.pad;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (y[e] != -INFINITY && (((unsigned long long)key_of(y[e]) << 32) | (uint32_t)(v + e)) <= order) {
        sum.add(weight(R.weigh, y[e]));
        ++n;
      }
  });
  Sums r;
  r.w = cta_sum(sum.value(), S.red64[0]);
  r.n = cta_sum(n, S.red32);
  return r;
}

// The first token in the order whose sums are at least `least` (of the weights, or,
// with `count`, of the tokens); those of the last are.  The key bit by bit, then
// the token.
__device__ __noinline__ unsigned long long first_with(SaShared& S, const Row& R, bool count, unsigned long long least,
                                                      Sums& at) {
  unsigned long long key = 0;
  for (int part = 0; part < 2; ++part) {
    uint32_t lo = part ? 0u : key_of(R.weigh.mx), hi = part ? (uint32_t)R.V - 1u : key_of(R.mn);
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2;
      const Sums s = sums_upto(S, R, part ? key | mid : ((unsigned long long)mid << 32) | 0xFFFFFFFFull);
      if (s.n > 0 && (count ? (unsigned long long)s.n : s.w) >= least)
        hi = mid;
      else
        lo = mid + 1;
    }
    key = part ? key | lo : (unsigned long long)lo << 32;
  }
  at = sums_upto(S, R, key);
  return key;
}

// The whole answer; one CTA.
__device__ __noinline__ void sample_slowly(const SaArgs& A, SaShared& S, const Row& R, uint32_t finite, float u,
                                           int64_t m) {
  Sums all = sums_upto(S, R, ~0ull), at;
  uint32_t n = finite;
  unsigned long long s_n = all.w;
  bool rest;
  if (A.a.top_k > 0 && (uint32_t)A.a.top_k < finite) {
    first_with(S, R, true, (uint32_t)A.a.top_k, at);
    n = at.n;
    s_n = at.w;
  }
  if (A.a.top_p < 1.f) {
    const unsigned long long t = times(s_n, A.a.top_p, rest);
    first_with(S, R, false, t + (rest ? 1u : 0u), at);
    if (at.n < n) {
      n = at.n;
      s_n = at.w;
    }
  }
  if (A.a.min_p > 0.f) {
    uint32_t c = 0;
    each_chunk(R.x, R.V, R.pad, 0, (R.V + R.pad + 3) / 4, S.first.ring, [&](const float(&y)[4], int) {
#pragma unroll
      for (int e = 0; e < 4; ++e) c += y[e] != -INFINITY && at_least(weight(R.weigh, y[e]), A.a.min_p) ? 1u : 0u;
    });
    c = cta_sum(c, S.red32);
    if (c < n) {
      first_with(S, R, true, c, at);
      n = at.n;
      s_n = at.w;
    }
  }
  const unsigned long long order = first_with(S, R, false, times(s_n, u, rest) + 1u, at);
  if (threadIdx.x == 0) {
    A.a.token[m] = (int32_t)(uint32_t)order;
    if (A.a.logprob) A.a.logprob[m] = share_log(value_of(order), R.weigh.mx, A.a.temperature, s_n);
    if (A.a.kept) A.a.kept[m] = (int32_t)n;
  }
}

// ---------------------------------------------------------------------------
// Clusters
// ---------------------------------------------------------------------------
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint2 ld_cluster_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_v2(uint32_t addr, uint2 v) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
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

// max(a, b), NaN where one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// The bin of the histogram in which sums from the first token on reach `target`, at
// least 1: the last one with less before it.  By a warp.
__device__ __forceinline__ int reach(const uint32_t* before, uint32_t target) {
  const int lane = threadIdx.x & 31;
  int b = 0;
#pragma unroll
  for (int step = kBins / 32; step > 0; step = step == 4 ? 1 : step / 32)  // 128, 4, 1
    b += step * (__popc(__ballot_sync(0xffffffffu, (step > 1 || lane < 4) && before[b + step * lane] < target)) - 1);
  return b;
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
  float T = A.a.temperature;
  const bool with_p = A.a.top_p < 1.f, with_m = A.a.min_p > 0.f;
  if (C > 1) {
    __syncwarp();
    cluster_arrive();  // its wait is before the first write to another CTA
  }
  for (int i = tid; i < kBins / 2; i += kSaThreads)
    reinterpret_cast<uint4*>(S.first.cnt)[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = tid; i < kTable; i += kSaThreads) {
    const float2 a = A.factors.coarse[i / kFine], b = A.factors.fine[i % kFine];
    const float p = a.x * b.x, e = fmaf(a.x, b.y, fmaf(a.y, b.x, fmaf(a.x, b.x, -p)));
    const float h = __fadd_rn(p, e);
    S.table.h[i] = h;
    S.table.l[i] = __fsub_rn(e, __fsub_rn(h, p));
  }
  if (tid < 4) S.found[tid] = 0;
  if (tid == 0) S.ncand = S.listed = 0u, S.best = 0xFFFFFFFFu;
  dependent_wait();

  // ---- 1. the largest and the least finite logit
  float mx = -INFINITY, mn = INFINITY, cut = -INFINITY;
  uint32_t finite = 0;
  each_chunk(row, V, pad, c0, c1, S.second.ring, [&](const float(&y)[4], int) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool is = y[e] != -INFINITY;
      mx = max_nan(mx, y[e]);
      mn = fminf(mn, is ? y[e] : INFINITY);
      finite += is ? 1u : 0u;
    }
  });
  const bool by_k = A.a.top_k > 0 && A.a.top_k <= kSaThreads;
  const float own = mx;
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
    mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
  }
  finite = __reduce_add_sync(0xffffffffu, finite);
  if (lane == 0) {
    S.redf[0][warp] = mx;
    S.redf[1][warp] = mn;
    S.red32[warp] = finite;
  }
  // The share-th largest of this CTA's maxima: the least that fewer than `share` are
  // larger than; C CTAs' together are top_k logits at least.  Where few are asked for
  // the warps' maxima will do, which need no pass over all threads': 14.0 -> 9.7 us
  // for one row of 128256 logits with top_k 40 (3 of each of 16 CTAs' maxima).
  const int share = by_k ? (A.a.top_k + C - 1) / C : 0;
  const bool by_warps = share <= kSaWarps / 2;
  if (!by_warps) {
    __syncthreads();  // the rings are idle
    S.second.maxima[tid] = own;
    __syncthreads();
    int larger = 0;
    const float4* maxima = reinterpret_cast<const float4*>(S.second.maxima);
#pragma unroll 4
    for (int i = 0; i < kSaThreads / 4; ++i) {
      const float4 x = maxima[i];
      larger += (x.x > own) + (x.y > own) + (x.z > own) + (x.w > own);
    }
    float least = larger < share ? own : INFINITY;
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
    if (lane == 0) S.redf[2][warp] = least;
  }
  __syncthreads();  // also: the histogram is clear
  if (C > 1) {
    __syncwarp();
    cluster_wait();  // every CTA of the cluster is running
  }
  if (warp == 0) {
    const int i = lane & (kSaWarps - 1);
    mx = S.redf[0][i];
    mn = S.redf[1][i];
    if (by_warps) {
      int larger = 0;
#pragma unroll
      for (int o = 1; o < kSaWarps; ++o) larger += __shfl_xor_sync(0xffffffffu, mx, o) > mx ? 1 : 0;
      cut = larger < share ? mx : by_k ? INFINITY : -INFINITY;
    } else {
      cut = S.redf[2][i];
    }
    finite = lane < kSaWarps ? S.red32[i] : 0u;
#pragma unroll 1
    for (int o = kSaWarps / 2; o > 0; o >>= 1) {
      mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      cut = fminf(cut, __shfl_xor_sync(0xffffffffu, cut, o));
    }
    finite = __reduce_add_sync(0xffffffffu, finite);
    if (lane < C)
      st_cluster_v4(mapa_shared(smem_u32(&S.stat[rank]), (uint32_t)lane),
                    make_uint4(__float_as_uint(mx), __float_as_uint(mn), __float_as_uint(cut), finite));
  }
  cluster_meet(C);
  {
    SaStat st{-INFINITY, INFINITY, INFINITY, 0u};
    if (lane < C) st = S.stat[lane];
    mx = st.mx;
    mn = st.mn;
    cut = st.cut;
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) {
      mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      cut = fminf(cut, __shfl_xor_sync(0xffffffffu, cut, o));
    }
    finite = __reduce_add_sync(0xffffffffu, st.finite);
  }
  if (!(fabsf(mx) < INFINITY)) {  // NaN, +inf, or nothing but -inf
    if (rank == 0 && tid == 0) {
      A.a.token[m] = -1;
      if (A.a.logprob) A.a.logprob[m] = NAN;
      if (A.a.kept) A.a.kept[m] = 0;
    }
    return;
  }
  if (T == 0.f) {  // the first of the largest
    uint32_t best = 0xFFFFFFFFu;
    each_chunk(row, V, pad, c0, c1, S.second.ring, [&](const float(&y)[4], int k) {
#pragma unroll
      for (int e = 3; e >= 0; --e)
        if (y[e] == mx) best = min(best, (uint32_t)(4 * k - pad + e));
    });
    best = __reduce_min_sync(0xffffffffu, best);
    if (lane == 0)
      asm volatile("red.shared::cluster.min.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&S.best), 0)), "r"(best) : "memory");
    cluster_meet(C);
    if (rank == 0 && tid == 0) {
      A.a.token[m] = (int32_t)S.best;
      if (A.a.logprob) A.a.logprob[m] = 0.f;
      if (A.a.kept) A.a.kept[m] = 1;
    }
    return;
  }
  float u = A.a.u[m];
  u = u > 0.f ? fminf(u, 0.99999994f) : 0.f;
  // Where the next number below mx is more than 87 T away, all weights but the largest
  // are 0 in every sum; a larger T says the same.  Otherwise mx - least is between
  // 43 T and 87 T, or 2^-62 and 2^-125.5.
  float ch = A.ch, cl = A.cl;
  {
    const uint32_t bits = __float_as_uint(mx);
    const float below = mx > 0.f ? __uint_as_float(bits - 1u) : mx < 0.f ? __uint_as_float(bits + 1u) : 0.f;
    const float step = fminf(mx - below, 2.028241e31f);  // 2^104: the largest numbers'
    if (kFar * T < step) {
      T = step * (1.f / 64.f);
      ch = kPerOctaveH / T;
      cl = kPerOctaveL / T;
    }
  }
  const Weigh W{mx, __fsub_ru(mx, kFar * T), ch, cl, &S.table};

  const bool with_k = A.a.top_k > 0 && (uint32_t)A.a.top_k < finite;
  const float span = fminf(mx - mn, (with_k ? kSpanK : kSpan) * T);
  const float scale = span > 1e-30f ? (float)(kBins - 1) / span : 0.f;
  // Logits below the cut, -inf among them, are of no account.
  if (!with_k || !by_k) cut = -INFINITY;
  cut = fmaxf(cut, -3.4028235e38f);
  const float log_m = with_m ? -logf(A.a.min_p) * T : 0.f;
  if (with_m && !with_p && !with_k) cut = fmaxf(cut, mx - log_m * 1.001f - 4.f * span / (float)kBins);
  auto bin_of = [&](float x, float& at) {  // the nearest bin, and the position less it
    at = fminf(__fmul_rn(__fsub_rn(mx, x), scale), (float)(kBins - 1));
    const float mag = __fadd_rn(at, kMagic);
    at = __fsub_rn(at, __fsub_rn(mag, kMagic));
    return (int)(__float_as_uint(mag) & (uint32_t)(kBins - 1));
  };
  int lo[4] = {kBins, kBins, kBins, kBins}, hi[4] = {kBins, kBins, kBins, kBins};
  auto seg_of = [&](int b) { return (hi[0] < b) + (hi[1] < b) + (hi[2] < b) + (hi[3] < b); };
  const uint32_t cand0 = mapa_shared(smem_u32(&S.cand[0]), 0), count0 = mapa_shared(smem_u32(&S.ncand), 0);
  auto list = [&](float x, int v) {  // a candidate, to rank 0; false where there is no room
    const uint32_t j = atom_cluster_add(count0, 1u);
    if (j < kCap) st_cluster_u64(cand0 + 8 * j, ((unsigned long long)key_of(x) << 32) | (uint32_t)v);
    return j < kCap;
  };
  int n = kCap + 1;  // candidates
  const bool direct = (with_k && by_k) || (with_m && !with_p && !with_k);
  if (direct) {
    uint32_t mine = 0;
    bool room = true;
    each_chunk(row, V, pad, c0, c1, S.second.ring, [&](const float(&y)[4], int k) {
      if (fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) < cut) return;
#pragma unroll 1
      for (int e = 0; e < 4; ++e) {
        const float x = e < 2 ? (e ? y[1] : y[0]) : (e == 2 ? y[2] : y[3]);
        if (x < cut) continue;
        ++mine;
        if (room) room = list(x, 4 * k - pad + e);
      }
    });
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0 && mine) atomicAdd(&S.listed, mine);
    __syncthreads();
    if (tid < C)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&S.listed_by[rank]), (uint32_t)tid)),
                   "r"(S.listed)
                   : "memory");
    cluster_meet(C);
    n = (int)min(__reduce_add_sync(0xffffffffu, lane < C ? S.listed_by[lane] : 0u), (uint32_t)kCap + 1u);
  }
  bool k_far = false;  // the last of the top_k has the weight 0 in every sum
  const bool listed_all = n <= kCap;  // everything from the cut on
  int segs = 0;
  if (listed_all) {
    if (rank != 0) return;
    if (tid < kSegs) S.base[tid] = 0ull, S.base_cnt[tid] = 0u;
  } else {
    // ---- 2. the histogram.  Logits further below the maximum than `span` are in the last
    // bin; those that cannot be kept are left out.
    const float means = mx - (with_k ? kMeansK : kMeans) * T;
    if (rank == 0 && tid == 0) S.ncand = 0u;  // what did not fit is listed again
    each_chunk(row, V, pad, c0, c1, S.second.ring, [&](const float(&y)[4], int) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (y[e] >= cut) {
          float at;
          const int b = bin_of(y[e], at);
          atomicAdd(&S.first.cnt[b], 1u);
          if (y[e] >= means)  // (at + 1/2) 4096 + 1, 1 at least
            atomicAdd(&S.first.frac[b], __float_as_uint(__fmaf_rn(at, 4096.f, kMagic + 2049.f)) - 0x4B400000u);
        }
    });
    if (C > 1) {
      cluster_meet(C);
      // Each rank adds up a run of bins of all CTAs and gives each CTA the sums; a bin
      // is read by its own rank alone, so it may be overwritten at once.
      const int mine = kBins / 2 / C;  // pairs of bins
#pragma unroll 1
      for (int i = tid; i < 2 * mine; i += kSaThreads) {
        const uint32_t at =
            smem_u32(i < mine ? &S.first.cnt[2 * (rank * mine + i)] : &S.first.frac[2 * (rank * mine + i - mine)]);
        uint2 n = make_uint2(0u, 0u);
#pragma unroll 1
        for (int r0 = 0; r0 < C; r0 += 8) {
          uint2 x[8];
#pragma unroll
          for (int r = 0; r < 8; ++r)
            x[r] = r0 + r < C ? ld_cluster_v2(mapa_shared(at, (uint32_t)(r0 + r))) : make_uint2(0u, 0u);
#pragma unroll
          for (int r = 0; r < 8; ++r) n.x += x[r].x, n.y += x[r].y;
        }
#pragma unroll 4
        for (int r = 0; r < C; ++r) st_cluster_v2(mapa_shared(at, (uint32_t)r), n);
      }
    }
    cluster_meet(C);

    // What lies before each bin: tokens, and weights as integers, 2^31 in all, so that
    // no thread's sums differ from another's.  This thread's bins are kBinsPer
    // consecutive ones.
    const float per_bin = scale > 0.f ? 1.44269504f / (T * scale) : 0.f;  // octaves
    {
      uint4* cnt = reinterpret_cast<uint4*>(S.first.cnt) + 2 * tid;
      uint4* frac = reinterpret_cast<uint4*>(S.first.frac) + 2 * tid;
      const uint4 k0 = cnt[0], k1 = cnt[1], q0 = frac[0], q1 = frac[1];
      uint32_t k[kBinsPer] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
      uint32_t q[kBinsPer] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
      float f[kBinsPer], sum = 0.f;
      uint32_t cn = 0;
#pragma unroll
      for (int i = 0; i < kBinsPer; ++i) {
        // the middle where no positions were added
        const float kf = (float)k[i], mean = q[i] ? __fdividef((float)q[i], 4096.f * kf) - 2049.f / 4096.f : 0.f;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(f[i]) : "f"(-per_bin * ((float)(tid * kBinsPer + i) + mean)));
        f[i] *= kf;
        sum += f[i];
        cn += k[i];
      }
      const float part = warp_sum(sum);
      if (lane == 0) S.redf[0][warp] = part;
      __syncthreads();
      const float all = warp_sum(lane < kSaWarps ? S.redf[0][lane] : 0.f);
      const float per_unit = 2147000000.f / all;  // the roundings of kBins sums stay below 2^31
      uint32_t cf = 0;
#pragma unroll
      for (int i = 0; i < kBinsPer; ++i) {
        q[i] = __float2uint_rn(f[i] * per_unit);
        cf += q[i];
      }
      uint32_t xn = warp_upto(cn), xf = warp_upto(cf);
      if (lane == 31) S.red32[warp] = xn, S.redf[1][warp] = __uint_as_float(xf);
      __syncthreads();
      xn += __reduce_add_sync(0xffffffffu, lane < warp ? S.red32[lane & (kSaWarps - 1)] : 0u) - cn;
      xf += __reduce_add_sync(0xffffffffu, lane < warp ? __float_as_uint(S.redf[1][lane & (kSaWarps - 1)]) : 0u) - cf;
#pragma unroll
      for (int i = 0; i < kBinsPer; ++i) {
        const uint32_t n = k[i], w = q[i];
        k[i] = xn;
        q[i] = xf;
        xn += n;
        xf += w;
      }
      cnt[0] = make_uint4(k[0], k[1], k[2], k[3]);
      cnt[1] = make_uint4(k[4], k[5], k[6], k[7]);
      frac[0] = make_uint4(q[0], q[1], q[2], q[3]);
      frac[1] = make_uint4(q[4], q[5], q[6], q[7]);
      if (tid == kSaThreads - 1) S.included = xn, S.total = xf;
    }
    __syncthreads();
    const uint32_t included = S.included, total = S.total;
    auto sum_before = [&](int b) { return (float)(b < kBins ? S.first.frac[b] : total); };
    auto count_before = [&](int b) { return b < kBins ? S.first.cnt[b] : included; };

    // The bins where the borders are: ranges [lo, hi] for k, p, m and the token.  Every
    // warp finds them.
    // A share f of a sum S is found within 2 kSlack f (1 - f) S, as the errors of what
    // lies before it and behind it are relative to these: towards the end of a row,
    // where thousands of tokens share 1e-4 of the sum, that is a few of them.  (8 times
    // that, for single tokens' places in their bins.)
    auto range = [&](float f, float from, float to, int& first, int& last) {
      const float slack = kSlack * to * fminf(16.f * (1.f - f), 1.f) + 256.f;
      from = f * from - slack;
      to = f * to + slack;
      first = reach(S.first.frac, from > 1.f ? (uint32_t)from : 1u);
      last = reach(S.first.frac, to > 1.f ? min((uint32_t)to, total) : 1u);
      return slack;
    };
    float s_lo = (float)total, s_hi = s_lo;  // the kept weights, within kSlack
    int b_hi = kBins - 1;                    // the last bin that may hold the last kept token
    if (with_k) {
      const int b = reach(S.first.cnt, (uint32_t)A.a.top_k);
      k_far = b == kBins - 1 && span < mx - mn;
      if (!k_far) {
        lo[0] = hi[0] = b_hi = b;
        s_lo = sum_before(b);
        s_hi = sum_before(b + 1);
      }
    }
    if (with_p) {
      const float slack = range(A.a.top_p, s_lo, s_hi, lo[1], hi[1]);
      s_lo = A.a.top_p * s_lo - slack;
      if (hi[1] < b_hi) {
        b_hi = hi[1];
        s_hi = sum_before(b_hi + 1);
      }
    }
    if (with_m) {
      const int b = (int)fminf(log_m * scale, (float)(kBins - 1));
      lo[2] = max(0, b - 1);
      hi[2] = min(kBins - 1, b + 2);
      s_lo = fminf(s_lo, sum_before(lo[2]));
      if (hi[2] < b_hi) {
        b_hi = hi[2];
        s_hi = sum_before(b_hi + 1);
      }
    }
    if (count_before(b_hi + 1) <= kWhole) {
      lo[3] = 0;
      hi[3] = b_hi;
    } else {
      range(u, s_lo, s_hi, lo[3], hi[3]);
    }
    // Classes of the bins: kListed for the candidates', else how many of the ranges
    // end before.
    const bool all = (!with_k || k_far) && (with_p || !with_m);  // every weight counts
    int last = all ? kBins - 1 : -1;                  // the last bin that matters
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (hi[r] < kBins) last = max(last, hi[r]);
#pragma unroll 1
    for (int b = tid; b < kBins; b += kSaThreads) {
      bool in = false;
#pragma unroll
      for (int r = 0; r < 4; ++r) in = in || (b >= lo[r] && b <= hi[r]);
      S.cls[b] = (uint8_t)(in ? kListed : seg_of(b));
    }
    // Lane s: the tokens of class s, whose bins are those behind the s-th range to end
    // and before the first of the ranges that end later.
    uint32_t seg_cnt = 0;
    if (lane < kSegs) {
      int from = lane ? kBins : 0, to = kBins;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (lane && hi[r] < kBins && seg_of(hi[r]) < lane && seg_of(hi[r] + 1) >= lane) from = hi[r] + 1;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (hi[r] >= from) to = min(to, lo[r]);
      if (from < to && seg_of(from) == lane) seg_cnt = count_before(to) - count_before(from);
    }
    n = (int)(included - __reduce_add_sync(0xffffffffu, seg_cnt));
    segs = last < 0 ? 0 : seg_of(last) + 1;  // classes whose sums are wanted
    seg_cnt = warp_upto(seg_cnt);
    if (warp == 0 && lane < kSegs) S.base_cnt[lane] = seg_cnt;
#pragma unroll 1
    for (int s = 0; s < segs; ++s) S.second.acc[s][tid] = make_float2(1.f, 0.f);
    __syncthreads();

    // ---- 3. exact sums, candidates
    if (n <= kCap) {
      auto add = [&](int cls, float2 w) {
        const float2 a = S.second.acc[cls][tid];
        Sum p;
        p.h = a.x;
        p.l = a.y;
        p.add(w);
        S.second.acc[cls][tid] = make_float2(p.h, p.l);
      };
      each_chunk(row, V, pad, c0, c1, S.first.ring, [&](const float(&y)[4], int k) {
        int cls[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          cls[e] = kNone;
          if (y[e] >= cut) {
            float at;
            const int b = bin_of(y[e], at);
            if (b <= last) cls[e] = S.cls[b];
          }
        }
        if (max(max(cls[0], cls[1]), max(cls[2], cls[3])) == kListed) {
#pragma unroll 1
          for (int e = 0; e < 4; ++e) {
            const int c = e < 2 ? (e ? cls[1] : cls[0]) : (e == 2 ? cls[2] : cls[3]);
            const float x = e < 2 ? (e ? y[1] : y[0]) : (e == 2 ? y[2] : y[3]);
            if (c == kListed) list(x, 4 * k - pad + e);
          }
        }
        if (min(min(cls[0], cls[1]), min(cls[2], cls[3])) < kSegs) {
#pragma unroll
          for (int e = 0; e < 4; e += 2) {  // the weight of a logit that is not wanted goes to a sum that is not either
            float2 w0, w1;
            weights(W, y[e], y[e + 1], w0, w1);
            add(cls[e], w0);
            add(cls[e + 1], w1);
          }
        }
      });
#pragma unroll 1
      for (int s = 0; s < segs; ++s) {
        Sum p;
        p.h = S.second.acc[s][tid].x;
        p.l = S.second.acc[s][tid].y;
        const unsigned long long w = warp_sum(p.value());
        if (lane == 0) S.red64[s][warp] = w;
      }
      __syncthreads();
      if (tid < kSegs) {
        unsigned long long w = 0;
        if (tid < segs)
#pragma unroll 4
          for (int i = 0; i < kSaWarps; ++i) w += S.red64[tid][i];
        st_cluster_u64(mapa_shared(smem_u32(&S.seg_sum[rank][tid]), 0), w);
      }
    }
    cluster_meet(C);
    if (rank != 0) return;
    if (warp < kSegs) {
      unsigned long long w = 0;
#pragma unroll 1
      for (int i = 0; i <= warp; ++i) w += lane < C ? S.seg_sum[lane][i] : 0ull;
      w = warp_sum(w);
      if (lane == 0) S.base[warp] = w;
    }
  }

  // ---- rank 0: the candidates in order, and the answers
  bool done = false;
  if (n <= kCap && S.ncand == (uint32_t)n) {
    const unsigned long long* sorted = S.second.sorted;
    if (n <= kSaThreads) {  // each finds its place by counting; four threads for one where they are few
      const int by = n <= kSaThreads / 4 ? 4 : 1, mine = by == 4 ? tid >> 2 : tid;
      const unsigned long long own = mine < n ? S.cand[mine] : 0ull;
      int place = 0;
#pragma unroll 4
      for (int i = by == 4 ? tid & 3 : 0; i < n; i += by) place += S.cand[i] < own ? 1 : 0;
      if (by == 4) {
        place += __shfl_xor_sync(0xffffffffu, place, 1);
        place += __shfl_xor_sync(0xffffffffu, place, 2);
      }
      if (mine < n) S.second.sorted[place] = own;
    } else {
      int size = kSaThreads;
      while (size < n) size *= 2;
      for (int i = n + tid; i < size; i += kSaThreads) S.cand[i] = ~0ull;
      __syncthreads();
      for (int k = 2; k <= size; k *= 2)
        for (int j = k / 2; j > 0; j /= 2) {
          for (int i = tid; i < size / 2; i += kSaThreads) {
            const int x = 2 * i - (i & (j - 1)), y = x + j;  // pairs j apart
            const unsigned long long a = S.cand[x], b = S.cand[y];
            if ((a > b) == ((x & k) == 0)) S.cand[x] = b, S.cand[y] = a;
          }
          __syncthreads();
        }
      sorted = S.cand;
    }
    __syncthreads();
    // This thread's candidates are `per` consecutive ones.
    const int per = n <= kSaThreads ? 1 : kCapPer, j0 = tid * per, j1 = min(n, j0 + per);
    unsigned long long own = 0;
#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
      const float2 f = weight(W, value_of(sorted[j]));
      const unsigned long long w = fixed(f.x, f.y);
      S.first.w[j] = w;
      S.second.place[j] = with_m && at_least(f, A.a.min_p) ? 0x80000000u : 0u;
      own += w;
    }
    unsigned long long c = warp_upto(own);
    if (lane == 31) S.red64[0][warp] = c;
    __syncthreads();
    c += warp_sum(lane < warp ? S.red64[0][lane & (kSaWarps - 1)] : 0ull) - own;
    const unsigned long long listed = warp_sum(lane < kSaWarps ? S.red64[0][lane] : 0ull);
#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
      c += S.first.w[j];
      float at;
      const int seg = seg_of(bin_of(value_of(sorted[j]), at));
      S.first.upto[j] = S.base[seg] + c;
      S.second.place[j] |= S.base_cnt[seg] + (uint32_t)j + 1u;
    }
    __syncthreads();
    uint32_t n_keep = k_far ? (uint32_t)A.a.top_k : finite;
    unsigned long long s_keep = S.base[kSegs - 1] + listed;  // of all, where `all`
    bool ok = true, rest;
    if (with_k && !k_far) {
#pragma unroll 1
      for (int j = tid; j < n; j += kSaThreads)
        if ((S.second.place[j] & 0x7FFFFFFFu) == (uint32_t)A.a.top_k) S.s_k = S.first.upto[j], S.found[0] = 1;
      __syncthreads();
      ok = S.found[0] != 0;
      n_keep = (uint32_t)A.a.top_k;
      s_keep = S.s_k;
    }
    if (with_p && ok) {
      unsigned long long t = times(s_keep, A.a.top_p, rest);
      t += rest ? 1u : 0u;
#pragma unroll 1
      for (int j = tid; j < n; j += kSaThreads) {
        const unsigned long long to = S.first.upto[j];
        const uint32_t place = S.second.place[j] & 0x7FFFFFFFu;
        if (to >= t && (place == 1u || to - S.first.w[j] < t)) S.n_p = place, S.s_p = to, S.found[1] = 1;
      }
      __syncthreads();
      ok = S.found[1] != 0;
      if (S.n_p < n_keep) n_keep = S.n_p, s_keep = S.s_p;
    }
    if (with_m && ok) {
      // those before the range in the bins are all large enough
      uint32_t large = 0;
      unsigned long long sum = 0;
#pragma unroll 1
      for (int j = tid; j < n; j += kSaThreads)
        if (S.second.place[j] >> 31) ++large, sum += S.first.w[j];
      large = cta_sum(large, S.red32) + S.base_cnt[seg_of(lo[2])];
      sum = cta_sum(sum, S.red64[0]) + S.base[seg_of(lo[2])];
      if (large < n_keep) n_keep = large, s_keep = sum;
    }
    if (ok) {
      const unsigned long long t = times(s_keep, u, rest);
#pragma unroll 1
      for (int j = tid; j < n; j += kSaThreads) {
        const unsigned long long to = S.first.upto[j];
        if ((S.second.place[j] & 0x7FFFFFFFu) <= n_keep && to > t && to - S.first.w[j] <= t) {
          const unsigned long long order = sorted[j];
          A.a.token[m] = (int32_t)(uint32_t)order;
          if (A.a.logprob) A.a.logprob[m] = share_log(value_of(order), mx, A.a.temperature, s_keep);
          if (A.a.kept) A.a.kept[m] = (int32_t)n_keep;
          S.found[3] = 1;
        }
      }
      __syncthreads();
      done = S.found[3] != 0;
    }
  }
  if (!done) sample_slowly(A, S, Row{row, V, pad, mn, W}, finite, u, m);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s) {
  static const SaFactors factors = [] {  // made once for the process
    SaFactors t;
    auto power = [](float2& to, double x) {
      x = std::exp2(x);
      to.x = (float)x;
      to.y = (float)(x - (double)to.x);
    };
    for (int i = 0; i < kTable / kFine; ++i) power(t.coarse[i], -i * (double)kFine / kTable);
    for (int i = 0; i < kFine; ++i) power(t.fine[i], -i / (double)kTable);
    return t;
  }();
  SaArgs A;
  A.a = a;
  const double c = a.temperature > 0.f ? kPerOctave / (double)a.temperature : 0.0;
  A.ch = (float)c;
  A.cl = (float)(c - (double)A.ch);
  A.factors = factors;
  static PerDeviceFlag attr_set;
  const int dev = current_device();
  if (!attr_set.done(dev)) {
    cudaError_t e =
        cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SaShared));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_set.mark(dev);
  }
  // CTAs for each row: as many as fill two CTAs an SM, up to 8; 16 for four rows at
  // most.  Where a long row's sums are needed, which keep the SMs busy, some SMs may
  // have more.  us with 1, 2, 4, 8, 16 CTAs, 128256 logits from HBM: one row, top_k 40: 33.4, 23.8,
  // 18.5, 11.7, 11.2; 8 rows 34.2, 24.8, 19.8, 13.3, 14.5; 64 rows 45, 34, 28, 28, 51; 512 rows
  // 108, 119, 170, 195, 361.  top_p 0.9: one row 95, 57, 36, 26, 21; 8 rows 100, 60, 39, 35, 29;
  // 64 rows 144, 89, 59, 77, 126; 80 rows 146, 92, 85, 100, 152; 160 rows 164, 139, 136, 176.
  // No bounds: 200 rows 166, 141, 154; 300 rows 174, 180, 217; 512 rows 308, 302, 357; 1216
  // rows 612, 669, 814.  Greedy: one row 22, 13, 7.9, 5.4, 4.3; 64 rows 30, 19, 13, 17; 512
  // rows 83, 76, 91.
  const bool sums = a.temperature > 0.f && (a.top_k == 0 ? a.top_p < 1.f || a.min_p == 0.f : a.top_k > kSaThreads);
  const int64_t fill = (sums && a.V >= 65536 ? 5 : 4) * (int64_t)device_sms() / 2;
  int C = 1;
  while (C < kSaMaxCluster && a.M * 2 * C <= (C < 4 ? fill : C < 8 ? 2 * (int64_t)device_sms() : 64) &&
         a.V >= 2048 * 2 * C)
    C *= 2;
  A.C = C;
  return launch_dependent(sample_kernel, dim3((unsigned)(a.M * C)), kSaThreads, sizeof(SaShared), (unsigned)C, s, A);
}

}  // namespace qk
