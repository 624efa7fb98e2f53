// qk_attn_q4.cu -- grouped-query attention over a KV cache held in 4 bits, and
// the cache's rows as fp16.
//
// Source: DAMASCUS project overview, "[02] the pipeline" (a decoder layer is GQA
// with a KV cache) and "[04] one decode step"; the 4-bit cache is this library's.
//
// A row of one position and key/value head holds groups of 32 values as v = d q + m
// (q in 0 .. 15, d and m fp16): 64 bytes of quants and 16 of (d, m) for 128
// values, 80 bytes where fp16 takes 256.
//
// Few tokens (a decode step, or drafted tokens: M * H / H_kv <= 32 columns, a
// column being a query head of one token).  A warp takes 16 positions at a time
// through a ring of its own in shared memory, three more 16s on their way.
// mma.sync, whose 8-wide N side holds the columns, multiplies:
//   S^T = K Q^T (16 positions x 8 columns), a group of the dimensions at a time:
//     the sum over the groups of d (q . Q) + m (sum of Q), d applied to the fp32
//     products.  The quants are exact operands, so K is not rounded at all;
//   O^T = V^T P (dimensions x columns): fp16(d (q - 8)) P, and 8 d + m of the groups
//     through one more product, whose other rows add up the weights.  movmatrix
//     transposes 8 positions of 4 nibbles each, which are four dimensions' k pairs.
// A nibble becomes an fp16 by OR with an exponent (1024 + q, or 64 + q where it
// sits 4 bits higher); for K the offsets come off with the product of (d, m).
// Rounded to fp16: weights (against a reference 7 below the largest, so that those
// down to 2^-32 of it count), d (q - 8), and the outputs.  The 2-norm of the error is
// 2.8e-4 of the output's after 500 positions, 3.3e-4 after 65536; the output's own
// rounding is 2.1e-4 of it.  With fp16(d q + m) for K and fp16(d q) for V it was 6.0e-4
// and 7.4e-4 (0.1 and 0.6 us faster).
// Every warp keeps its own running maximum, sums and O; the warps of a CTA join
// in order through shared memory.  The CTAs of a key/value head join
//   - as a cluster of up to 16 through distributed shared memory, each writing a
//     share of the outputs; or,
//   - from 65536 positions of all heads on, through the scratch and a second kernel
//     (attn_q4_join_kernel): a GPC takes few clusters of 16, so that 8 heads' leave
//     SMs idle, while this split uses all of them (kQSplitFrom).
//
// One token, 24 heads over 8, 65536 positions (84 MB: 12.4 us at a copy's rate): 22.5 us.
// Bound by instructions at long lengths (375 for a warp's 16 positions, issued in
// 57 % of the cycles, the ends included; the DRAM is 48 % busy) and by the latency of
// a launch, or two, at short ones.
//
// More tokens: the visible rows are written as fp16(d q + m) to the caller's scratch once
// and the windowed prefill runs over them: a query tile's 128 rows would unpack each key
// again.  K and V are rounded there, and the error is 5.8e-4 of the output's.  1023 tokens
// after 7001, 24 heads over 8: 117 us, 10 of them for the rows; 104 CTAs of two query
// tiles each on 152 SMs.  (Clusters of 2, 4 and 8 that share the keys of a pair of tiles:
// 134, 118, 171.)
//
// The kernels have no waits but the cluster barriers, which every thread reaches.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "qk_attn.cuh"
#include "qk_device.cuh"
#include "qk_internal.h"

namespace qk {

namespace {

constexpr int kQMaxCluster = 16;
// Columns that read the 4-bit rows directly: four tiles of 8, whose O and scores are what the
// registers of a warp hold.  us over 8 key/value heads, 24 columns so / through fp16 rows and
// the prefill: 500 positions 9.4 / 10.0, 2000 11.7 / 11.7, 8000 20.3 / 26.3, 20000 24.4 / 55.4,
// 65536 49 / 165; 32 columns 9.9 / 10.6, 12.4 / 11.7, 21.0 / 26.4, 24.9 / 55.5, 50 / 165.  33
// to 64 take what the fp16 rows take: 10.5, 11.9, 26.5, 55.7, 165.
constexpr int kQMaxCols = 32;
constexpr int kQMaxSplit = 160;   // CTAs of a call that join through the scratch
// Positions of all key/value heads from which a call's CTAs need not be clusters.  us as
// clusters / over all SMs, one token:
//   24 heads over 8: 4096 positions 7.1 / 8.3, 8192 9.2 / 9.6, 16384 13.5 / 12.2, 32768 21.3 / 15.4,
//   131072 68 / 35; 32 over 4: 8192 7.6 / 9.8, 16384 11.7 / 11.1, 32768 19.6 / 13.8;
//   8 over 2: 16384 8.7 / 9.4, 32768 13.3 / 10.7; 8 over 1: 16384 8.8 / 10.8, 32768 13.4 / 11.7.
// More tokens cross a little earlier, at half as many positions with 32 columns:
//   15 columns of each of 8: 4096 9.8 / 9.9, 8192 13.4 / 11.8; 30 of 8: 4096 15.3 / 14.8, 8192 20.9 /
//   17.8; 32 of 4: 8192 15.9 / 15.3, 16384 21.5 / 18.4; 20 of 2: 8192 14.3 / 14.0, 16384 19.9 / 15.8;
//   32 of 1: 8192 15.1 / 16.7, 16384 20.9 / 17.1, 32768 31.8 / 19.1.
// With one or two heads the product is thus late: one token over 65535 positions of one head
// takes 22.5 us where all SMs would take 12.9.
constexpr int64_t kQSplitFrom = 8 * 8192;
constexpr int kUnit = 16;  // positions of a warp's step

// The shape of a CTA for NT tiles of 8 columns and W warps.
template <int NT, int W>
struct Q4Shape {
  static constexpr int kWarps = W;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPerSm = NT == 1 ? 16 / W : 1;  // CTAs of an SM: registers for the columns' O
  static constexpr int kCols = 8 * NT;
  static constexpr bool kSharedQ = NT > 2;
};

// 16 rows of one key/value head.
struct Q4Stage {
  uint4 k[64], v[64];  // lane l copies and reads chunks l and l + 32: group l % 4 of rows l / 4 and l / 4 + 8
  uint4 ks[16], vs[16];
};
constexpr int kStages = 4;  // 16s in flight or in use for each warp

template <int NT, int W>
struct Q4Shared {
  using Sh = Q4Shape<NT, W>;
  union {
    Q4Stage ring[kStages];
    float part[Sh::kCols * kD];  // after its last rows: the warp's O
  } warp[Sh::kWarps];
  float red[kQMaxCluster * 4 + Sh::kCols * kD];  // what the CTAs send: [rank][this CTA's share of the outputs]
  float2 stat[kQMaxCluster][Sh::kCols];    // and their (max, sum)
  float wmax[Sh::kWarps][Sh::kCols], wsum[Sh::kWarps][Sh::kCols];
  uint2 q[Sh::kSharedQ ? 8 * NT : 1][32];  // Q's fragments, where registers do not hold them
};

struct Q4Args {
  const __half* q;
  __half* out;
  const uint4 *k_q4, *v_q4;     // 4 groups of 16 bytes a row
  const uint32_t *k_dm, *v_dm;  // 4 words a row
  int H, Hkv, G, M;
  int64_t pos0, Lmax, window, sinks;
  int64_t sink_rows, gap, total;  // visible position u is u, or u + gap from sink_rows on: `total` of them
  float scale_log2e;
  int C;         // CTAs that share a key/value head: a cluster, or, with `part`, any number
  float* part;   // [H_kv][columns][C] partial O of 128, and after them their (max, sum)
};

__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

// The nibbles of a word as four pairs of fp16 (nibble i of the low half and of
// the high half) with the exponent of 2^10, 1024 + q, or, 4 bits higher, of 2^6, 64 + q.
__device__ __forceinline__ void spread(uint32_t w, uint32_t (&u)[4]) {
  const uint32_t h = w >> 8;
  u[0] = lop_and_or<0x000f000fu>(w, 0x64006400u);
  u[1] = lop_and_or<0x00f000f0u>(w, 0x54005400u);
  u[2] = lop_and_or<0x000f000fu>(h, 0x64006400u);
  u[3] = lop_and_or<0x00f000f0u>(h, 0x54005400u);
}

// The same without the offsets, exact.
__device__ __forceinline__ void unpack_pairs(uint32_t w, __half2 (&q)[4]) {
  uint32_t u[4];
  spread(w, u);
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = __hsub2(as_h2(u[i]), as_h2(i & 1 ? 0x54005400u : 0x64006400u));
}

// Transposes an 8 x 8 matrix of 16-bit values: lane 4 r + c holds row r, columns 2 c and 2 c + 1.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}
__device__ __forceinline__ void st_cluster_v2(uint32_t addr, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Up to 8 NT columns against the visible positions of one key/value head.  Rank r
// of the cluster takes visible positions [r n / C, (r + 1) n / C) in multiples of
// 16, its warps every kWarps-th 16 of them.  kMulti: more than one token, so that
// columns see different positions.
template <int NT, int W, bool kMulti>
__global__ void __launch_bounds__(Q4Shape<NT, W>::kThreads, Q4Shape<NT, W>::kPerSm)
    attn_q4_decode_kernel(const __grid_constant__ Q4Args A) {
  using Sh = Q4Shape<NT, W>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Q4Shared<NT, W>& S = *reinterpret_cast<Q4Shared<NT, W>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane >> 2, tq = lane & 3;
  const int g = blockIdx.y;
  const int rank = (int)blockIdx.x;
  const int units = (int)((A.total + kUnit - 1) / kUnit);
  const int unit1 = (int)((int64_t)(rank + 1) * units / A.C);
  int unit = (int)((int64_t)rank * units / A.C) + warp;
  const int total = (int)A.total, sink_rows = (int)A.sink_rows, gap = (int)A.gap, last_p = (int)A.pos0 + A.M - 1;
  const uint4 *kq = A.k_q4 + (int64_t)g * A.Lmax * 4 + tq, *vq = A.v_q4 + (int64_t)g * A.Lmax * 4 + tq;
  const uint4* dm = reinterpret_cast<const uint4*>(lane < 16 ? A.k_dm : A.v_dm) + (int64_t)g * A.Lmax;
  auto& ring = S.warp[warp].ring;
  __syncwarp();
  if (!A.part) cluster_arrive();  // its wait is before the first write to another CTA
  dependent_wait();

  // Rows past the last visible one are copies of it.
  auto position = [&](int u) -> int64_t {
    u = min(u, total - 1);
    return u < sink_rows ? u : u + gap;
  };
  auto fetch = [&](int at, int stage) {
    if (at < unit1) {
      Q4Stage& R = ring[stage];
      const int kl = 4 * grp + (tq ^ ((grp >> 1) & 3));
      const int64_t j0 = 4 * position(kUnit * at + grp), j1 = 4 * position(kUnit * at + grp + 8);
      copy16(&R.k[kl], kq + j0);
      copy16(&R.k[kl + 32], kq + j1);
      copy16((lane < 16 ? R.ks : R.vs) + (lane & 15), dm + position(kUnit * at + (lane & 15)));
      copy16(&R.v[lane], vq + j0);
      copy16(&R.v[lane + 32], vq + j1);
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(unit + i * Sh::kWarps, i);

  // Q: the product's k axis in step (group j, half h) is dims 32 j + 8 tq + 2 h and + 4
  // (first register), and those + 1 (second).
  uint2 qb[NT][4][2];
  // of column grp and group tq: (what takes the offsets off the product, the sum of Q) 2^-k, as high and low parts
  uint32_t kb[NT][2];
  float kup[NT][2];    // 2^k of this lane's columns
  int cpos[NT][2];    // the positions of this lane's columns
  // [column tile][2 j + h]: dims 32 (grp / 2) + 8 j + 4 (grp % 2) + 2 h (+ 1: elements 2, 3), columns 2 tq (+ 1)
  float o[NT][8][4];
  // elements 0, 1: weights times d (even grp) or m (odd) of group grp / 2; 2, 3: the columns' sums of weights
  float om[NT][4];
  float m[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int col = 8 * n + grp;
    const int token = kMulti ? col / A.G : 0;
    const int64_t row = (int64_t)token * A.H + g * A.G + (col - token * A.G);
    const uint4* qr = reinterpret_cast<const uint4*>(A.q + row * kD) + tq;
    float even[4] = {0.f, 0.f, 0.f, 0.f}, odd[4] = {0.f, 0.f, 0.f, 0.f};  // of the nibbles with the offsets 1024 and 64
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 y = col < A.M * A.G ? qr[4 * j] : make_uint4(0u, 0u, 0u, 0u);
      const uint2 b0 = make_uint2(prmt(y.x, y.z, 0x5410), prmt(y.x, y.z, 0x7632));
      const uint2 b1 = make_uint2(prmt(y.y, y.w, 0x5410), prmt(y.y, y.w, 0x7632));
      if (!Sh::kSharedQ) {
        qb[n][j][0] = b0;
        qb[n][j][1] = b1;
      } else if (warp == 0) {
        S.q[8 * n + 2 * j][lane] = b0;
        S.q[8 * n + 2 * j + 1][lane] = b1;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 a = __half22float2(as_h2(i ? b1.x : b0.x)), b = __half22float2(as_h2(i ? b1.y : b0.y));
        even[j] += a.x + a.y;
        odd[j] += b.x + b.y;
      }
    }
    // lane tq gets the sums of group tq, of its column
#pragma unroll
    for (int x = 2; x > 0; x >>= 1)
#pragma unroll
      for (int j = 0; j < x; ++j) {
        const bool up = (tq & x) != 0;
        even[j] = (up ? even[j + x] : even[j]) + __shfl_xor_sync(0xffffffffu, up ? even[j] : even[j + x], x);
        odd[j] = (up ? odd[j + x] : odd[j]) + __shfl_xor_sync(0xffffffffu, up ? odd[j] : odd[j + x], x);
      }
    const float off = -fmaf(1024.f, even[0], 64.f * odd[0]), sum = even[0] + odd[0];
    float most = fmaxf(fabsf(off), fabsf(sum));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
    const uint32_t ex = max(__float_as_uint(most) >> 23, 64u);  // the largest becomes 2^13 .. 2^14
    const float down = __uint_as_float((267u - ex) << 23), up = __uint_as_float((ex - 13u) << 23);
    const __half2 hi = __floats2half2_rn(off * down, sum * down);
    kb[n][0] = as_u32(hi);
    kb[n][1] = as_u32(__floats2half2_rn(off * down - __low2float(hi), sum * down - __high2float(hi)));
    kup[n][0] = __shfl_sync(0xffffffffu, up, 8 * tq);
    kup[n][1] = __shfl_sync(0xffffffffu, up, 8 * tq + 4);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      cpos[n][e] = (int)A.pos0 + (kMulti ? min((8 * n + 2 * tq + e) / A.G, A.M - 1) : 0);
      m[n][e] = -INFINITY;
      om[n][e] = om[n][e + 2] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
  }

  if (Sh::kSharedQ) __syncthreads();
  for (int stage = 0; unit < unit1; unit += Sh::kWarps, stage = stage + 1 == kStages ? 0 : stage + 1) {
    copy_wait<kStages - 2>();
    __syncwarp();  // the scales are other lanes' copies; and all lanes are done with the stage before
    fetch(unit + (kStages - 1) * Sh::kWarps, stage == 0 ? kStages - 1 : stage - 1);
    const Q4Stage& R = ring[stage];
    const uint4 v0 = R.v[lane], v1 = R.v[lane + 32];
    const uint32_t* sv = reinterpret_cast<const uint32_t*>(R.vs) + lane;
    const uint32_t vs0 = sv[0], vs1 = sv[32];
    const int u = kUnit * unit, rows = total - u;  // rows past them are copies
    // ---- scores of rows grp and grp + 8: the sum over the groups of d (q . Q) + m (sum of Q),
    // without a rounding of K.  The quants go to the tensor core with their offsets, a
    // group at a time; one more product of the rows' (d, m) takes those off and adds m.
    float sc[NT][4];
    {
      const uint32_t* sk = reinterpret_cast<const uint32_t*>(R.ks) + lane;
      const uint32_t dm[4] = {sk[0], sk[32], sk[0], sk[32]};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
        mma16816(sc[n], dm, kb[n][0], kb[n][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][e] *= kup[n][e & 1];
      }
      // lane l gives the address of row l % 8 of group l / 8
      uint32_t k0[4], k1[4];
      const uint32_t at = smem_u32(&R.k[4 * (lane & 7) + ((lane >> 3) ^ ((lane >> 1) & 3))]);
      ldsm_x4(at, k0);
      ldsm_x4(at + 512u, k1);
      const uint4 ks0 = R.ks[grp], ks1 = R.ks[grp + 8];
      const uint32_t dm0[4] = {ks0.x, ks0.y, ks0.z, ks0.w}, dm1[4] = {ks1.x, ks1.y, ks1.z, ks1.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t p0[4], p1[4];
        spread(k0[j], p0);
        spread(k1[j], p1);
        const float d0 = __low2float(as_h2(dm0[j])), d1 = __low2float(as_h2(dm1[j]));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float dot[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {p0[2 * h], p1[2 * h], p0[2 * h + 1], p1[2 * h + 1]};
            const uint2 b = Sh::kSharedQ ? S.q[8 * n + 2 * j + h][lane] : qb[n][j][h];
            mma16816(dot, a, b.x, b.y);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][e] = fmaf(e < 2 ? d0 : d1, dot[e], sc[n][e]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][e] *= A.scale_log2e;
    }
    // ---- hidden positions; none where every column sees all 16
    const int j0 = u + (u < sink_rows ? 0 : gap), j1 = u + kUnit - 1 + (u + kUnit - 1 < sink_rows ? 0 : gap);
    const bool whole = rows >= kUnit && (!kMulti || (j1 <= (int)A.pos0 && (j0 > last_p - A.window || j1 < A.sinks)));
    if (!whole) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // e: column e & 1, row grp + 8 (e >> 1)
          const int r = grp + 8 * (e >> 1);
          bool seen = r < rows;
          if (kMulti) {
            const int j = u + r + (u + r < sink_rows ? 0 : gap), p = cpos[n][e & 1];
            seen = seen && j <= p && (p - j < A.window || j < A.sinks);
          }
          if (!seen) sc[n][e] = -INFINITY;
        }
    }
    // ---- weights, relative to a reference that is 7 below a column's largest score
    // and moves only when that grows by more than 8: weights reach 2^15, O is
    // rescaled rarely, and fp16 keeps weights down to 2^-32 of the largest.  A column
    // that has seen nothing keeps -inf, and its weights, all 0, are relative to 0.
    // NaN, which the maximum passes over, stays.
    bool moves = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) moves = moves || fmaxf(sc[n][e], sc[n][e + 2]) > m[n][e] + 15.f;
    if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = fmaxf(sc[n][e], sc[n][e + 2]);
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
          if (t > m[n][e] + 15.f) {
            const float corr = ex2_approx(m[n][e] - (t - 7.f));
            m[n][e] = t - 7.f;
            om[n][e] *= corr;
            om[n][e + 2] *= corr;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[n][i][e] *= corr;
              o[n][i][e + 2] *= corr;
            }
          }
        }
    }
    uint32_t pb[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float ref = m[n][e & 1];
        p[e] = ex2_approx(sc[n][e] - (ref == -INFINITY ? 0.f : ref));
      }
      pb[n][0] = transpose8(pack_h2(p[0], p[1]));
      pb[n][1] = transpose8(pack_h2(p[2], p[3]));
    }
    // ---- O^T += V^T P: after transposing, this lane has group grp / 2 of the
    // dimensions and rows 2 tq, 2 tq + 1 (and those + 8)
    uint32_t dv[2], dm[2];
    bool odd = false;  // a row has a value that is not finite
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // even lanes' rows get d, odd ones m, of the pair of positions
      dm[i] = transpose8(grp + 8 * i < rows ? (i ? vs1 : vs0) : 0u);
      const uint32_t other = __shfl_xor_sync(0xffffffffu, dm[i], 4);
      dv[i] = grp & 1 ? other : dm[i];
      if (kMulti) {
        // infinity and NaN have the exponent's bits all set
        const uint32_t top = as_u32(__hmul2(__float2half2_rn(15.f), as_h2(dv[i]))), mv = grp & 1 ? dm[i] : other;
        const bool b0 = (top & 0x7C00u) == 0x7C00u || (mv & 0x7C00u) == 0x7C00u;
        const bool b1 = (top & 0x7C000000u) == 0x7C000000u || (mv & 0x7C000000u) == 0x7C000000u;
        const uint32_t keep = (b0 ? 0u : 0xFFFFu) | (b1 ? 0u : 0xFFFF0000u);
        dv[i] &= keep;
        dm[i] &= keep;
        odd = odd || b0 || b1;
      }
    }
    {
      const uint32_t a0[4] = {v0.x, v0.y, v0.z, v0.w}, a1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t p0[4], p1[4];
        spread(transpose8(a0[j]), p0);
        spread(transpose8(a1[j]), p1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 off = as_h2(i & 1 ? 0x54805480u : 0x64086408u);  // 72, 1032
          p0[i] = as_u32(__hmul2(__hsub2(as_h2(p0[i]), off), as_h2(dv[0])));
          p1[i] = as_u32(__hmul2(__hsub2(as_h2(p1[i]), off), as_h2(dv[1])));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a[4] = {p0[2 * h], p0[2 * h + 1], p1[2 * h], p1[2 * h + 1]};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(o[n][2 * j + h], a, pb[n][0], pb[n][1]);
        }
      }
      const uint32_t a[4] = {dm[0], 0x3C003C00u, dm[1], 0x3C003C00u};
#pragma unroll
      for (int n = 0; n < NT; ++n) mma16816(om[n], a, pb[n][0], pb[n][1]);
    }
    if (kMulti && __any_sync(0xffffffffu, odd)) {
      // Such a value has entered the product as 0: it is NaN for the columns that
      // see its row, and nothing for the others.
      for (int r = 0; r < kUnit && r < rows; ++r) {
        const int j = u + r + (u + r < sink_rows ? 0 : gap);
        const uint32_t w = reinterpret_cast<const uint32_t*>(R.vs)[4 * r + (grp >> 1)];
        const uint32_t top = as_u32(__hmul2(__float2half2_rn(15.f), as_h2(w)));
        if ((top & 0x7C00u) != 0x7C00u && (w & 0x7C000000u) != 0x7C000000u) continue;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int p = cpos[n][e];
            if (j <= p && (p - j < A.window || j < A.sinks)) om[n][e] = NAN;
          }
      }
    }
  }
  copy_wait<0>();
  __syncwarp();
  // What 8 d + m of their group adds to this lane's values.
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float other = __shfl_xor_sync(0xffffffffu, om[n][e], 4);
      om[n][e] = grp & 1 ? fmaf(8.f, other, om[n][e]) : fmaf(8.f, om[n][e], other);
    }
  // The warp's references and sums of weights.
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // -inf: it saw nothing.  A warp that saw NaN alone has no reference either, but
      // a NaN sum: with NaN as its reference it counts, and the column is NaN.
      if (m[n][e] == -INFINITY && om[n][e + 2] != 0.f) m[n][e] = NAN;
      if (grp == 0) {
        S.wmax[warp][8 * n + 2 * tq + e] = m[n][e];
        S.wsum[warp][8 * n + 2 * tq + e] = om[n][e + 2];
      }
    }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = 8 * n + 2 * tq + e;
      float M = -INFINITY;
      for (int w = 0; w < Sh::kWarps; ++w) M = fmaxf(M, S.wmax[w][col]);
      const float f = m[n][e] == -INFINITY ? 0.f : exp2f(m[n][e] - M);
      if (col >= A.M * A.G) continue;
      float* dst = &S.warp[warp].part[col * kD + 32 * (grp >> 1) + 4 * (grp & 1)];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4*>(dst + 8 * j) =
            make_float4(f * (o[n][2 * j][e] + om[n][e]), f * (o[n][2 * j][e + 2] + om[n][e]),
                        f * (o[n][2 * j + 1][e] + om[n][e]), f * (o[n][2 * j + 1][e + 2] + om[n][e]));
    }
  __syncthreads();
  __syncwarp();
  if (!A.part) cluster_wait();  // every CTA of the cluster is running
  // The CTA's sums, the warps in order, go to the CTA of the cluster that writes
  // them out, shares of the M G 128 outputs in runs of four, or to the scratch.
  const int cols = A.M * A.G, quads = cols * (kD / 4);
  const int share = (quads + A.C - 1) / A.C;
  for (int i = threadIdx.x; i < quads; i += Sh::kThreads) {
    float4 a = *reinterpret_cast<const float4*>(&S.warp[0].part[4 * i]);
    for (int w = 1; w < Sh::kWarps; ++w) {
      const float4 b = *reinterpret_cast<const float4*>(&S.warp[w].part[4 * i]);
      a.x += b.x;
      a.y += b.y;
      a.z += b.z;
      a.w += b.w;
    }
    if (A.part) {
      const int64_t at = ((int64_t)g * cols + i / (kD / 4)) * A.C + rank;
      reinterpret_cast<float4*>(A.part)[at * (kD / 4) + i % (kD / 4)] = a;
    } else {
      const int to = i / share;
      st_cluster_v4(mapa_shared(smem_u32(&S.red[4 * (rank * share + i - to * share)]), (uint32_t)to), a);
    }
  }
  for (int i = threadIdx.x; i < cols * (A.part ? 1 : A.C); i += Sh::kThreads) {
    const int to = i / cols, col = i - to * cols;
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < Sh::kWarps; ++w) M = fmaxf(M, S.wmax[w][col]);
    bool nan = false;
    for (int w = 0; w < Sh::kWarps; ++w) {
      const float mw = S.wmax[w][col];
      if (mw != -INFINITY) L = fmaf(exp2f(mw - M), S.wsum[w][col], L);
      nan = nan || mw != mw;
    }
    const float2 st = make_float2(nan ? NAN : M, L);
    if (A.part)
      reinterpret_cast<float2*>(A.part + (int64_t)A.Hkv * cols * A.C * kD)[((int64_t)g * cols + col) * A.C + rank] = st;
    else
      st_cluster_v2(mapa_shared(smem_u32(&S.stat[rank][col]), (uint32_t)to), st);
  }
  if (A.part) return;
  __syncwarp();
  cluster_sync_all();
  for (int i = threadIdx.x; i < share && rank * share + i < quads; i += Sh::kThreads) {
    const int at = rank * share + i, col = at / (kD / 4), d = 4 * (at % (kD / 4));
    float M = -INFINITY;
    for (int r = 0; r < A.C; ++r) M = fmaxf(M, S.stat[r][col].x);
    float L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < A.C; ++r) {
      const float2 st = S.stat[r][col];
      if (st.x == -INFINITY) continue;  // it saw nothing
      const float f = exp2f(st.x - M);
      const float4 b = *reinterpret_cast<const float4*>(&S.red[4 * (r * share + i)]);
      L = fmaf(f, st.y, L);
      a.x = fmaf(f, b.x, a.x);
      a.y = fmaf(f, b.y, a.y);
      a.z = fmaf(f, b.z, a.z);
      a.w = fmaf(f, b.w, a.w);
    }
    const float inv = 1.0f / L;
    const int token = kMulti ? col / A.G : 0;
    __half* dst = A.out + ((int64_t)token * A.H + g * A.G + (col - token * A.G)) * kD + d;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_h2(within_half(a.x * inv), within_half(a.y * inv)),
                                                pack_h2(within_half(a.z * inv), within_half(a.w * inv)));
  }
}

// One column of one key/value head from its C partial results, in order.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(32 * kJoinWarps) attn_q4_join_kernel(const __grid_constant__ Q4Args A) {
  __shared__ float4 sums[kJoinWarps][32];
  __shared__ float totals[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cols = A.M * A.G, g = blockIdx.x / cols, col = blockIdx.x - g * cols;
  const float4* o = reinterpret_cast<const float4*>(A.part) + (int64_t)blockIdx.x * A.C * (kD / 4) + lane;
  const float2* st =
      reinterpret_cast<const float2*>(A.part + (int64_t)A.Hkv * cols * A.C * kD) + (int64_t)blockIdx.x * A.C;
  dependent_wait();
  float M = -INFINITY;
  for (int r = lane; r < A.C; r += 32) M = fmaxf(M, st[r].x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  float L = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int r = warp; r < A.C; r += kJoinWarps) {
    const float2 s = st[r];
    const float4 b = o[(int64_t)r * (kD / 4)];
    const float f = s.x == -INFINITY ? 0.f : exp2f(s.x - M);  // -inf: it saw nothing, and has zeros
    L = fmaf(f, s.y, L);
    a.x = fmaf(f, b.x, a.x);
    a.y = fmaf(f, b.y, a.y);
    a.z = fmaf(f, b.z, a.z);
    a.w = fmaf(f, b.w, a.w);
  }
  sums[warp][lane] = a;
  if (lane == 0) totals[warp] = L;
  __syncthreads();
  if (warp > 0) return;
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) {
    const float4 b = sums[w][lane];
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
    L += totals[w];
  }
  const float inv = 1.0f / L;
  const int token = col / A.G;
  __half* dst = A.out + ((int64_t)token * A.H + g * A.G + (col - token * A.G)) * kD + 4 * lane;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_h2(within_half(a.x * inv), within_half(a.y * inv)),
                                              pack_h2(within_half(a.z * inv), within_half(a.w * inv)));
}

// How many clusters of `c` CTAs of the kernel the device runs at once (a cluster
// lies within one GPC).  Asked once per device and size; attributes are set before.
template <int NT, int W, bool kMulti>
int max_clusters(int c) {
  static std::atomic<int> known[kMaxDevices][kQMaxCluster + 1];
  const int dev = current_device();
  if (dev < 0) return 0;
  int n = known[dev][c].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c);
    cfg.blockDim = dim3(Q4Shape<NT, W>::kThreads);
    cfg.dynamicSmemBytes = sizeof(Q4Shared<NT, W>);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)c;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, attn_q4_decode_kernel<NT, W, kMulti>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    n = n > 0 ? n : -1;  // -1: none
    known[dev][c].store(n, std::memory_order_relaxed);
  }
  return n;
}

// CTAs for each key/value head where they need not be a cluster: one for every SM.
int split_ctas(int64_t units, int Hkv, int per_sm) {
  const int64_t c = std::max(1, std::min(per_sm * device_sms(), kQMaxSplit) / Hkv);
  return (int)std::min<int64_t>(c, units);
}

template <int NT, int W, bool kMulti>
cudaError_t launch_decode(Q4Args A, cudaStream_t s) {
  static_assert(sizeof(Q4Shared<NT, W>) <= 227 * 1024, "shared memory of a CTA");
  static PerDeviceFlag attr_set;
  const int dev = current_device();
  if (!attr_set.done(dev)) {
    cudaError_t e = cudaFuncSetAttribute(attn_q4_decode_kernel<NT, W, kMulti>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(Q4Shared<NT, W>));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(attn_q4_decode_kernel<NT, W, kMulti>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_set.mark(dev);
  }
  const int64_t units = (A.total + kUnit - 1) / kUnit;
  if (A.part) {
    A.C = split_ctas(units, A.Hkv, Q4Shape<NT, W>::kPerSm);
    const cudaError_t e = launch_dependent(attn_q4_decode_kernel<NT, W, kMulti>, dim3((unsigned)A.C, (unsigned)A.Hkv),
                                           Q4Shape<NT, W>::kThreads, sizeof(Q4Shared<NT, W>), 1, s, A);
    if (e != cudaSuccess) return e;
    return launch_dependent(attn_q4_join_kernel, dim3((unsigned)(A.Hkv * A.M * A.G)), 32 * kJoinWarps, 0, 1, s, A);
  }
  // Every warp has 16 positions at least, and all clusters run at once.
  int c = 1;
  while (c < kQMaxCluster && units > Q4Shape<NT, W>::kWarps * c && A.Hkv <= max_clusters<NT, W, kMulti>(2 * c)) c *= 2;
  A.C = c;
  return launch_dependent(attn_q4_decode_kernel<NT, W, kMulti>, dim3((unsigned)c, (unsigned)A.Hkv), Q4Shape<NT, W>::kThreads,
                          sizeof(Q4Shared<NT, W>), (unsigned)c, s, A);
}

// ---------------------------------------------------------------------------
// The cache's rows as fp16
// ---------------------------------------------------------------------------
constexpr int kDqThreads = 256;

struct DqArgs {
  const uint32_t* q4[2];
  const uint32_t* dm[2];
  uint4* out[2];
  int per_row, step;  // words of a row; rows of a CTA
  int64_t Lmax, rows, sinks, gap;
};

// The values of rows of a 4-bit cache, into fp16. A thread has one word of 8 values: a warp reads
// 128 bytes and writes 512, and the many small CTAs of a call hide the latency: 8 x 4200 rows of
// 128 in 3.6 us (11.3 MB, 1.7 us at a copy's rate), K and V of 8 x 8024 rows of a chunk in about
// 10. Two, four and eight words a thread, all in flight, made calls with both exports of 8 x 4200
// rows 0.2, 2.3 and 5.4 us longer.
__global__ void __launch_bounds__(kDqThreads) dequant_kv_q4_kernel(const __grid_constant__ DqArgs A) {
  const int rr = threadIdx.x / A.per_row, c = threadIdx.x - rr * A.per_row;
  const int64_t r = (int64_t)blockIdx.x * A.step + rr;
  const int64_t j = (int64_t)blockIdx.y * A.Lmax + r + (r < A.sinks ? 0 : A.gap);
  dependent_wait();
  if (rr >= A.step || r >= A.rows) return;
  const uint32_t w = ldg_stream4(A.q4[blockIdx.z] + j * A.per_row + c);
  const uint32_t sc = __ldg(A.dm[blockIdx.z] + j * (A.per_row >> 2) + (c >> 2));
  // pairs (nibble k of the low half, of the high half) are values k and 4 + k
  __half2 q[4];
  unpack_pairs(w, q);
  const __half2 d = as_h2(prmt(sc, sc, 0x1010)), mm = as_h2(prmt(sc, sc, 0x3232));
  uint32_t v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = as_u32(__hfma2(q[k], d, mm));
  A.out[blockIdx.z][((int64_t)blockIdx.y * A.rows + r) * A.per_row + c] =
      make_uint4(prmt(v[0], v[1], 0x5410), prmt(v[2], v[3], 0x5410), prmt(v[0], v[1], 0x7632),
                 prmt(v[2], v[3], 0x7632));
}

// What a call's queries see, numbered without holes: visible position u is
// position u, or u + gap from sink_rows on; `total` of them.
struct Visible {
  int64_t sink_rows, gap, total;
};
Visible visible(int64_t M, int64_t pos0, int64_t window, int64_t sinks) {
  const int64_t end = pos0 + M;
  sinks = std::min(sinks, end);
  if (window == 0) return {sinks, 0, sinks};  // the sinks alone
  const int64_t first = std::max<int64_t>(0, pos0 - window + 1);
  if (first <= sinks) return {0, 0, end};
  return {sinks, first - sinks, sinks + end - first};
}

// Whether a call of few tokens splits its positions over all SMs, joined by a
// second kernel through the scratch, rather than over a cluster for each key/value
// head, of which a GPC takes few.
bool over_all_sms(int64_t total, int Hkv) { return total * Hkv >= kQSplitFrom; }

bool few_tokens(int64_t M, int H, int Hkv) { return M * (H / Hkv) <= kQMaxCols; }

}  // namespace

cudaError_t launch_dequant_kv_q4(const Q4Cache& c, uint16_t* k_out, uint16_t* v_out, int Hkv, int D, int64_t Lmax,
                                 int64_t rows, int64_t sinks, int64_t gap, cudaStream_t s) {
  DqArgs a = {};
  const uint8_t* q[2] = {c.k_q4, c.v_q4};
  const uint16_t* dm[2] = {c.k_dm, c.v_dm};
  uint16_t* out[2] = {k_out, v_out};
  for (int i = 0; i < 2; ++i) {
    a.q4[i] = reinterpret_cast<const uint32_t*>(q[i]);
    a.dm[i] = reinterpret_cast<const uint32_t*>(dm[i]);
    a.out[i] = reinterpret_cast<uint4*>(out[i]);
  }
  a.per_row = D / 8;
  a.step = kDqThreads / a.per_row;
  a.Lmax = Lmax;
  a.rows = rows;
  a.sinks = sinks;
  a.gap = gap;
  const dim3 grid((unsigned)((rows + a.step - 1) / a.step), (unsigned)Hkv, v_out ? 2u : 1u);
  return launch_dependent(dequant_kv_q4_kernel, grid, kDqThreads, 0, 1, s, a);
}

int64_t attn_q4_scratch(int64_t M, int H, int Hkv, int64_t pos0, int64_t window, int64_t sinks) {
  if (M == 0 || (window == 0 && sinks == 0)) return 0;
  const int64_t total = visible(M, pos0, window, sinks).total;
  if (!few_tokens(M, H, Hkv)) return 2 * Hkv * total * kRowBytes;
  return !over_all_sms(total, Hkv) ? 0 : std::max(kQMaxSplit, Hkv) * M * (H / Hkv) * (kD + 2) * (int64_t)sizeof(float);
}

cudaError_t launch_gqa_attention_q4(const uint16_t* q, const Q4Cache& c, uint16_t* out, int64_t M, int H, int Hkv,
                                    int64_t pos0, int64_t Lmax, float scale, int64_t window, int64_t sinks,
                                    void* scratch, cudaStream_t s) {
  if (window == 0 && sinks == 0) return cudaMemsetAsync(out, 0, (size_t)M * H * kRowBytes, s);  // nothing is visible
  window = std::min(window, pos0 + M);
  sinks = std::min(sinks, pos0 + M);
  const Visible see = visible(M, pos0, window, sinks);
  if (!few_tokens(M, H, Hkv)) {
    // The visible rows next to each other: positions past the sinks move by the gap.
    uint16_t* k16 = static_cast<uint16_t*>(scratch);
    uint16_t* v16 = k16 + Hkv * see.total * kD;
    const cudaError_t e = launch_dequant_kv_q4(c, k16, v16, Hkv, kD, Lmax, see.total, see.sink_rows, see.gap, s);
    if (e != cudaSuccess) return e;
    return launch_gqa_attention_window(q, k16, v16, out, M, H, Hkv, pos0 - see.gap, see.total, scale, window, sinks, s);
  }
  const Q4Args A{reinterpret_cast<const __half*>(q),
                 reinterpret_cast<__half*>(out),
                 reinterpret_cast<const uint4*>(c.k_q4),
                 reinterpret_cast<const uint4*>(c.v_q4),
                 reinterpret_cast<const uint32_t*>(c.k_dm),
                 reinterpret_cast<const uint32_t*>(c.v_dm),
                 H,
                 Hkv,
                 H / Hkv,
                 (int)M,
                 pos0,
                 Lmax,
                 window,
                 sinks,
                 see.sink_rows,
                 see.gap,
                 see.total,
                 scale * 1.4426950408889634f,
                 1,
                 over_all_sms(see.total, Hkv) ? static_cast<float*>(scratch) : nullptr};
  const int nt = (int)((M * (H / Hkv) + 7) / 8);
  if (nt == 1 && A.part) return M == 1 ? launch_decode<1, 16, false>(A, s) : launch_decode<1, 16, true>(A, s);
  if (nt == 1) return M == 1 ? launch_decode<1, 8, false>(A, s) : launch_decode<1, 8, true>(A, s);
  return nt == 2 ? launch_decode<2, 8, true>(A, s) : launch_decode<4, 8, true>(A, s);
}

}  // namespace qk
