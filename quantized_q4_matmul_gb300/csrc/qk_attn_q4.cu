// qk_attn_q4.cu -- grouped-query attention over a KV cache held in 4 bits, and
// the cache's rows as fp16.
//
// Source: DAMASCUS project overview, "[02] the pipeline" (a decoder layer is GQA
// with a KV cache) and "[04] one decode step"; the 4-bit cache is this library's.
//
// A row of one position and key/value head holds groups of 32 values as v = d q + m
// (q in 0 .. 15, d and m fp16): 64 bytes of quants and 16 of (d, m) for 128
// values, 80 bytes where fp16 takes 256.  Every path uses fp16(d q + m), one
// rounding, so that they agree with the rows that qk_dequant_kv_q4 gives.
//
// Few tokens (a decode step, or drafted tokens: M * H / H_kv <= 32 columns, a
// column being a query head of one token).  A cluster of up to 16 CTAs per
// key/value head splits the visible positions; a warp takes 16 of them at a time,
// straight from global memory into registers (a lane has one whole group of 32
// key and value quants of a position, 16 bytes, so a warp's load is 512
// contiguous bytes), with the next 16 on their way.  mma.sync, whose 8-wide N side
// holds the columns, multiplies:
//   S^T = K Q^T  (16 positions x 8 columns): the product's k axis is permuted to
//     what the lanes hold, so nothing is exchanged;
//   O^T = V^T P  (dimensions x columns): movmatrix transposes 8 positions of 4
//     nibbles each, which are four dimensions' k pairs.
// A nibble becomes an fp16 by OR with an exponent (1024 + q, or 64 + q where it
// sits 4 bits higher), a subtraction and one fused multiply-add for its pair.
// Every warp keeps its own running maximum, sums and O; the warps of a CTA join
// in order through shared memory, the CTAs through distributed shared memory,
// each writing a share of the outputs.
//
// More tokens: the visible rows are written as fp16 to the caller's scratch once
// and the windowed prefill runs over them: a query tile's 128 rows would unpack
// each key again.
//
// The kernel has no waits but the cluster barriers, which every thread reaches.
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
constexpr int kQMaxCols = 32;
constexpr int kUnit = 16;  // positions of a warp's step

// The shape of a CTA for NT tiles of 8 columns.
template <int NT>
struct Q4Shape {
  static constexpr int kWarps = NT == 1 ? 16 : 8;  // registers for the columns' O
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kCols = 8 * NT;
};

template <int NT>
struct Q4Shared {
  using Sh = Q4Shape<NT>;
  float part[Sh::kWarps][Sh::kCols * kD];  // the warps' O
  float red[kQMaxCluster * 4 + Sh::kCols * kD];  // what the CTAs send: [rank][this CTA's share of the outputs]
  float2 stat[kQMaxCluster][Sh::kCols];    // and their (max, sum)
  float wmax[Sh::kWarps][Sh::kCols], wsum[Sh::kWarps][Sh::kCols];
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
  int C;
};

// The nibbles of a word as four pairs of fp16 (nibble i of the low half and of
// the high half), exact.
__device__ __forceinline__ void unpack_pairs(uint32_t w, __half2 (&q)[4]) {
  const uint32_t k1024 = 0x64006400u, k64 = 0x54005400u;
  const __half2 o1024 = *reinterpret_cast<const __half2*>(&k1024), o64 = *reinterpret_cast<const __half2*>(&k64);
  const uint32_t h = w >> 8;
  const uint32_t u[4] = {lop_and_or<0x000f000fu>(w, k1024), lop_and_or<0x00f000f0u>(w, k64),
                         lop_and_or<0x000f000fu>(h, k1024), lop_and_or<0x00f000f0u>(h, k64)};
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = __hsub2(*reinterpret_cast<const __half2*>(&u[i]), i & 1 ? o64 : o1024);
}

__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

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

// A lane's part of 16 rows: group lane % 4 of rows lane / 4 and lane / 4 + 8.
struct Q4Unit {
  uint4 k[2], v[2];
  uint32_t ks[2], vs[2];
};

// Up to 8 NT columns against the visible positions of one key/value head.  Rank r
// of the cluster takes visible positions [r n / C, (r + 1) n / C) in multiples of
// 16, its warps every kWarps-th 16 of them.  kMulti: more than one token, so that
// columns see different positions.
template <int NT, bool kMulti>
__global__ void __launch_bounds__(Q4Shape<NT>::kThreads, 1) attn_q4_decode_kernel(const __grid_constant__ Q4Args A) {
  using Sh = Q4Shape<NT>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Q4Shared<NT>& S = *reinterpret_cast<Q4Shared<NT>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane >> 2, tq = lane & 3;
  const int g = blockIdx.y;
  const int rank = (int)cluster_rank();
  const int units = (int)((A.total + kUnit - 1) / kUnit);
  const int unit1 = (int)((int64_t)(rank + 1) * units / A.C);
  int unit = (int)((int64_t)rank * units / A.C) + warp;
  const int total = (int)A.total, sink_rows = (int)A.sink_rows, gap = (int)A.gap;
  const uint4 *kq = A.k_q4 + (int64_t)g * A.Lmax * 4 + tq, *vq = A.v_q4 + (int64_t)g * A.Lmax * 4 + tq;
  const uint32_t *kd = A.k_dm + (int64_t)g * A.Lmax * 4 + tq, *vd = A.v_dm + (int64_t)g * A.Lmax * 4 + tq;
  __syncwarp();
  cluster_arrive();  // its wait is before the first write to another CTA
  dependent_wait();

  auto load = [&](int at, Q4Unit& x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int u = min(kUnit * at + grp + 8 * i, total - 1);  // past the end: the last row again
      const int64_t j = 4 * (int64_t)(u < sink_rows ? u : u + gap);
      x.k[i] = ldg_stream16(kq + j);
      x.ks[i] = ldg_stream4(kd + j);
      x.v[i] = ldg_stream16(vq + j);
      x.vs[i] = ldg_stream4(vd + j);
    }
  };
  Q4Unit x;
  if (unit < unit1) load(unit, x);

  // Q: the product's k axis in step (word j, half h) is dims 32 tq + 8 j + 2 h and + 4
  // (first register), and those + 1 (second), of this lane's tq.
  uint32_t qb[NT][4][2][2];
  int cpos[NT][2];    // the positions of this lane's columns
  float o[NT][8][4];  // [column tile][2 j + h]: dims 32 (grp / 2) + 8 j + 4 (grp % 2) + 2 h (+ 1: elements 2, 3), columns 2 tq (+ 1)
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int col = 8 * n + grp;
    const int token = kMulti ? col / A.G : 0;
    const uint4* qr = reinterpret_cast<const uint4*>(A.q + ((int64_t)token * A.H + g * A.G + (col - token * A.G)) * kD) + 4 * tq;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 y = col < A.M * A.G ? qr[j] : make_uint4(0u, 0u, 0u, 0u);
      qb[n][j][0][0] = prmt(y.x, y.z, 0x5410);
      qb[n][j][0][1] = prmt(y.x, y.z, 0x7632);
      qb[n][j][1][0] = prmt(y.y, y.w, 0x5410);
      qb[n][j][1][1] = prmt(y.y, y.w, 0x7632);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      cpos[n][e] = (int)A.pos0 + (kMulti ? min((8 * n + 2 * tq + e) / A.G, A.M - 1) : 0);
      m[n][e] = -INFINITY;
      l[n][e] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
  }

  for (; unit < unit1; unit += Sh::kWarps) {
    const int u = kUnit * unit, rows = total - u;  // rows past them are copies
    Q4Unit next = x;
    if (unit + Sh::kWarps < unit1) load(unit + Sh::kWarps, next);
    // ---- scores: rows grp and grp + 8, this lane's group of the dimensions
    float sc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
    {
      const __half2 d0 = as_h2(prmt(x.ks[0], x.ks[0], 0x1010)), m0 = as_h2(prmt(x.ks[0], x.ks[0], 0x3232));
      const __half2 d1 = as_h2(prmt(x.ks[1], x.ks[1], 0x1010)), m1 = as_h2(prmt(x.ks[1], x.ks[1], 0x3232));
      const uint32_t a0[4] = {x.k[0].x, x.k[0].y, x.k[0].z, x.k[0].w}, a1[4] = {x.k[1].x, x.k[1].y, x.k[1].z, x.k[1].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        __half2 p0[4], p1[4];
        unpack_pairs(a0[j], p0);
        unpack_pairs(a1[j], p1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a[4] = {as_u32(__hfma2(p0[2 * h], d0, m0)), as_u32(__hfma2(p1[2 * h], d1, m1)),
                                 as_u32(__hfma2(p0[2 * h + 1], d0, m0)), as_u32(__hfma2(p1[2 * h + 1], d1, m1))};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(sc[n], a, qb[n][j][h][0], qb[n][j][h][1]);
        }
      }
    }
    // ---- weights
    uint32_t pb[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float tmax[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // e: column e & 1, row grp + 8 (e >> 1)
        const int r = grp + 8 * (e >> 1);
        bool seen = r < rows;
        if (kMulti) {
          const int j = u + r + (u + r < sink_rows ? 0 : gap), p = cpos[n][e & 1];
          seen = seen && j <= p && (p - j < A.window || j < A.sinks);
        }
        const float v = seen ? sc[n][e] * A.scale_log2e : -INFINITY;
        sc[n][e] = v;
        tmax[e & 1] = fmaxf(tmax[e & 1], v);
      }
      bool grows = false;
      float mn[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        tmax[e] = fmaxf(tmax[e], __shfl_xor_sync(0xffffffffu, tmax[e], 4));
        tmax[e] = fmaxf(tmax[e], __shfl_xor_sync(0xffffffffu, tmax[e], 8));
        tmax[e] = fmaxf(tmax[e], __shfl_xor_sync(0xffffffffu, tmax[e], 16));
        mn[e] = fmaxf(m[n][e], tmax[e]);
        grows = grows || mn[e] > m[n][e];
      }
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float corr = mn[e] == -INFINITY ? 1.f : ex2_approx(m[n][e] - mn[e]);
          m[n][e] = mn[e];
          l[n][e] *= corr;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[n][i][e] *= corr;
            o[n][i][e + 2] *= corr;
          }
        }
      }
      // relative to 0 where no visible score is a number yet: hidden scores have
      // weight 0 there too, and NaN, which the maximum passes over, stays
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float ref = m[n][e & 1];
        p[e] = ex2_approx(sc[n][e] - (ref == -INFINITY ? 0.f : ref));
        l[n][e & 1] += p[e];
      }
      pb[n][0] = transpose8(pack_h2(p[0], p[1]));
      pb[n][1] = transpose8(pack_h2(p[2], p[3]));
    }
    // ---- O^T += V^T P: after transposing, this lane has group grp / 2 of the
    // dimensions and rows 2 tq, 2 tq + 1 (and those + 8)
    __half2 dv[2], mv[2];
    bool odd = false;  // a row has a value that is not finite
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // even lanes' rows get d, odd ones m, of the pair of positions
      const uint32_t mine = transpose8(grp + 8 * i < rows ? x.vs[i] : 0u);
      const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 4);
      uint32_t d = grp & 1 ? other : mine, mm = grp & 1 ? mine : other;
      if (kMulti) {
        // the largest value; infinity and NaN have the exponent's bits all set
        const uint32_t top = as_u32(__hfma2(__float2half2_rn(15.f), as_h2(d), as_h2(mm)));
        const bool b0 = (top & 0x7C00u) == 0x7C00u, b1 = (top & 0x7C000000u) == 0x7C000000u;
        const uint32_t keep = (b0 ? 0u : 0xFFFFu) | (b1 ? 0u : 0xFFFF0000u);
        d &= keep;
        mm &= keep;
        odd = odd || b0 || b1;
      }
      dv[i] = as_h2(d);
      mv[i] = as_h2(mm);
    }
    const uint32_t v0[4] = {x.v[0].x, x.v[0].y, x.v[0].z, x.v[0].w}, v1[4] = {x.v[1].x, x.v[1].y, x.v[1].z, x.v[1].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      __half2 p0[4], p1[4];
      unpack_pairs(transpose8(v0[j]), p0);
      unpack_pairs(transpose8(v1[j]), p1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t a[4] = {as_u32(__hfma2(p0[2 * h], dv[0], mv[0])), as_u32(__hfma2(p0[2 * h + 1], dv[0], mv[0])),
                               as_u32(__hfma2(p1[2 * h], dv[1], mv[1])), as_u32(__hfma2(p1[2 * h + 1], dv[1], mv[1]))};
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816(o[n][2 * j + h], a, pb[n][0], pb[n][1]);
      }
    }
    if (kMulti && __any_sync(0xffffffffu, odd)) {
      // Such a value has entered the product as 0: it is NaN for the columns that
      // see its row, and nothing for the others.
      for (int r = 0; r < kUnit && r < rows; ++r) {
        const int j = u + r + (u + r < sink_rows ? 0 : gap);
        const uint32_t w = (vd - tq)[4 * (int64_t)j + (grp >> 1)];
        const __half2 top = __hfma2(__float2half2_rn(15.f), as_h2(w), as_h2(w >> 16));
        if ((as_u32(top) & 0x7C00u) != 0x7C00u) continue;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int p = cpos[n][e];
            if (j <= p && (p - j < A.window || j < A.sinks))
#pragma unroll
              for (int i = 0; i < 8; ++i) o[n][i][e] = o[n][i][e + 2] = NAN;
          }
      }
    }
    x = next;
  }
  // The lanes of a column join their sums; the warp's maximum and sum.
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
      l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
      l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
      // -inf: it saw nothing.  A warp that saw NaN alone has no maximum either, but
      // a NaN sum: with NaN as its maximum it counts, and the column is NaN.
      if (m[n][e] == -INFINITY && l[n][e] != 0.f) m[n][e] = NAN;
      if (grp == 0) {
        S.wmax[warp][8 * n + 2 * tq + e] = m[n][e];
        S.wsum[warp][8 * n + 2 * tq + e] = l[n][e];
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
      float* dst = &S.part[warp][col * kD + 32 * (grp >> 1) + 4 * (grp & 1)];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4*>(dst + 8 * j) =
            make_float4(f * o[n][2 * j][e], f * o[n][2 * j][e + 2], f * o[n][2 * j + 1][e], f * o[n][2 * j + 1][e + 2]);
    }
  __syncthreads();
  __syncwarp();
  cluster_wait();  // every CTA of the cluster is running
  // The CTA's sums, the warps in order, go to the CTA of the cluster that writes
  // them out: shares of the M G 128 outputs in runs of four.
  const int cols = A.M * A.G, quads = cols * (kD / 4);
  const int share = (quads + A.C - 1) / A.C;
  for (int i = threadIdx.x; i < quads; i += Sh::kThreads) {
    float4 a = *reinterpret_cast<const float4*>(&S.part[0][4 * i]);
    for (int w = 1; w < Sh::kWarps; ++w) {
      const float4 b = *reinterpret_cast<const float4*>(&S.part[w][4 * i]);
      a.x += b.x;
      a.y += b.y;
      a.z += b.z;
      a.w += b.w;
    }
    const int to = i / share;
    st_cluster_v4(mapa_shared(smem_u32(&S.red[4 * (rank * share + i - to * share)]), (uint32_t)to), a);
  }
  for (int i = threadIdx.x; i < cols * A.C; i += Sh::kThreads) {
    const int to = i / cols, col = i - to * cols;
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < Sh::kWarps; ++w) M = fmaxf(M, S.wmax[w][col]);
    bool nan = false;
    for (int w = 0; w < Sh::kWarps; ++w) {
      const float mw = S.wmax[w][col];
      if (mw != -INFINITY) L = fmaf(exp2f(mw - M), S.wsum[w][col], L);
      nan = nan || mw != mw;
    }
    st_cluster_v2(mapa_shared(smem_u32(&S.stat[rank][col]), (uint32_t)to), make_float2(nan ? NAN : M, L));
  }
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

// How many clusters of `c` CTAs of the kernel the device runs at once (a cluster
// lies within one GPC).  Asked once per device and size; attributes are set before.
template <int NT, bool kMulti>
int max_clusters(int c) {
  static std::atomic<int> known[kMaxDevices][kQMaxCluster + 1];
  const int dev = current_device();
  if (dev < 0) return 0;
  int n = known[dev][c].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c);
    cfg.blockDim = dim3(Q4Shape<NT>::kThreads);
    cfg.dynamicSmemBytes = sizeof(Q4Shared<NT>);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)c;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, attn_q4_decode_kernel<NT, kMulti>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    n = n > 0 ? n : -1;  // -1: none
    known[dev][c].store(n, std::memory_order_relaxed);
  }
  return n;
}

template <int NT, bool kMulti>
cudaError_t launch_decode(Q4Args A, cudaStream_t s) {
  static_assert(sizeof(Q4Shared<NT>) <= 227 * 1024, "shared memory of a CTA");
  static PerDeviceFlag attr_set;
  const int dev = current_device();
  if (!attr_set.done(dev)) {
    cudaError_t e = cudaFuncSetAttribute(attn_q4_decode_kernel<NT, kMulti>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(Q4Shared<NT>));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(attn_q4_decode_kernel<NT, kMulti>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_set.mark(dev);
  }
  // Every warp has 16 positions at least, and all clusters run at once.
  const int64_t units = (A.total + kUnit - 1) / kUnit;
  int c = 1;
  while (c < kQMaxCluster && units > Q4Shape<NT>::kWarps * c && A.Hkv <= max_clusters<NT, kMulti>(2 * c)) c *= 2;
  A.C = c;
  return launch_dependent(attn_q4_decode_kernel<NT, kMulti>, dim3((unsigned)c, (unsigned)A.Hkv), Q4Shape<NT>::kThreads,
                          sizeof(Q4Shared<NT>), (unsigned)c, s, A);
}

// ---------------------------------------------------------------------------
// The cache's rows as fp16
// ---------------------------------------------------------------------------
constexpr int kDqThreads = 256;
constexpr int kDqItems = 4;  // words of 8 values of a thread

struct DqArgs {
  const uint32_t* q4[2];
  const uint32_t* dm[2];
  uint4* out[2];
  int per_row, rows_per_cta;  // words of a row; rows of a CTA
  int64_t Lmax, rows, sinks, gap;
};

__global__ void __launch_bounds__(kDqThreads) dequant_kv_q4_kernel(const __grid_constant__ DqArgs A) {
  const int64_t r0 = (int64_t)blockIdx.x * A.rows_per_cta;
  const int items = (int)min((int64_t)A.rows_per_cta, A.rows - r0) * A.per_row;
  const int64_t in = (int64_t)blockIdx.y * A.Lmax, out = (int64_t)blockIdx.y * A.rows;
  const uint32_t *q4 = A.q4[blockIdx.z], *dm = A.dm[blockIdx.z];
  uint4* dst = A.out[blockIdx.z];
  dependent_wait();
  for (int i0 = threadIdx.x; i0 < items; i0 += kDqItems * kDqThreads) {
    uint32_t w[kDqItems], sc[kDqItems];
#pragma unroll
    for (int b = 0; b < kDqItems; ++b) {
      const int i = i0 + b * kDqThreads;
      if (i < items) {
        const int rr = i / A.per_row, c = i - rr * A.per_row;
        const int64_t r = r0 + rr, j = (in + r + (r < A.sinks ? 0 : A.gap)) * A.per_row + c;
        w[b] = ldg_stream4(q4 + j);
        sc[b] = __ldg(dm + (j >> 2));
      }
    }
#pragma unroll
    for (int b = 0; b < kDqItems; ++b) {
      const int i = i0 + b * kDqThreads;
      if (i >= items) continue;
      // pairs (nibble k of the low half, of the high half) are values k and 4 + k
      __half2 q[4];
      unpack_pairs(w[b], q);
      const __half2 d = as_h2(prmt(sc[b], sc[b], 0x1010)), mm = as_h2(prmt(sc[b], sc[b], 0x3232));
      uint32_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = as_u32(__hfma2(q[k], d, mm));
      dst[(out + r0) * A.per_row + i] =
          make_uint4(prmt(v[0], v[1], 0x5410), prmt(v[2], v[3], 0x5410), prmt(v[0], v[1], 0x7632),
                     prmt(v[2], v[3], 0x7632));
    }
  }
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
  a.rows_per_cta = std::max(1, 2 * kDqItems * kDqThreads / a.per_row);
  a.Lmax = Lmax;
  a.rows = rows;
  a.sinks = sinks;
  a.gap = gap;
  const dim3 grid((unsigned)((rows + a.rows_per_cta - 1) / a.rows_per_cta), (unsigned)Hkv, v_out ? 2u : 1u);
  return launch_dependent(dequant_kv_q4_kernel, grid, kDqThreads, 0, 1, s, a);
}

int64_t attn_q4_scratch(int64_t M, int H, int Hkv, int64_t pos0, int64_t window, int64_t sinks) {
  if (M == 0 || few_tokens(M, H, Hkv) || (window == 0 && sinks == 0)) return 0;
  return 2 * Hkv * visible(M, pos0, window, sinks).total * kRowBytes;
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
                 1};
  const int nt = (int)((M * (H / Hkv) + 7) / 8);
  if (nt == 1) return M == 1 ? launch_decode<1, false>(A, s) : launch_decode<1, true>(A, s);
  return nt == 2 ? launch_decode<2, true>(A, s) : launch_decode<4, true>(A, s);
}

}  // namespace qk
