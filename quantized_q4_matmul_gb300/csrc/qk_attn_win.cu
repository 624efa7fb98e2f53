// qk_attn_win.cu -- grouped-query attention with a sliding window and sinks
// over the KV cache: position j <= p is visible to the query at position p when
// j > p - window or j < sinks.
//
// Source: DAMASCUS project overview, "[02] the pipeline" (a decoder layer is GQA
// with a KV cache) and "[04] one decode step"; the window and the sinks bound
// the cache that one step reads.
//
// Layouts: q [M][H][128] fp16 (query i at position pos0 + i), caches
// [H_kv][L_max][128] fp16, out [M][H][128] fp16 (the O projection's x).
//
// Prefill (M >= 2) on the 5th-generation tensor cores.  A query tile is 128
// rows: the G heads of one key/value head for floor(128 / G) consecutive
// queries, so that a key or value tile is read once for all of them and a
// tile's queries span few positions (a window of 512 over 42 queries touches 5
// tiles of keys, over 128 queries 6).  A CTA has two query tiles and one stream
// of key and value tiles (128 positions, TMA, a ring of five): while one tile's
// four softmax warps work, the tensor core runs the other tile's S = Q K^T and
// O += P V.  P (fp16) takes the place of its S in tensor memory, O stays there.
// One thread owns one row: no exchange between threads, and the running maximum
// moves only when it grows by more than 2^8, so O is rarely rescaled.
//
// The tiles of a CTA are the sinks' (from maps that hold the sinks alone) and
// then those from the first position that its first query sees; where the two
// meet, one run from position 0.  A position that no query of the CTA sees is
// never loaded.
//
// Few queries (a short chunk after a long context) make few CTAs, so a cluster of
// up to eight shares a CTA's work: each takes a run of its key tiles, and they
// join their (maximum, sum, O) through distributed shared memory, in rank order.
// Pairs of query tiles that would leave most of a last round of SMs idle are
// taken apart: a CTA for each tile.
//
// Rows whose result is not finite are computed again without the positions that
// they do not see (attend_row), each by one warp: where one infinite value
// reaches every row, 38.6 ms for the 4095 queries below, 6.3 ms for the 2048.
//
// Bound by the hand-over between a tile's softmax and its products, which share
// tensor-memory columns: 4095 queries after 4001, 24 heads over 8, window 2048:
// 109 us, 955 TFLOP/s of the visible pairs (the tensor pipe is active in 44 % of
// the cycles, the schedulers issue in 42 %: neither is full); 2048 queries,
// window 512: 27.3 us (1.6 rounds of SMs of 5 or 6 key tiles each).
//
// Decode (M = 1) runs in qk_attn.cu.
//
// Waits on mbarriers are bounded; a timeout raises the device status word.  The
// named barrier and the two cluster barriers of a shared tile have no limit of
// their own: all role loops end on bounded waits, and every thread reaches the
// barriers on every path.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "qk_attn.cuh"
#include "qk_device.cuh"
#include "qk_internal.h"

namespace qk {

__device__ uint32_t g_attn_win_status = 0;

namespace {

constexpr int kWK = 128;         // positions per key / value tile
constexpr int kWRing = 5;        // key and value tiles in flight, in the order of their use: K0 V0 K1 V1 ...
constexpr int kWWarps = 12;      // copy, 2 UMMA issuers, 1 idle, 4 softmax warps for each query tile
constexpr int kWThreads = 32 * kWWarps;
constexpr int kWMaxSplit = 8;    // CTAs that share the key tiles of a pair of query tiles

struct WpShared {
  uint8_t q[2][kTTile];
  uint8_t kv[kWRing][kTTile];
  uint64_t q_full;
  uint64_t full[kWRing];
  uint64_t empty[kWRing];
  uint64_t s_full[2];     // [query tile] S is in tensor memory
  uint64_t p_full[2][2];  // [query tile][half]: 64 positions of P are in tensor memory
  uint64_t pv_done[2];    // O holds the tile's product, P's columns are free for the next S
  uint64_t mma_done[2];
  uint64_t turn[2];       // whose turn on the tensor core
  uint32_t tmem_base;
  uint32_t abort_flag;
};

struct WpArgs {
  const __half *q, *kc, *vc;
  __half* out;
  int H, Hkv, G, queries;  // query heads, key/value heads, heads per key/value head, queries per tile
  int64_t M, pos0, Lmax, window, sinks;
  float scale_log2e;
  unsigned units, pairs;  // pairs of query tiles of all key/value heads; those of them that are one CTA's
  int split;              // CTAs (of a cluster) that share a pair of query tiles
};

// What a CTA of a cluster leaves for the others, where its key and value tiles
// were: O of its query tiles, rows of 512 bytes whose 16-byte chunks are
// permuted by the row (a warp writes one chunk of 32 rows at a time), and each
// row's reference and sum.
__device__ __forceinline__ uint32_t part_chunk(const WpShared& S, int t, int r, int c) {
  return smem_u32(S.kv[2 * t]) + (uint32_t)(r * 512 + ((c ^ (r & 31)) << 4));
}
__device__ __forceinline__ uint32_t part_stat(const WpShared& S, int t, int r) {
  return smem_u32(S.kv[4]) + (uint32_t)(8 * (128 * t + r));
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

// Packed pairs of fp32 (one instruction for two values).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// One query row of one head by one warp, over the positions that it sees and no
// other; lane t takes the dimensions 4 t .. 4 t + 3 of the result.  The tensor
// core multiplies a hidden position's value row by the weight 0, and 0 times
// infinity is not 0: rows that come out non-finite are done again here, so that
// a non-finite value row reaches those queries alone that see it.
__device__ __noinline__ void attend_row(const WpArgs& A, int64_t row, int head) {
  const int lane = threadIdx.x & 31;
  const int64_t p = A.pos0 + row, kv = (int64_t)(head / A.G) * A.Lmax * kD;
  const uint4* qr = reinterpret_cast<const uint4*>(A.q + (row * A.H + head) * kD);
  const int64_t end1 = min(A.sinks, p + 1), from2 = max(end1, p - A.window + 1);
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int run = 0; run < 2; ++run) {
    const int64_t end = run == 0 ? end1 : p + 1;
    for (int64_t base = run == 0 ? 0 : from2; base < end; base += 32) {
      const int64_t j = base + lane;
      float s = -INFINITY;
      if (j < end) {
        const uint4* kr = reinterpret_cast<const uint4*>(A.kc + kv + j * kD);
        s = 0.f;
        for (int i = 0; i < kD / 8; ++i) {
          const uint4 a = qr[i], b = kr[i];
          const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&x[e]));
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&y[e]));
            s = fmaf(u.y, v.y, fmaf(u.x, v.x, s));
          }
        }
        s *= A.scale_log2e;
      }
      float mn = s;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      mn = fmaxf(mn, m);
      const float ref = mn == -INFINITY ? 0.f : mn, corr = exp2f(m - ref);
      m = mn;
      const float w = exp2f(s - ref);
      float sum = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l = fmaf(l, corr, sum);
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] *= corr;
      for (int e = 0; e < 32 && base + e < end; ++e) {
        const float we = __shfl_sync(0xffffffffu, w, e);
        const uint2 v = *reinterpret_cast<const uint2*>(A.vc + kv + (base + e) * kD + 4 * lane);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
        acc[0] = fmaf(we, a.x, acc[0]);
        acc[1] = fmaf(we, a.y, acc[1]);
        acc[2] = fmaf(we, b.x, acc[2]);
        acc[3] = fmaf(we, b.y, acc[3]);
      }
      // nothing more to find out about a row that is NaN throughout
      const bool nan = acc[0] != acc[0] && acc[1] != acc[1] && acc[2] != acc[2] && acc[3] != acc[3];
      if (__all_sync(0xffffffffu, nan || l != l)) {
        run = 2;
        break;
      }
    }
  }
  const float inv = 1.0f / l;
  *reinterpret_cast<uint2*>(A.out + (row * A.H + head) * kD + 4 * lane) =
      make_uint2(pack_h2(within_half(acc[0] * inv), within_half(acc[1] * inv)),
                 pack_h2(within_half(acc[2] * inv), within_half(acc[3] * inv)));
}

// Bits e of 0 .. 31 with lo <= e < hi.
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
  lo = max(0, min(32, lo));
  hi = max(0, min(32, hi));
  const uint32_t below_hi = hi >= 32 ? 0xffffffffu : (1u << hi) - 1u;
  const uint32_t below_lo = lo >= 32 ? 0xffffffffu : (1u << lo) - 1u;
  return below_hi & ~below_lo;
}

__global__ void __launch_bounds__(kWThreads, 1)
    attn_win_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_ks,
                            const __grid_constant__ CUtensorMap tm_vs, const __grid_constant__ WpArgs A) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  WpShared& S = *reinterpret_cast<WpShared*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // every head's latest queries, which see the most, first; after A.pairs pairs
  // of query tiles a CTA has one tile
  unsigned unit = blockIdx.x / (unsigned)A.split;
  const int rank = (int)(blockIdx.x - unit * (unsigned)A.split);
  const unsigned single = unit < A.pairs ? 0u : unit - A.pairs;
  if (unit >= A.pairs) unit = A.pairs + single / 2u;
  const int g = (int)(unit % (unsigned)A.Hkv), G = A.G;
  const int64_t q0 = ((int64_t)((A.units - 1u - unit) / (unsigned)A.Hkv) * 2 + (single & 1u)) * A.queries;
  const bool two = unit < A.pairs && q0 + A.queries < A.M;
  // positions of each query tile's first and last query
  const int64_t pf0 = A.pos0 + q0, pf1 = pf0 + A.queries, end = A.pos0 + A.M - 1;
  const int64_t pl0 = min(pf1 - 1, end), pl1 = min(pf1 + A.queries - 1, end);
  const int64_t last = two ? pl1 : pl0;
  int64_t first = pf0 - A.window + 1;  // first position of the window's run of tiles
  int nt, sink_tiles = 0;
  if (A.window == 0) {  // the sinks alone
    sink_tiles = (int)(((A.sinks <= last ? A.sinks : last + 1) + kWK - 1) / kWK);
    nt = sink_tiles;
  } else {
    if (first <= A.sinks)
      first = 0;
    else
      sink_tiles = (int)((A.sinks + kWK - 1) / kWK);
    nt = sink_tiles + (int)((last - first + kWK) / kWK);
  }
  if (q0 >= A.M) nt = 0;  // the second tile of a pair that has one
  // This CTA's run of them, numbered from 0 from here on.
  const int j0 = (int)((int64_t)rank * nt / A.split);
  nt = (int)((int64_t)(rank + 1) * nt / A.split) - j0;
  sink_tiles -= j0;
  // Position of the first row of tile j: in the sinks' map, or in the cache.
  auto tile_pos = [&](int j) -> int64_t {
    return j < sink_tiles ? (int64_t)(j + j0) * kWK : first + (int64_t)(j - sink_tiles) * kWK;
  };
  // Query tile u has rows that see something of tile j: those up to its last
  // query, but for a gap between the sinks and its first query's window.
  struct Active {
    int end, gap0, gap1;
    __device__ __forceinline__ bool operator()(int j) const { return j < end && (j < gap0 || j >= gap1); }
  };
  auto actives = [&](int u) {
    Active r{0, 0, 0};
    if (u == 1 && !two) return r;
    const int64_t pf = u ? pf1 : pf0, pl = u ? pl1 : pl0;
    if (A.window == 0) {
      r.end = min(nt, (int)(pl / kWK) + 1 - j0);
      return r;
    }
    r.end = min(nt, sink_tiles + (int)((pl - first) / kWK) + 1);
    const int64_t hidden = pf - A.window - first + 1;  // positions of the run before the window
    const int64_t kept = A.sinks - first;              // those of them that are sinks
    r.gap0 = sink_tiles + (int)(kept > 0 ? (kept + kWK - 1) / kWK : 0);
    r.gap1 = sink_tiles + (int)(hidden > 0 ? hidden / kWK : 0);
    return r;
  };

  if (threadIdx.x == 0) {
    mbar_init(&S.q_full, 1);
    for (int s = 0; s < kWRing; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], two ? 2 : 1);  // released by each query tile's issuer
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&S.s_full[t], 1);
      mbar_init(&S.p_full[t][0], 4);
      mbar_init(&S.p_full[t][1], 4);
      mbar_init(&S.pv_done[t], 1);
      mbar_init(&S.mma_done[t], 1);
      mbar_init(&S.turn[t], 1);
    }
    S.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&S.tmem_base, 512);  // S (then P) of the tiles at columns 0 and 128, O at 256 and 384
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  volatile uint32_t* abort_flag = &S.abort_flag;
  dependent_wait();

  if (warp == 0) {
    // ---------------------------------------------------------------- copy warp
    if (lane == 0 && nt > 0) {
      prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
      const uint32_t qbytes = (uint32_t)(kRowBytes * G * A.queries);
      mbar_arrive_expect_tx(&S.q_full, qbytes * (two ? 2u : 1u));
      for (int t = 0; t < (two ? 2 : 1); ++t)
        for (int b = 0; b < 2; ++b)
          tma_load_3d(S.q[t] + b * kTBox, &tm_q, 64 * b, g * G, (int)(q0 + t * A.queries), &S.q_full);
      bool ok = true;
      int n = 0;  // tiles issued: K0 V0 K1 V1 ...
      for (; n < 2 * nt && ok; ++n) {
        const int s = n % kWRing;
        if (n >= kWRing)
          ok = mbar_wait(&S.empty[s], (uint32_t)(n / kWRing - 1) & 1u, abort_flag, &g_attn_win_status);
        if (!ok) break;
        const int j = n >> 1;
        const bool sink = j < sink_tiles;
        const CUtensorMap* m = n & 1 ? (sink ? &tm_vs : &tm_v) : (sink ? &tm_ks : &tm_k);
        mbar_arrive_expect_tx(&S.full[s], (uint32_t)kTTile);
        tma_load_3d(S.kv[s], m, 0, (int)tile_pos(j), g, &S.full[s]);
        tma_load_3d(S.kv[s] + kTBox, m, 64, (int)tile_pos(j), g, &S.full[s]);
      }
      // Drain: every copy issued has landed before the CTA exits.
      mbar_wait(&S.q_full, 0u, abort_flag, &g_attn_win_status, true);
      for (int u = (n > kWRing ? n - kWRing : 0); u < n; ++u)
        mbar_wait(&S.full[u % kWRing], (uint32_t)(u / kWRing) & 1u, abort_flag, &g_attn_win_status, true);
    }
    __syncwarp();
  } else if (warp <= 2) {
    // ---------------------------------------------------------------- UMMA issuers
    // One warp for each query tile.  The whole warp runs this code and an
    // elected lane issues.  The tiles take turns, each with its P V and its next
    // S, so that the tensor core works for one while the other's softmax runs:
    // left alone, the two fall into step, share the tensor core and then leave
    // it idle together.  Within a turn P is taken in halves, as the softmax makes
    // it; the turn ends when the next S is issued, not when it is done.  4095
    // queries after 4001, 24 heads over 8, window 2048: 149 us with one issuing
    // thread for both, 121 with turns, 114 with the halves, 109 with the softmax's
    // sums in four chains.
    const int u = warp - 1;
    if (nt > 0 && (u == 0 || two)) {
      constexpr uint32_t idesc_s = umma_idesc_f16(128, kWK);
      constexpr uint32_t idesc_pv = umma_idesc_f16(128, kD) | (1u << 16);  // B (V) MN-major
      const uint32_t t_s = __shfl_sync(0xffffffffu, tmem, 0) + (uint32_t)(128 * u), t_o = t_s + 256u;
      const uint32_t qa = smem_u32(S.q[u]), kv_s = smem_u32(S.kv[0]);
      const Active act = actives(u);
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        return (bool)__all_sync(0xffffffffu, mbar_wait(bar, phase, abort_flag, &g_attn_win_status));
      };
      struct Slot {  // ring position of the key (or value) tiles: every second slot
        int s;
        uint32_t phase;
        __device__ __forceinline__ void next() {
          s += 2;
          if (s >= kWRing) {
            s -= kWRing;
            phase ^= 1u;
          }
        }
      } ks{0, 0u}, vs{1, 0u};
      uint32_t done = 0;  // tiles whose P V is issued
      bool ok = wait(&S.q_full, 0u);
      // The end of P V holds the next S up (they share columns).
      auto qk = [&]() {
        tc_fence_after();
        const uint32_t ka = kv_s + (uint32_t)(ks.s * kTTile);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_f16_ss_warp(t_s, kmajor_desc(qa, kk), kmajor_desc(ka, kk), idesc_s, kk > 0 ? 1u : 0u);
        if (two && lane == 0) mbar_arrive(&S.turn[1 - u]);
        umma_commit_warp(&S.s_full[u]);
      };
      auto release = [&](int slot, bool used) {
        if (used)
          umma_commit_warp(&S.empty[slot]);
        else if (lane == 0)
          mbar_arrive(&S.empty[slot]);
        __syncwarp();
      };
      if (ok) ok = wait(&S.full[ks.s], ks.phase);
      if (u == 1 && ok) ok = wait(&S.turn[1], 0u);
      if (ok && act(0))
        qk();
      else if (two && lane == 0)
        mbar_arrive(&S.turn[1 - u]);
      if (ok) release(ks.s, act(0));
      for (int j = 0; j < nt && ok; ++j) {
        const bool now = act(j), next = act(j + 1);
        ks.next();
        ok = wait(&S.full[vs.s], vs.phase);
        if (ok && j + 1 < nt) ok = wait(&S.full[ks.s], ks.phase);
        if (two && ok) ok = wait(&S.turn[u], (uint32_t)(u == 0 ? j : j + 1) & 1u);
        if (ok && now) ok = wait(&S.p_full[u][0], done & 1u);
        if (!ok) break;
        if (now) {
          tc_fence_after();
          const uint32_t va = kv_s + (uint32_t)(vs.s * kTTile);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_f16_ts_warp(t_o, t_s + (uint32_t)(8 * kk), mnmajor_desc(va, kk), idesc_pv,
                             (done > 0 || kk > 0) ? 1u : 0u);
          ok = wait(&S.p_full[u][1], done & 1u);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 4; kk < 8; ++kk)
            umma_f16_ts_warp(t_o, t_s + (uint32_t)(8 * kk), mnmajor_desc(va, kk), idesc_pv, 1u);
          ++done;
          umma_commit_warp(&S.pv_done[u]);
        }
        if (next) {
          if (done > 0) ok = wait(&S.pv_done[u], (done - 1u) & 1u);  // P is read, its columns free
          if (!ok) break;
          qk();
        } else {
          __syncwarp();
          if (two && lane == 0) mbar_arrive(&S.turn[1 - u]);
        }
        release(vs.s, now);
        if (j + 1 < nt) release(ks.s, next);
        vs.next();
      }
      // every UMMA issued has completed before tensor memory is freed
      umma_commit_warp(&S.mma_done[u]);
      mbar_wait(&S.mma_done[u], 0u, abort_flag, &g_attn_win_status, true);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------- softmax warps
    const int t = (warp - 4) >> 2;
    const int r = 32 * (warp & 3) + lane;  // row of the query tile = tensor-memory lane
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + lane_off + (uint32_t)(128 * t), t_o = tmem + lane_off + 256u + (uint32_t)(128 * t);
    const int64_t row = q0 + t * A.queries + r / G;  // this row's query
    const int64_t p = A.pos0 + row;
    const float scale = A.scale_log2e;
    const bool neg = scale < 0.f;
    float m = -INFINITY;
    uint64_t l2 = 0, l3 = 0;  // the row's sum, as four partial sums (short chains)
    bool ok = true;
    int n = 0;  // active tiles so far
    const Active act = actives(t);
    for (int j = 0; j < act.end && ok; ++j) {
      if (!act(j)) continue;
      // row p sees positions k0 + e of the tile with e < lim and (e >= from or e < sk)
      const int64_t k0 = tile_pos(j);
      const bool sink = j < sink_tiles;
      auto clamp = [](int64_t x) { return x >= kWK ? kWK : (x <= 0 ? 0 : (int)x); };
      const int lim = clamp((sink && A.sinks <= p ? A.sinks : p + 1) - k0);
      const int from = sink ? 0 : clamp(p - A.window + 1 - k0);
      const int sk = sink ? 0 : clamp(A.sinks - k0);
      const bool full = __all_sync(0xffffffffu, lim == kWK && from <= sk);
      ok = mbar_wait(&S.s_full[t], (uint32_t)n & 1u, abort_flag, &g_attn_win_status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t v[kWK];
#pragma unroll
      for (int c = 0; c < kWK / 16; ++c)
        tmem_ld16(t_s + (uint32_t)(16 * c), *reinterpret_cast<uint32_t(*)[16]>(v + 16 * c));
      tmem_wait_ld();
      if (!full) {  // hidden positions get the score that has weight 0 (and whatever was there is dropped)
        const uint32_t hidden = neg ? 0x7F800000u : 0xFF800000u;
#pragma unroll
        for (int c = 0; c < kWK / 32; ++c) {
          const uint32_t sees = bits_between(0, lim - 32 * c) &
                                (bits_between(from - 32 * c, 32) | bits_between(0, sk - 32 * c));
#pragma unroll
          for (int e = 0; e < 32; ++e) v[32 * c + e] = (sees >> e) & 1u ? v[32 * c + e] : hidden;
        }
      }
      // max_e(s_e * c) is c * max_e(s_e) for c >= 0 (rounding is monotonic) and c * min_e(s_e) for c < 0
      float ext[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) ext[c] = __uint_as_float(v[c]);
      if (!neg) {
#pragma unroll
        for (int e = 4; e < kWK; ++e) ext[e & 3] = fmaxf(ext[e & 3], __uint_as_float(v[e]));
        ext[0] = fmaxf(fmaxf(ext[0], ext[1]), fmaxf(ext[2], ext[3]));
      } else {
#pragma unroll
        for (int e = 4; e < kWK; ++e) ext[e & 3] = fminf(ext[e & 3], __uint_as_float(v[e]));
        ext[0] = fminf(fminf(ext[0], ext[1]), fminf(ext[2], ext[3]));
      }
      const float tmax = ext[0] * scale;
      // The reference m is 7 below the row's maximum and moves only when that
      // grows by more than 8: the weights 2^(s - m) then reach 2^15 (fp16 holds
      // them) and O is rescaled rarely; O and l use the same reference, so the
      // result is the same softmax.  The 7 keep small weights: fp16 drops what is
      // 2^-32 of the largest or less, where it dropped 2^-25, of which 2^17
      // positions hold 2^-8 of the sum.  A row that has seen nothing yet keeps
      // m = -inf, and its weights, all 0, are taken relative to 0.
      const bool upd = (m == -INFINITY && tmax != -INFINITY) || tmax > m + 15.0f;
      const float mn = upd ? tmax - 7.0f : m;
      const float corr = upd ? exp2f(m - mn) : 1.0f;
      m = mn;
      const float mref = m == -INFINITY ? 0.f : m;
      if (__any_sync(0xffffffffu, upd)) {
        float a, b;
        l2 = add2(l2, l3);
        l3 = 0;
        unpack2(l2, a, b);
        l2 = pack2(a * corr, b * corr);
        if (n > 0) {  // S was issued after the tile before was added to O
#pragma unroll 1
          for (int c = 0; c < kD / 16; ++c) {
            uint32_t w[16];
            tmem_ld16(t_o + (uint32_t)(16 * c), w);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * corr);
            tmem_st16(t_o + (uint32_t)(16 * c), w);
          }
        }
      }
      const uint64_t sc2 = pack2(scale, scale), mm2 = pack2(-mref, -mref);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int e0 = 64 * half + 32 * c;
          uint32_t hp[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float a, b;
            unpack2(fma2(pack2(__uint_as_float(v[e0 + e]), __uint_as_float(v[e0 + e + 1])), sc2, mm2), a, b);
            a = ex2_approx(a);
            b = ex2_approx(b);
            if (e & 2)
              l3 = add2(l3, pack2(a, b));
            else
              l2 = add2(l2, pack2(a, b));
            hp[e >> 1] = pack_h2(a, b);
          }
          tmem_st16(t_s + (uint32_t)(e0 / 2), hp);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_full[t][half]);
      }
      ++n;
    }
    if (ok && n > 0) ok = mbar_wait(&S.pv_done[t], (uint32_t)(n - 1) & 1u, abort_flag, &g_attn_win_status);
    ok = __all_sync(0xffffffffu, ok) && n > 0;
    float a, b;
    l2 = add2(l2, l3);
    unpack2(l2, a, b);
    if (A.split > 1) {
      // Every UMMA of both query tiles is done: their key and value tiles may go.
      named_bar_sync(1, 256u);
      asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(part_stat(S, t, r)), "f"(ok ? m : -INFINITY),
                   "f"(ok ? a + b : 0.f)
                   : "memory");
      if (ok) {
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < kD / 16; ++c) {
          uint32_t w[16];
          tmem_ld16(t_o + (uint32_t)(16 * c), w);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sts128_u(part_chunk(S, t, r, 4 * c + e), w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        }
      }
    } else if (ok) {
      tc_fence_after();
      const float inv = 1.0f / (a + b);
      const bool on = r < G * A.queries && row < A.M;
      __half* dst = A.out + (row * A.H + g * G + r % G) * kD;
      uint64_t check2 = 0;  // 0, or NaN from a product of 0 and a value that is not finite
#pragma unroll 1
      for (int c = 0; c < kD / 16; ++c) {
        uint32_t w[16], o[8];
        tmem_ld16(t_o + (uint32_t)(16 * c), w);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          check2 = fma2(pack2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1])), 0, check2);
          o[e] = pack_h2_finite(__uint_as_float(w[2 * e]) * inv, __uint_as_float(w[2 * e + 1]) * inv);
        }
        if (on) {
          uint4* d = reinterpret_cast<uint4*>(dst + 16 * c);
          d[0] = make_uint4(o[0], o[1], o[2], o[3]);
          d[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
      unpack2(check2, a, b);
      uint32_t again = __ballot_sync(0xffffffffu, on && !(a + b + inv * 0.f == 0.f));
      __syncwarp();
      for (; again; again &= again - 1) {
        const int rr = 32 * (warp & 3) + __ffs((int)again) - 1;
        attend_row(A, q0 + t * A.queries + rr / G, g * G + rr % G);
      }
    }
    __syncwarp();
  }
  if (A.split > 1) {
    __syncwarp();        // each warp arrives converged (the cluster barrier is .aligned)
    cluster_sync_all();  // every CTA's part is in its shared memory
    // A warp joins one row at a time, a lane four of its columns.
    for (int i = warp * A.split + rank; i < 256; i += kWWarps * A.split) {
      const int t = i >> 7, r = i & 127;
      const int64_t row = q0 + t * A.queries + r / G;
      if (r >= G * A.queries || row >= A.M) continue;
      float2 st[kWMaxSplit];
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < kWMaxSplit; ++c) {
        st[c] = make_float2(-INFINITY, 0.f);
        if (c < A.split) st[c] = ld_cluster2(mapa_shared(part_stat(S, t, r), (uint32_t)c));
        mx = fmaxf(mx, st[c].x);
      }
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < kWMaxSplit; ++c) {
        // It saw nothing of this row.  One that saw NaN alone has no maximum
        // either, but its sum is NaN, and so is the row's then.
        if (st[c].x == -INFINITY && st[c].y == 0.f) continue;
        const float w = exp2f(st[c].x - mx);
        const float4 v = ld_cluster4(mapa_shared(part_chunk(S, t, r, lane), (uint32_t)c));
        l = fmaf(w, st[c].y, l);
        o.x = fmaf(w, v.x, o.x);
        o.y = fmaf(w, v.y, o.y);
        o.z = fmaf(w, v.z, o.z);
        o.w = fmaf(w, v.w, o.w);
      }
      const float inv = 1.0f / l;
      if (__any_sync(0xffffffffu, !((o.x + o.y + o.z + o.w + inv) * 0.f == 0.f)))
        attend_row(A, row, g * G + r % G);
      else
        *reinterpret_cast<uint2*>(A.out + (row * A.H + g * G + r % G) * kD + 4 * lane) =
            make_uint2(pack_h2(within_half(o.x * inv), within_half(o.y * inv)),
                       pack_h2(within_half(o.z * inv), within_half(o.w * inv)));
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while its part is read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr size_t kWpSmem = sizeof(WpShared) + 1024;  // + alignment slack
static_assert(kWpSmem <= 227 * 1024, "shared memory of a CTA");

// How many clusters of `split` CTAs of the prefill kernel the device runs at
// once: a cluster lies within one GPC, so fewer than SMs / split.  Asked once per
// device and size; the kernel's attributes are set before.
int max_clusters(int split) {
  static std::atomic<int> known[kMaxDevices][kWMaxSplit + 1];
  const int dev = current_device();
  if (dev < 0) return 0;
  int n = known[dev][split].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split);
    cfg.blockDim = dim3(kWThreads);
    cfg.dynamicSmemBytes = kWpSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)split;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, attn_win_prefill_kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    n = n > 0 ? n : -1;  // -1: none
    known[dev][split].store(n, std::memory_order_relaxed);
  }
  return n;
}

cudaError_t launch_prefill(const uint16_t* q, const uint16_t* kc, const uint16_t* vc, uint16_t* out, int64_t M, int H,
                           int Hkv, int64_t pos0, int64_t Lmax, float scale, int64_t window, int64_t sinks,
                           cudaStream_t s) {
  const int G = H / Hkv;
  const int queries = 128 / G;
  const uint64_t qd[3] = {(uint64_t)kD, (uint64_t)H, (uint64_t)M};
  const uint64_t qs[2] = {(uint64_t)kRowBytes, (uint64_t)H * kRowBytes};
  const uint32_t qbox[3] = {64u, (uint32_t)G, (uint32_t)queries};
  const uint64_t strides[2] = {(uint64_t)kRowBytes, (uint64_t)Lmax * kRowBytes};
  const uint32_t box[3] = {64u, (uint32_t)kWK, 1u};
  // Maps over the caches' first rows: positions past them read as zero.
  auto encode = [&](CUtensorMap* tk, CUtensorMap* tv, int64_t rows) {
    const uint64_t dims[3] = {(uint64_t)kD, (uint64_t)rows, (uint64_t)Hkv};
    return encode_tensor_map_f16(tk, kc, 3, dims, strides, box, true) &&
           encode_tensor_map_f16(tv, vc, 3, dims, strides, box, true);
  };
  alignas(64) CUtensorMap tq, tk, tv, tks, tvs;
  if (!encode_tensor_map_f16(&tq, q, 3, qd, qs, qbox, true) || !encode(&tk, &tv, pos0 + M)) return cudaErrorInvalidValue;
  if (sinks > 0) {
    if (!encode(&tks, &tvs, sinks)) return cudaErrorInvalidValue;
  } else {
    tks = tk;
    tvs = tv;
  }
  static PerDeviceFlag attr_set;
  const int dev = current_device();
  if (!attr_set.done(dev)) {
    const cudaError_t e =
        cudaFuncSetAttribute(attn_win_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWpSmem);
    if (e != cudaSuccess) return e;
    attr_set.mark(dev);
  }
  // A scale of 0 (every visible position alike) must still tell hidden
  // positions, whose score is infinite, from visible ones.
  float sl2e = scale * 1.4426950408889634f;
  if (sl2e == 0.f) sl2e = 1e-37f;
  const int64_t nqb = (M + 2 * queries - 1) / (2 * queries);
  if (nqb * Hkv > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  // A cluster shares the work while all clusters run at once and each CTA has
  // two key tiles of the longest query tiles at least (the joining costs about
  // as much as one).  8 key/value heads, us with 1, 2, 4, 8 CTAs: 10 queries
  // after 15000 positions, window 2500: 36, 22, 14, 10; 128 after 8000, window
  // 2048: 39, 28, 19, 30 (16 clusters of 8 take two turns).
  const int64_t units = nqb * Hkv, span = std::min(window + 2 * queries, pos0 + M);
  const int64_t tiles = (std::min(sinks, pos0 + M - span) + kWK - 1) / kWK + (span + kWK - 1) / kWK;
  int split = 1;
  while (split < kWMaxSplit && tiles >= 4 * split && units <= max_clusters(2 * split)) split *= 2;
  // Pairs beyond whole rounds of the SMs that would fill at most half of another
  // go to a CTA for each query tile.  24 heads over 8, us with one CTA for a pair
  // and with one for each: 600 queries after 300, window 128 (64 pairs): 11.8,
  // 9.6; 2048 after 8000, window 2048 (200): 70.0, 64.8.
  const int64_t sms = device_sms(), over = units % sms;
  const int64_t singles = split == 1 && M > queries && 2 * over <= sms ? over : 0;
  const WpArgs A{reinterpret_cast<const __half*>(q),
                 reinterpret_cast<const __half*>(kc),
                 reinterpret_cast<const __half*>(vc),
                 reinterpret_cast<__half*>(out),
                 H,
                 Hkv,
                 G,
                 queries,
                 M,
                 pos0,
                 Lmax,
                 window,
                 sinks,
                 sl2e,
                 (unsigned)units,
                 (unsigned)(units - singles),
                 split};
  return launch_dependent(attn_win_prefill_kernel, dim3((unsigned)((units + singles) * split)), kWThreads, kWpSmem, (unsigned)split,
                          s, tq, tk, tv, tks, tvs, A);
}

}  // namespace

uint32_t attn_win_take_status() {
  uint32_t v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_attn_win_status, sizeof(v)) != cudaSuccess) return 0;
  cudaMemcpyToSymbol(g_attn_win_status, &zero, sizeof(zero));
  v |= take_debug_status();
  return v;
}

cudaError_t launch_gqa_attention_window(const uint16_t* q, const uint16_t* kc, const uint16_t* vc, uint16_t* out,
                                        int64_t M, int H, int Hkv, int64_t pos0, int64_t Lmax, float scale,
                                        int64_t window, int64_t sinks, cudaStream_t s) {
  if (window == 0 && sinks == 0) return cudaMemsetAsync(out, 0, (size_t)M * H * kRowBytes, s);  // nothing is visible
  const int64_t end = pos0 + M;
  if (window > end) window = end;
  if (sinks > end) sinks = end;
  if (M == 1) return launch_attn_window_decode(q, kc, vc, out, H, Hkv, pos0, Lmax, scale, window, sinks, s);
  return launch_prefill(q, kc, vc, out, M, H, Hkv, pos0, Lmax, scale, window, sinks, s);
}

}  // namespace qk
