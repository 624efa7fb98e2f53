// qk_norm.cu -- RMSNorm in front of a linear, for the problems the GEMV does
// not take (M > 16, or a K it cannot stage): the normalized activations
//   xhat[m][k] = fp16( x[m][k] * r_m * gamma[k] ),  r_m = 1 / sqrt(mean_k x[m][k]^2 + eps)
// go to a caller-provided fp16 buffer that the tensor-core GEMM then reads.
// (The GEMV computes the same expression inside its x-table build.)
//
// Source: DAMASCUS project overview, "[04] one decode step" (an RMSNorm comes
// before the QKV projections and before the SwiGLU FFN); "Building DAMASCUS",
// "Read the model, then reproduce its operations".
//
// HBM-bound: one CTA per token row reads the row once (16-byte loads kept in
// registers), reduces the sum of squares in a fixed order (fp32, lane partials
// in k order, a shuffle tree, then the warps in order) and writes the row once.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "qk_device.cuh"
#include "qk_internal.h"

#ifndef QK_NORM_PER
#define QK_NORM_PER 2
#endif

namespace qk {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormChunks = 4;  // 8-value chunks per thread kept in registers: K <= 8192 in one pass

__device__ __forceinline__ float hlo(uint32_t v) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(v & 0xFFFFu)));
}

__device__ __forceinline__ uint32_t h2pack(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__global__ void __launch_bounds__(kNormThreads) rmsnorm_rows_kernel(const uint16_t* __restrict__ x,
                                                                     const uint16_t* __restrict__ gamma, float eps,
                                                                     uint16_t* __restrict__ out, int K) {
  __shared__ float wsum[kNormThreads / 32];
  __shared__ float r_sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t row = (size_t)blockIdx.x * (size_t)K;
  const int nc = K / 8;
  float ss = 0.f;
  uint4 v[kNormChunks];
  // first pass over the chunks this thread keeps (K <= 8 * 256 * kNormChunks)
#pragma unroll
  for (int i = 0; i < kNormChunks; ++i) {
    const int c = tid + i * kNormThreads;
    if (c < nc) {
      v[i] = ldg_stream16(x + row + 8 * c);
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = hlo(w[j]), b = hlo(w[j] >> 16);
        ss = fmaf(b, b, fmaf(a, a, ss));
      }
    }
  }
  // longer rows: the remaining chunks, read again in the second pass
  for (int c = tid + kNormChunks * kNormThreads; c < nc; c += kNormThreads) {
    const uint4 u = ldg_stream16(x + row + 8 * c);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = hlo(w[j]), b = hlo(w[j] >> 16);
      ss = fmaf(b, b, fmaf(a, a, ss));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (lane == 0) wsum[warp] = ss;
  __syncthreads();
  if (tid == 0) {
    float t = 0.f;
    for (int w = 0; w < kNormThreads / 32; ++w) t += wsum[w];
    r_sh = 1.0f / sqrtf(t / (float)K + eps);
  }
  __syncthreads();
  const float r = r_sh;
  auto emit = [&](int c, uint4 u) {
    const uint4 g = ldg_stream16(gamma + 8 * c);
    uint4 o;
    o.x = h2pack(hlo(u.x) * r * hlo(g.x), hlo(u.x >> 16) * r * hlo(g.x >> 16));
    o.y = h2pack(hlo(u.y) * r * hlo(g.y), hlo(u.y >> 16) * r * hlo(g.y >> 16));
    o.z = h2pack(hlo(u.z) * r * hlo(g.z), hlo(u.z >> 16) * r * hlo(g.z >> 16));
    o.w = h2pack(hlo(u.w) * r * hlo(g.w), hlo(u.w >> 16) * r * hlo(g.w >> 16));
    *reinterpret_cast<uint4*>(out + row + 8 * c) = o;
  };
#pragma unroll
  for (int i = 0; i < kNormChunks; ++i) {
    const int c = tid + i * kNormThreads;
    if (c < nc) emit(c, v[i]);
  }
  for (int c = tid + kNormChunks * kNormThreads; c < nc; c += kNormThreads) emit(c, ldg_stream16(x + row + 8 * c));
}

// ---------------------------------------------------------------------------
// Residual addition + RMSNorm
// ---------------------------------------------------------------------------
// h = residual + delta (fp32), residual_out = h in the residual's type, and
// xhat = fp16(h * r * gamma), r = 1 / sqrt(mean h^2 + eps), taken from the
// unrounded h; or xhat in int8 with a scale per 32 values.  One CTA per row: a
// thread keeps 8-value chunks of h in registers, so each input is read once
// (rows above 32768 values: the rest of them twice, the second time mostly from
// L2).  Many rows are bound by HBM: 2048 rows of 8192, fp32 residual, 43.5 us or
// 5.4 TB/s; 2048 of 4096, fp16 residual, 12 us.  One row of 4096 is latency:
// 1.9 us between calls of a graph.
struct AddNormArgs {
  const void* res;
  const float* delta;
  const uint16_t* gamma;
  void* res_out;
  uint16_t* xhat;
  int8_t* xq;
  float* xd;
  float eps;
  int K;
};

// 16-byte load that may read what this kernel also writes (the residual in
// place): not through the read-only path.
__device__ __forceinline__ uint4 ldg16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

template <bool F32>
__device__ __forceinline__ void load_h(const AddNormArgs& A, size_t at, float (&h)[8]) {
  if (F32) {
    const float* p = static_cast<const float*>(A.res) + at;
    const uint4 a = ldg16(p), b = ldg16(p + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = __uint_as_float(w[i]);
  } else {
    const uint4 a = ldg16(static_cast<const uint16_t*>(A.res) + at);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[2 * i] = hlo(w[i]);
      h[2 * i + 1] = hlo(w[i] >> 16);
    }
  }
  if (A.delta) {
    const uint4 a = ldg_stream16(A.delta + at), b = ldg_stream16(A.delta + at + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] += __uint_as_float(w[i]);
  }
}

// Writes one chunk: the residual, and the normalized values in fp16 or int8.
// Every lane of the warp calls this (the int8 scales are maxima over 4 lanes);
// `on` is false for lanes past the row's end.
template <bool F32, bool Q8>
__device__ __forceinline__ void emit_h(const AddNormArgs& A, size_t row, int c, bool on, const float (&h)[8], float r) {
  const size_t at = row + 8 * (size_t)c;
  uint32_t x[4] = {0u, 0u, 0u, 0u};
  if (on) {
    if (A.res_out) {
      if (F32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(A.res_out) + at);
        o[0] = make_float4(h[0], h[1], h[2], h[3]);
        o[1] = make_float4(h[4], h[5], h[6], h[7]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.res_out) + at) =
            make_uint4(h2pack(h[0], h[1]), h2pack(h[2], h[3]), h2pack(h[4], h[5]), h2pack(h[6], h[7]));
      }
    }
    const uint4 g = ldg_stream16(A.gamma + 8 * c);
    const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = h2pack(h[2 * i] * r * hlo(gw[i]), h[2 * i + 1] * r * hlo(gw[i] >> 16));
    if (!Q8) *reinterpret_cast<uint4*>(A.xhat + at) = make_uint4(x[0], x[1], x[2], x[3]);
  }
  if (Q8) {
    float v[8], a = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = hlo(x[i]);
      v[2 * i + 1] = hlo(x[i] >> 16);
      a = fmaxf(a, fmaxf(fabsf(v[2 * i]), fabsf(v[2 * i + 1])));
    }
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
    const float d = __fdiv_rn(a, 127.0f);
    if (on) {
      uint32_t q[2] = {0u, 0u};
      if (d != 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int b = (int)fminf(fmaxf(roundf(__fdiv_rn(v[i], d)), -127.0f), 127.0f);
          q[i >> 2] |= ((uint32_t)b & 0xFFu) << (8 * (i & 3));
        }
      }
      *reinterpret_cast<uint2*>(A.xq + at) = make_uint2(q[0], q[1]);
      if ((c & 3) == 0) A.xd[at / 32] = d;
    }
  }
}

constexpr int kAddNormThreads = 1024;  // at most

template <bool F32, bool Q8>
__global__ void __launch_bounds__(kAddNormThreads) add_rmsnorm_kernel(const __grid_constant__ AddNormArgs A) {
  __shared__ float wsum[kAddNormThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x;
  const size_t row = (size_t)blockIdx.x * (size_t)A.K;
  const int nc = A.K / 8;
  float h[kNormChunks][8];
  float ss = 0.f;
  dependent_wait();
#pragma unroll
  for (int i = 0; i < kNormChunks; ++i) {
    const int c = tid + i * T;
    if (c < nc) load_h<F32>(A, row + 8 * (size_t)c, h[i]);
  }
#pragma unroll
  for (int i = 0; i < kNormChunks; ++i) {
    if (tid + i * T < nc) {
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(h[i][e], h[i][e], ss);
    }
  }
  // longer rows: the remaining chunks, read again in the second pass (a thread
  // writes only chunks that it alone reads, after reading them: in place is fine)
  for (int c = tid + kNormChunks * T; c < nc; c += T) {
    float t[8];
    load_h<F32>(A, row + 8 * (size_t)c, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(t[e], t[e], ss);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (lane == 0) wsum[warp] = ss;
  __syncthreads();
  // every warp adds the warps' sums in the same tree
  float t = lane < T / 32 ? wsum[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const float r = 1.0f / sqrtf(t / (float)A.K + A.eps);
#pragma unroll
  for (int i = 0; i < kNormChunks; ++i) {
    const int c0 = i * T + 32 * warp;  // the warp's first chunk: the warp stays together
    if (c0 < nc) emit_h<F32, Q8>(A, row, c0 + lane, c0 + lane < nc, h[i], r);
  }
  for (int c0 = kNormChunks * T + 32 * warp; c0 < nc; c0 += T) {
    float u[8];
    if (c0 + lane < nc) load_h<F32>(A, row + 8 * (size_t)(c0 + lane), u);
    emit_h<F32, Q8>(A, row, c0 + lane, c0 + lane < nc, u, r);
  }
}

}  // namespace

cudaError_t launch_add_rmsnorm(const void* residual, bool f32, const float* delta, const uint16_t* gamma, float eps,
                               void* residual_out, uint16_t* xhat, int8_t* xq, float* xd, int64_t M, int64_t K,
                               cudaStream_t s) {
  const AddNormArgs A{residual, delta, gamma, residual_out, xhat, xq, xd, eps, (int)K};
  // Threads of a row: one 8-value chunk each where the rows are few (latency),
  // else QK_NORM_PER.  us with 1, 2, 4 chunks, fp32 residual: 1 row of 4096 2.35,
  // 2.64, 3.30; 300 rows of 4096 3.76, 4.63, 6.09; 2048 rows of 2048 9.2, 8.9,
  // 10.8, of 8192 55.1, 43.6, 42.9.
  const int64_t per = M <= 2 * (int64_t)device_sms() ? 1 : QK_NORM_PER;
  const int T = (int)std::min<int64_t>(kAddNormThreads, (K / 8 + 32 * per - 1) / (32 * per) * 32);
  auto kernel = xq ? (f32 ? add_rmsnorm_kernel<true, true> : add_rmsnorm_kernel<false, true>)
                   : (f32 ? add_rmsnorm_kernel<true, false> : add_rmsnorm_kernel<false, false>);
  return launch_dependent(kernel, dim3((unsigned)M), (unsigned)T, 0, 1, s, A);
}

// Scratch of qk_rmsnorm_matmul_batch_static, the entry point that allocates
// nothing: the normalized activations of the problems the tensor-core GEMM
// runs.  A file-scope array of fixed size that every GPU loading the library
// holds until the process exits; every call shares it.
static __device__ __align__(256) uint16_t g_static_scratch[kStaticScratchBytes / 2];

// The device address of g_static_scratch on the current device.  In host code
// the array's name is only a host-side stand-in, so its address comes from
// cudaGetSymbolAddress, once per device with that device current, and is kept.
cudaError_t static_scratch_address(void** out) {
  static std::atomic<void*> cache[kMaxDevices];
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  void* p = cache[dev].load(std::memory_order_acquire);
  if (!p) {
    const cudaError_t e = cudaGetSymbolAddress(&p, g_static_scratch);
    if (e != cudaSuccess) return e;
    cache[dev].store(p, std::memory_order_release);
  }
  *out = p;
  return cudaSuccess;
}

cudaError_t launch_rmsnorm_rows(const uint16_t* x, const uint16_t* gamma, float eps, uint16_t* out, int64_t M,
                                int64_t K, cudaStream_t s) {
  if (M <= 0) return cudaSuccess;
  if (M > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  rmsnorm_rows_kernel<<<(unsigned)M, kNormThreads, 0, s>>>(x, gamma, eps, out, (int)K);
  return cudaGetLastError();
}

}  // namespace qk
