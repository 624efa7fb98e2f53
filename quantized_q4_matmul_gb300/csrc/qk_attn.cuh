// qk_attn.cuh -- what the attention kernels share: head geometry, tile
// addressing, UMMA descriptors of the tiles, warp-level MMA helpers.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "qk_device.cuh"

namespace qk {

namespace {

constexpr int kD = 128;               // head dimension
constexpr int kRowBytes = kD * 2;     // one position of one head, fp16
constexpr int kMaxGroup = 8;          // query heads per key/value head


__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// 2^x with the hardware approximation (relative error about 2^-22, far below
// the fp16 rounding the weights get next; subnormal results flush to zero).
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// An average of fp16 values, in fp32, for its rounding to fp16: weights that are
// rounded one by one can carry it past the largest finite value, which the exact
// average never passes.  Infinities stay.
__device__ __forceinline__ float within_half(float x) {
  return fabsf(x) < INFINITY ? fminf(fmaxf(x, -65504.f), 65504.f) : x;
}

// The same in the rounding itself; infinities become the largest finite value.
__device__ __forceinline__ uint32_t pack_h2_finite(float a, float b) {
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %2, %1;" : "=r"(d) : "f"(a), "f"(b));
  return d;
}

constexpr int kTBox = 128 * 128;           // one 64-wide box of 128 rows of 128 bytes: 16 KB
constexpr int kTTile = 2 * kTBox;          // 32 KB: Q, one key or value tile, or P

// UMMA shared-memory descriptor of 16-wide K slice kk (0..7) of a K-major tile
// stored as two 64-wide boxes of 128 rows with the 128-byte swizzle.
__device__ __forceinline__ uint64_t kmajor_desc(uint32_t tile, int kk) {
  return umma_desc_sw128(tile + (uint32_t)((kk >> 2) * kTBox)) + (uint64_t)(2 * (kk & 3));
}

// The same for an MN-major operand (N contiguous): rows are K (positions) of
// 128 bytes = 64 N; the two 64-wide N atoms are kTBox apart (leading byte
// offset) and groups of 8 rows 1024 bytes apart (stride byte offset); slice kk
// starts 16 rows further on.
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t tile, int kk) {
  const uint32_t a = tile + (uint32_t)(kk * 16 * 128);
  uint64_t d = 0;
  d |= (uint64_t)((a & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kTBox >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

}  // namespace

}  // namespace qk
