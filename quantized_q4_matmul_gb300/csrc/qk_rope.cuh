// qk_rope.cuh -- the turns of one token's position, which the kernels that apply
// rotary positions share.
#pragma once

#include <cuda_runtime.h>

#include "qk_internal.h"

namespace qk {

namespace {

// Cosine and sine of pair j of the token at position p, times the magnitude.
__device__ __forceinline__ float2 turn(const RopeArgs& A, int64_t p, int j) {
  const double t = (double)p * A.inv_freq[j] * 0.15915494309189533577;  // turns
  float s, c;
  sincospif(2.0f * (float)(t - rint(t)), &s, &c);
  return make_float2(c * A.magnitude, s * A.magnitude);
}

// Those of every pair, by `threads` threads.
__device__ __forceinline__ void fill_table(const RopeArgs& A, int64_t p, float2* cs, int threads) {
  for (int j = threadIdx.x; j < A.n_rot / 2; j += threads) cs[j] = turn(A, p, j);
}

}  // namespace

}  // namespace qk
