// qk_rope.cuh -- the turns of one token's position, which the kernels that apply
// rotary positions share.
#pragma once

#include <cuda_runtime.h>

#include "qk_internal.h"

namespace qk {

namespace {

// Sine and cosine of every pair of the token at position p, times the magnitude,
// by `threads` threads.
__device__ __forceinline__ void fill_table(const RopeArgs& A, int64_t p, float2* cs, int threads) {
  for (int j = threadIdx.x; j < A.n_rot / 2; j += threads) {
    const double t = (double)p * A.inv_freq[j] * 0.15915494309189533577;  // turns
    float s, c;
    sincospif(2.0f * (float)(t - rint(t)), &s, &c);
    cs[j] = make_float2(c * A.magnitude, s * A.magnitude);
  }
}

}  // namespace

}  // namespace qk
