// swiglu_device.cuh -- the logistic function in fp32 for the gated activation and its gradient.
#pragma once

namespace moe {
namespace {

// 1 / (1 + exp(-g)), with the exponential of -|g| so that nothing overflows.  The fast exponential is documented to
// 2 + 1.173 |g| units in the last place, the fast division to 2: below 2^-18 (relative) for |g| < 20, where sums of
// fp32 products of FP8 codes are no better.
__device__ __forceinline__ float sigmoid(float g) {
  const float e = __expf(-fabsf(g)), r = __fdividef(1.0f, 1.0f + e);
  return g < 0.0f ? e * r : r;
}

}  // namespace
}  // namespace moe
