// swiglu_device.cuh -- the logistic function in fp32 for the gated activation and its gradient.
#pragma once
#include <cstdint>

namespace moe {
namespace {

// 1 / (1 + 2^(-g log2(e))) in four instructions.  The exponent is off by 2^-23 |g| (its product and the constant),
// the approximations by 2^-22.5 and 2^-23 (PTX's bounds), the addition by 2^-24: below 2^-18 (relative) for |g| < 20,
// where sums of fp32 products of FP8 codes are no better.  A result below 2^-126 becomes 0.
__device__ __forceinline__ float sigmoid(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

}  // namespace
}  // namespace moe
