// swiglu_device.cuh -- the logistic function in fp32 for the gated activation and its gradient.
#pragma once
#include "fp8_block_device.cuh"

namespace moe {
namespace {

// 1 / (1 + 2^(-g log2(e))) in four instructions.  The exponent is off by 2^-23 |g| (its product and the constant),
// the approximations by 2^-22.5 and 2^-23 (PTX's bounds), the addition by 2^-24: below 2^-18 (relative) for |g| < 20,
// where sums of fp32 products of FP8 codes are no better.  A result below 2^-126 becomes 0.  (A Newton step on the
// reciprocal costs the activation's gradient 4 % and changes its codes' error by less than its own spread.)
__device__ __forceinline__ float sigmoid(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

// The same of two values with one reciprocal, 1 / a = b / (a b): the special-function unit, 16 lanes a clock, is what a
// tile's 16384 activations wait for.  Exponents are cut at 60 so that the product is finite: a gate below -41.6
// gets 2^-60.
__device__ __forceinline__ uint64_t sigmoid2(uint64_t g) {
  float t0, t1, a0, a1, r;
  apart(mul2(g, two(-1.4426950408889634f, -1.4426950408889634f)), t0, t1);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a0) : "f"(fminf(t0, 60.0f)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a1) : "f"(fminf(t1, 60.0f)));
  apart(add2(two(a0, a1), two(1.0f, 1.0f)), a0, a1);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a0 * a1));
  return mul2(two(r, r), two(a1, a0));
}

}  // namespace
}  // namespace moe
