// swiglu_device.cuh -- the logistic function in fp32 for the gated activation and its gradient.
#pragma once
#include "fp8_block_device.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float exp2_approx(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}

// 1 / (1 + 2^(-g log2(e))) in four instructions.  The exponent is off by 2^-23 |g| (its product and the constant),
// the approximations by 2^-22.5 and 2^-23 (PTX's bounds), the addition by 2^-24: below 2^-18 (relative) for |g| < 20,
// where sums of fp32 products of FP8 codes are no better.  A result below 2^-126 becomes 0.  (A Newton step on the
// reciprocal costs the activation's gradient 4 % and changes its codes' error by less than its own spread.)
__device__ __forceinline__ float sigmoid(float g) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + exp2_approx(g * -1.4426950408889634f)));
  return r;
}

// silu(g) u of two columns, whose logistic functions share a reciprocal, 1 / a = b / (a b): the special-function unit, 16
// lanes a clock, is what a tile's 16384 activations wait for.  The product stays finite up to exponents of t = 60.  FAR:
// there may be gates below kFarGate, or NaN; past 60 the logistic function is 2^-60 2^(60 - t) to within 2^-60 of itself,
// up to there the factor is 1 and a NaN's neighbour keeps its bits.  (Two selects in place of the factor: 148 bytes of
// spills a thread on pairs against 52.)
constexpr float kFarGate = -41.5f;  // t = 59.9
__device__ __forceinline__ float min_or_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <bool FAR>
__device__ __forceinline__ uint64_t gated2(uint64_t g, uint64_t u) {
  float t0, t1, a0, a1, r;
  apart(mul2(g, two(-1.4426950408889634f, -1.4426950408889634f)), t0, t1);
  apart(add2(two(exp2_approx(FAR ? fminf(t0, 60.0f) : t0), exp2_approx(FAR ? fminf(t1, 60.0f) : t1)), two(1.0f, 1.0f)),
        a0, a1);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a0 * a1));
  uint64_t s = mul2(two(r, r), two(a1, a0));
  if (FAR) s = mul2(s, two(exp2_approx(fminf(60.0f - t0, 0.0f)), exp2_approx(fminf(60.0f - t1, 0.0f))));
  return mul2(mul2(g, s), u);
}

}  // namespace
}  // namespace moe
