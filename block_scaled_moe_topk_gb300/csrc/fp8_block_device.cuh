// fp8_block_device.cuh -- E4M3 codes with one fp32 scale per block of 128 columns: the scale, the
// rounding and the packing, for the quantiser and the kernels that quantise what they compute.
//
// The quotient 448 x / m is formed as q = x * (448 / m), at most 2^-23 (relative) off.  A 16-bit x and m have
// at most 11 significant bits, so 448 x / m either is a tie between two codes or lies 2^-16
// (relative) or more away from every tie; ties are frequent (about one element in 300 of bf16
// data).  Rounding q to 20 significant bits first (tie_snap: three fp32 operations) puts it back
// on the tie, so the codes are those of the exact quotient at a fifth of an IEEE division's
// instructions.  For fp32 x a quotient within 2^-20 of a tie may take either neighbour.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "expert_internal.h"

namespace moe {
namespace {

constexpr float kMaxE4m3 = 448.0f;

// q rounded to 20 significant bits (Veltkamp's splitting; the _rn forms are never fused).
__device__ __forceinline__ float tie_snap(float q) {
  const float c = __fmul_rn(q, 17.0f);
  return __fsub_rn(c, __fsub_rn(c, q));
}

struct BlockScale {
  float scale, mult;
};
__device__ __forceinline__ BlockScale block_scale(float m) {
  if (m < 7.888609052210118e-31f) return {0.0f, 0.0f};  // 2^-100
  return {__fdiv_rn(m, kMaxE4m3), __fdiv_rn(kMaxE4m3, m)};
}

__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a <= 3.402823466e38f ? a : 0.0f;  // false for NaN and infinities
}

// Two values -> two E4M3 bytes, the first in the low one.  The conversion saturates, so an infinity is
// turned into a NaN first and NaN stays NaN.
__device__ __forceinline__ uint32_t encode2(float x0, float x1, float mult) {
  float q0 = tie_snap(__fmul_rn(x0, mult)), q1 = tie_snap(__fmul_rn(x1, mult));
  if (!(fabsf(x0) <= 3.402823466e38f)) q0 = __int_as_float(0x7fffffff);
  if (!(fabsf(x1) <= 3.402823466e38f)) q1 = __int_as_float(0x7fffffff);
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q0, q1), __NV_SATFINITE, __NV_E4M3);
}

// N values -> N E4M3 bytes, element 0 in the lowest byte of w[0].
template <int N>
__device__ __forceinline__ void encode(const float* v, float mult, uint32_t (&w)[N / 4]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    w[i] = encode2(v[4 * i], v[4 * i + 1], mult) | (encode2(v[4 * i + 2], v[4 * i + 3], mult) << 16);
}

// ---- Values that a kernel has computed in fp32 and quantises at once.  They do not sit on ties more often than any
// number does, so their quotients are not put back on them: one within 2^-20 of a tie may take either neighbour, as for
// fp32 rows above.  The scales are the same, bit for bit.

// Two fp32 values in a register pair: one instruction on both is half the issue slots, which bound
// the elementwise kernels that quantise.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void apart(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The largest finite magnitude of N values, and whether one of any lane's is infinite: a NaN loses every comparison,
// so only then (a branch of the whole warp) are the values looked at one by one.
template <int N>
__device__ __forceinline__ float finite_max(const float* v, bool& infinite) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) m = fmaxf(m, fabsf(v[j]));
  infinite = __any_sync(0xffffffffu, m > 3.402823466e38f);
  if (infinite) {
    m = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) m = fmaxf(m, finite_abs(v[j]));
  }
  return m;
}

// m / 448 and 448 / m, rounded once, without divisions: a quotient is corrected by its remainder times the reciprocal
// (Markstein), for which the fused multiply-add leaves the remainder exact.  Right for every significand of m, by trial of
// all of them; 448 / m from a reciprocal one unit off was wrong for one of 2^23, by an ulp.  The reciprocal is that of
// m / 256, so that it is a normal number whatever the m, after one Newton step.  (Without the corrections 55 % of the scales
// were one unit off; every unit of error in the multiplier moves as many quotients again across a tie.)
__device__ __forceinline__ BlockScale computed_scale(float m) {
  constexpr float kInv = 1.0f / kMaxE4m3, kMult = kMaxE4m3 * 0.00390625f;
  const float d = m * 0.00390625f;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  r = fmaf(r, fmaf(-d, r, 1.0f), r);
  float mult = __fmul_rn(r, kMult), scale = __fmul_rn(m, kInv);
  mult = fmaf(fmaf(-d, mult, kMult), r, mult);
  scale = fmaf(fmaf(-kMaxE4m3, scale, m), kInv, scale);
  const bool tiny = m < 7.888609052210118e-31f;
  return {tiny ? 0.0f : scale, tiny ? 0.0f : mult};
}

// N values times mult -> E4M3 codes, element 0 in the lowest byte of w[0].  The conversion saturates, so infinities, of
// which finite_max told, become NaN first.
template <int N>
__device__ __forceinline__ void encode_computed(const float* v, float mult, bool infinite, uint32_t (&w)[(N + 3) / 4]) {
  if (infinite) {
    float t[N];
#pragma unroll
    for (int j = 0; j < N; ++j) t[j] = fabsf(v[j]) > 3.402823466e38f ? __int_as_float(0x7fffffff) : v[j] * mult;
#pragma unroll
    for (int i = 0; i < (N + 3) / 4; ++i) {
      w[i] = 0;
#pragma unroll
      for (int j = 4 * i; j < N && j < 4 * i + 4; ++j)
        w[i] |= ((uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(t[j], 0.0f), __NV_SATFINITE, __NV_E4M3) & 0xffu) << (8 * (j - 4 * i));
    }
    return;
  }
  const uint64_t m = two(mult, mult);
#pragma unroll
  for (int i = 0; i < (N + 3) / 4; ++i) {
    w[i] = 0;
#pragma unroll
    for (int j = 4 * i; j < N && j < 4 * i + 4; j += 2) {
      float q0, q1;
      apart(mul2(two(v[j], j + 1 < N ? v[j + 1] : 0.0f), m), q0, q1);
      w[i] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q0, q1), __NV_SATFINITE, __NV_E4M3) << (8 * (j - 4 * i));
    }
  }
}

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if (DT == kDtBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  if (DT == kDtF16) return __half2float(static_cast<const __half*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

}  // namespace
}  // namespace moe
