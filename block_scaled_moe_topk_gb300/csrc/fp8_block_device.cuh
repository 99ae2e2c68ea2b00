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

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if (DT == kDtBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  if (DT == kDtF16) return __half2float(static_cast<const __half*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

}  // namespace
}  // namespace moe
