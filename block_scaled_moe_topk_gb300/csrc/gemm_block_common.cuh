// gemm_block_common.cuh -- what the kernels of the FP8 block-scaled product share: rounding to the
// output type and the clamped row ranges of the groups.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "expert_internal.h"

namespace moe {
namespace {

// Two fp32 values as the bits of two elements of a 16-bit output type.
__device__ __forceinline__ uint32_t out_pair(float lo, float hi, int dtype) {
  if (dtype == kDtBf16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// First row of group e (e = E: the end of the last), inside [0, M] whatever the offsets hold.
// Group e has the rows from group_start(e) up to group_start(e + 1), none if that is less.
__device__ __forceinline__ int64_t group_start(const int64_t* offsets, int e, int64_t M) {
  if (offsets == nullptr) return e == 0 ? 0 : M;
  const int64_t v = offsets[e];
  return v < 0 ? 0 : (v > M ? M : v);
}

}  // namespace
}  // namespace moe
