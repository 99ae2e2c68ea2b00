// gemm_swiglu.cu -- the gated FP8 product: both projections, h = silu(gate) up and its quantisation in one kernel
// (gemm_block_kernel.cuh; few rows: gemv_swiglu.cu).
//
// A tile has 128 columns of h.  Its 256 weight rows are loaded so that the first 64 accumulator columns of a half
// are gate and the next 64 the up columns that belong to them, whichever way the weights lie: the tensor map sees
// them as [E, I, 2, K] with the strides of either layout.  A summing thread then holds gate and up of the same 64
// columns of its row and forms h in registers.  The codes' blocks of 128 columns are two threads', which
// exchange their row's largest |h| through shared memory.
//
// What bounds it: with few rows the weight stream (64 tokens x 6 over 384 experts, I = 640, K = 5120, to codes: 248 us,
// 0.96 of the copy rate; 12288 rows over 128 experts, I = 1152, the products kept: 272-276 us, 0.90); with many, as the
// plain product of the same weights, the accumulator's round trip and the power limit (49152 rows over 48 experts, I =
// 2048, K = 7168: 1.21-1.32 ms, the plain product 1.21-1.30).  A tile's end adds 16384 activations, for which the
// special-function unit needs most of a microsecond: with K = 2048 405-408 us to codes, 378 to bf16 rows, plain 373 (of
// which 3-4 us look for gates that need more than a shared reciprocal).
#include "gemm_block_kernel.cuh"

namespace moe {

cudaError_t launch_gemm_swiglu(const GemmBlockArgs& a, cudaStream_t s) {
  if (a.M == 0) return cudaSuccess;
  if (use_gemv_swiglu(a)) return launch_gemv_swiglu(a, s);
  return launch_direction<kGated>(a, s);
}

}  // namespace moe
