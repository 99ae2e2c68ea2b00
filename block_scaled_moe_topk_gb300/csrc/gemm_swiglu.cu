// gemm_swiglu.cu -- the gated FP8 product: both projections, h = silu(gate) up and its quantisation in one kernel
// (gemm_block_kernel.cuh; few rows: gemv_swiglu.cu).
//
// A tile has 128 columns of h.  Its 256 weight rows are loaded so that the first 64 accumulator columns of a half
// are gate and the next 64 the up columns that belong to them, whichever way the weights lie: the tensor map sees
// them as [E, I, 2, K] with the strides of either layout.  A summing thread then holds gate and up of the same 64
// columns of its row and forms h in registers.  The codes' blocks of 128 columns are two threads', which
// exchange their row's largest |h| through shared memory.
#include "gemm_block_kernel.cuh"

namespace moe {

cudaError_t launch_gemm_swiglu(const GemmBlockArgs& a, cudaStream_t s) {
  if (a.M == 0) return cudaSuccess;
  if (use_gemv_swiglu(a)) return launch_gemv_swiglu(a, s);
  return launch_direction<kGated>(a, s);
}

}  // namespace moe
