// gemm_block.cu -- the FP8 product with block scales and its gradient (gemm_block_kernel.cuh), and which form runs.
#include "gemm_block_kernel.cuh"

namespace moe {

cudaError_t launch_gemm_block(const GemmBlockArgs& a, cudaStream_t s) {
  if (a.M == 0) return cudaSuccess;
  if (use_gemv(a)) return launch_gemv_block(a, s);
  return a.dgrad ? launch_direction<kDgrad>(a, s) : launch_direction<kForward>(a, s);
}

}  // namespace moe
