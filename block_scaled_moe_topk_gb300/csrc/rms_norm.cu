// rms_norm.cu -- the norm whose result leaves as it is, and which form runs (rms_norm_kernel.cuh).
#include "rms_norm_kernel.cuh"

namespace moe {

cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  if (a.quant == kQuantFp8Block) return launch_rms_norm_fp8(a, s);
  if (a.quant == kQuantMx) return launch_rms_norm_mx(a, s);
  return launch_quant<kQuantNone>(a, s);
}

}  // namespace moe
