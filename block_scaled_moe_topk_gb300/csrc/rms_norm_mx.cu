// rms_norm_mx.cu -- the norm to MX codes with one E8M0 scale per 1x32 block (rms_norm_kernel.cuh).
#include "rms_norm_kernel.cuh"

namespace moe {

cudaError_t launch_rms_norm_mx(const NormArgs& a, cudaStream_t s) { return launch_quant<kQuantMx>(a, s); }

}  // namespace moe
