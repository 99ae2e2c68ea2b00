// rms_norm_fp8.cu -- the norm to FP8 codes with one fp32 scale per 1x128 block (rms_norm_kernel.cuh).
#include "rms_norm_kernel.cuh"

namespace moe {

cudaError_t launch_rms_norm_fp8(const NormArgs& a, cudaStream_t s) { return launch_quant<kQuantFp8Block>(a, s); }

}  // namespace moe
