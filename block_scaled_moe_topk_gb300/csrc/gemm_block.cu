// gemm_block.cu -- the product in FP8 with a scale for each block of 128:
//   out[r, n] = sum_b sx[r, b] sw[e, n/128, b] sum_{c in block b} x[r, c] w[e, n, c]
// and its gradient with respect to the input, where the reduction runs over the weight's rows.
// Rows [offsets[e], offsets[e+1]) of x belong to expert e.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "expert_internal.h"

namespace moe {
namespace {

constexpr int kT = 64;  // tile: 64 rows x 64 output columns, 16 x 16 threads of 4 x 4

__device__ __forceinline__ float e4m3(uint8_t v) {
  __nv_fp8_e4m3 t;
  t.__x = v;
  return (float)t;
}

__device__ __forceinline__ void store_out(void* out, int dtype, int64_t i, float v) {
  if (dtype == kDtBf16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else if (dtype == kDtF16) static_cast<__half*>(out)[i] = __float2half_rn(v);
  else static_cast<float*>(out)[i] = v;
}

__global__ void __launch_bounds__(256) gemm_block_plain_kernel(GemmBlockArgs a) {
  __shared__ float xs[32][kT + 1], ws[32][kT + 1];
  if (blockIdx.x + blockIdx.y + blockIdx.z == 0 && threadIdx.x < 8) a.status[threadIdx.x] = 0;
  const int e = blockIdx.z;
  const int red = a.dgrad ? a.N : a.K, cols = a.dgrad ? a.K : a.N;
  const int64_t begin = a.offsets ? min(max(a.offsets[e], (int64_t)0), a.M) : 0;
  const int64_t end = a.offsets ? min(max(a.offsets[e + 1], begin), a.M) : a.M;
  const int n0 = blockIdx.x * kT, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int NB = (a.N + 127) / 128, KB = (a.K + 127) / 128, RB = (red + 127) / 128;
  const uint8_t* w = a.w + (int64_t)e * a.N * a.K;
  const float* wsc = a.w_scale + (int64_t)e * NB * KB;
  for (int64_t r0 = begin + (int64_t)blockIdx.y * kT; r0 < end; r0 += (int64_t)gridDim.y * kT) {
    float tot[4][4] = {};
    for (int b = 0; b < RB; ++b) {
      float acc[4][4] = {};
      for (int c0 = b * 128; c0 < min(red, b * 128 + 128); c0 += 32) {
        for (int i = threadIdx.x; i < 32 * kT; i += 256) {
          const int c = c0 + (i & 31), r = i >> 5;
          xs[i & 31][r] = r0 + r < end && c < red ? e4m3(a.x[(r0 + r) * red + c]) : 0.0f;
        }
        for (int i = threadIdx.x; i < 32 * kT; i += 256) {
          const int c = a.dgrad ? i / kT : i & 31, n = a.dgrad ? i % kT : i >> 5;
          const bool in = c0 + c < red && n0 + n < cols;
          ws[c][n] = in ? e4m3(a.dgrad ? w[(int64_t)(c0 + c) * a.K + n0 + n] : w[(int64_t)(n0 + n) * a.K + c0 + c]) : 0.0f;
        }
        __syncthreads();
        for (int c = 0; c < 32; ++c)
          for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[c][ty * 4 + i], ws[c][tx * 4 + j], acc[i][j]);
        __syncthreads();
      }
      for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + ty * 4 + i;
        if (r >= end) continue;
        const float sx = a.x_scale[r * RB + b];
        for (int j = 0; j < 4; ++j) {
          const int n = n0 + tx * 4 + j;
          if (n >= cols) continue;
          const float sw = a.dgrad ? wsc[b * KB + n / 128] : wsc[(n / 128) * KB + b];
          tot[i][j] = fmaf(acc[i][j], sx * sw, tot[i][j]);
        }
      }
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int64_t r = r0 + ty * 4 + i;
        const int n = n0 + tx * 4 + j;
        if (r < end && n < cols) store_out(a.out, a.out_dtype, r * cols + n, tot[i][j]);
      }
  }
}

}  // namespace

cudaError_t launch_gemm_block(const GemmBlockArgs& a, cudaStream_t s) {
  if (a.M == 0) return cudaSuccess;
  const int cols = a.dgrad ? a.K : a.N;
  const int64_t mt = (a.M + kT - 1) / kT;
  const dim3 grid((unsigned)((cols + kT - 1) / kT), (unsigned)std::min<int64_t>(mt, 64), (unsigned)a.E);
  gemm_block_plain_kernel<<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
