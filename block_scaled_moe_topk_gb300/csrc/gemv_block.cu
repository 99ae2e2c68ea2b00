// gemv_block.cu -- the FP8 block-scaled product for a few rows (a token through a
// shared expert or a dense projection):
//   out[r, n] = sum_b sx[r, b] sw[e, n/128, b] sum_{c in block b} x[r, c] w[e, n, c].
//
// One pass over the weights with plain 16-byte loads: a warp owns two weight rows, a lane 16
// consecutive columns of every 512.  Those lie in one block, so a lane sums its 16 products in fp32
// (E4M3 to f16 pairs, exact, then mixed-precision multiply-adds), adds them to the row's total with
// one multiply-add by sx * sw, and the lanes' totals meet in five shuffles.  No tensor core: the call
// is over before a pipeline of tiles is set up.  Bound by latency below about 16 MB of weights, by HBM
// above.  One row, device time against the tiles of gemm_block.cu (with the reduction split over a
// cluster): N = 2304, K = 5120 3.7 against 10.1 us; N = 6144, K = 7168 8.9 against 14.4; N = 65536,
// K = 8192 90 (6.0 TB/s) against 119.  Each further row adds a multiply-add per weight and its own
// loads: two rows 5.5 against 10.2 us, four 7.3 against 9.9 (N = 2304) but 18.9 against 15.0 (N =
// 6144), hence the rule in use_gemv.  Grouped rows run one by one: three rows of 384 experts 6.7
// against 14.5 us, six of N = 6144 67 against 55.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "gemm_block_common.cuh"

namespace moe {
namespace {

constexpr int kGvThreads = 256;
constexpr int kGvRows = 2;  // weight rows of a warp

// acc + the products of 4 E4M3 pairs (a 32-bit word holds two pairs).
__device__ __forceinline__ float dot4(uint32_t a, uint32_t b, float acc) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw x = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(a >> (16 * h)), __NV_E4M3);
    const __half2_raw y = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(b >> (16 * h)), __NV_E4M3);
    asm("fma.rn.f32.f16 %0, %1, %2, %0;" : "+f"(acc) : "h"(x.x), "h"(y.x));
    asm("fma.rn.f32.f16 %0, %1, %2, %0;" : "+f"(acc) : "h"(x.y), "h"(y.y));
  }
  return acc;
}

// MR rows of x a pass (one expert: they share the weights), U column chunks in flight.
template <int MR, int U>
__global__ void __launch_bounds__(kGvThreads) gemv_block_kernel(GemmBlockArgs a) {
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 8)
    a.status[threadIdx.x] = threadIdx.x == kFormWord ? kFormVector : 0;
  const int n0 = (blockIdx.x * (kGvThreads / 32) + (threadIdx.x >> 5)) * kGvRows;
  const int64_t r0 = (int64_t)blockIdx.y * MR;
  int e = 0;
  if (a.offsets != nullptr) {
    // the group that holds row r0 (one thread finds it; the block looks at all groups at once)
    __shared__ int group;
    if (threadIdx.x == 0) group = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < a.E; i += kGvThreads)
      if (r0 >= group_start(a.offsets, i, a.M) && r0 < group_start(a.offsets, i + 1, a.M)) group = i;
    __syncthreads();
    e = group;
  }
  if (n0 >= a.N || e < 0) return;
  const int K = a.K, KB = (K + kFp8Block - 1) / kFp8Block, NB = (a.N + kFp8Block - 1) / kFp8Block;
  const uint8_t* w = a.w + ((int64_t)e * a.N + n0) * K;
  const bool two = n0 + 1 < a.N;  // an odd N leaves the last warp one row
  const float* sw = a.w_scale + ((int64_t)e * NB + n0 / kFp8Block) * KB;  // n0 is even: both rows' block
  float tot[MR][kGvRows] = {};
  for (int c0 = lane * 16; c0 < K; c0 += 512 * U) {
    uint4 wv[U][kGvRows], xv[U][MR];
    float s[U][MR];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + 512 * u;
      const bool in = c < K;
      wv[u][0] = in ? __ldcs(reinterpret_cast<const uint4*>(w + c)) : make_uint4(0, 0, 0, 0);
      wv[u][1] = in && two ? __ldcs(reinterpret_cast<const uint4*>(w + K + c)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + 512 * u;
      const bool in = c < K;
      const float swv = in ? sw[c / kFp8Block] : 0.0f;
#pragma unroll
      for (int m = 0; m < MR; ++m) {
        const bool on = in && r0 + m < a.M;
        xv[u][m] = on ? *reinterpret_cast<const uint4*>(a.x + (r0 + m) * K + c) : make_uint4(0, 0, 0, 0);
        s[u][m] = on ? a.x_scale[(r0 + m) * KB + c / kFp8Block] * swv : 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int i = 0; i < kGvRows; ++i) {
          float d = dot4(xv[u][m].x, wv[u][i].x, 0.0f);
          d = dot4(xv[u][m].y, wv[u][i].y, d);
          d = dot4(xv[u][m].z, wv[u][i].z, d);
          d = dot4(xv[u][m].w, wv[u][i].w, d);
          tot[m][i] = fmaf(d, s[u][m], tot[m][i]);
        }
  }
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int i = 0; i < kGvRows; ++i) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) tot[m][i] += __shfl_xor_sync(0xffffffffu, tot[m][i], o);
      if (lane == 0 && r0 + m < a.M && n0 + i < a.N) {
        const int64_t at = (r0 + m) * a.N + n0 + i;
        if (a.out_dtype == kDtF32) static_cast<float*>(a.out)[at] = tot[m][i];
        else static_cast<uint16_t*>(a.out)[at] = (uint16_t)out_pair(tot[m][i], 0.0f, a.out_dtype);
      }
    }
}

template <int MR, int U>
cudaError_t launch_rows(const GemmBlockArgs& a, cudaStream_t s) {
  constexpr int per = kGvThreads / 32 * kGvRows;
  const dim3 grid((unsigned)((a.N + per - 1) / per), (unsigned)((a.M + MR - 1) / MR));
  gemv_block_kernel<MR, U><<<grid, kGvThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

bool use_gemv(const GemmBlockArgs& a) {
  if (a.dgrad) return false;
  if (a.offsets != nullptr) return a.M <= 4;
  return a.M <= 2 || (a.M <= 4 && (int64_t)a.N * a.K <= (int64_t)1 << 24);
}

cudaError_t launch_gemv_block(const GemmBlockArgs& a, cudaStream_t s) {
  if (a.offsets != nullptr || a.M == 1) return launch_rows<1, 5>(a, s);
  if (a.M == 2) return launch_rows<2, 4>(a, s);
  return launch_rows<4, 2>(a, s);
}

}  // namespace moe
