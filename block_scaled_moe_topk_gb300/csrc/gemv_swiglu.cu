// gemv_swiglu.cu -- the gated FP8 product for a few rows (a token through a shared expert or a dense gated block):
//   h[r, j] = silu(g) u,  g = <x_r, gate row j>,  u = <x_r, up row j>  with the blocks' scales.
//
// As gemv_block.cu: one pass over the weights with plain 16-byte loads, no tensor core.  A warp owns the gate and the
// up row of one (or two) columns of h, so both sums end in the same warp.  For codes the 128 columns of a block are a
// cluster of 16 (or 8) blocks of 8 warps, whose row maxima meet in every block's shared memory: the grid stays as wide as
// without codes, where one block for 128 columns would leave most SMs idle.  Latency bounds it: one row, I = 1152, K =
// 5120 4.0 us, to codes 5.5-5.8 (the cluster's barrier; the plain product of the same weights 4.4).
#include <atomic>

#include "fp8_block_device.cuh"
#include "gemm_block_common.cuh"
#include "ptx.cuh"
#include "swiglu_device.cuh"

namespace moe {
namespace {

constexpr int kGsThreads = 256;
constexpr int kGsWarps = kGsThreads / 32;

// MR rows of x a pass (one expert: they share the weights), U column chunks in flight, C columns of h a warp.
template <int MR, int U, int C, bool CODES>
__global__ void __launch_bounds__(kGsThreads) gemv_swiglu_kernel(const __grid_constant__ GemmBlockArgs a) {
  constexpr int kCluster = kFp8Block / (kGsWarps * C);  // blocks of a scale block
  __shared__ float warp_max[MR][kGsWarps], block_max[MR][kCluster];
  __shared__ int group;
  // Every block of the cluster has to run before another one stores into its shared memory; the wait stands before those
  // stores, so that the loads hide it.
  if (CODES) cluster_arrive_relaxed();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 8)
    a.status[threadIdx.x] = threadIdx.x == kFormWord ? kFormVector : 0;
  const int I = a.N / 2, j0 = (blockIdx.x * kGsWarps + warp) * C;
  const int64_t r0 = (int64_t)blockIdx.y * MR;
  int e = 0;
  if (a.offsets != nullptr) {  // the group that holds row r0
    if (threadIdx.x == 0) group = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < a.E; i += kGsThreads)
      if (r0 >= group_start(a.offsets, i, a.M) && r0 < group_start(a.offsets, i + 1, a.M)) group = i;
    __syncthreads();
    e = group;
    if (e < 0) {  // the whole cluster has this row
      if (CODES) cluster_wait();
      return;
    }
  }
  const int K = a.K, KB = (K + kFp8Block - 1) / kFp8Block, NB = (a.N + kFp8Block - 1) / kFp8Block;
  // gate and up rows of the warp's columns; a warp's columns share their scales (C divides 64, and j0 C)
  int n[C][2];
#pragma unroll
  for (int q = 0; q < C; ++q) {
    n[q][0] = a.stacked ? j0 + q : 2 * (j0 + q);
    n[q][1] = a.stacked ? I + j0 + q : 2 * (j0 + q) + 1;
  }
  const uint8_t* w = a.w + (int64_t)e * a.N * K;
  const float* sg = a.w_scale + ((int64_t)e * NB + n[0][0] / kFp8Block) * KB;
  const float* su = a.w_scale + ((int64_t)e * NB + n[0][1] / kFp8Block) * KB;
  const int end = j0 < I ? K : 0;
  float tot[MR][C][2] = {};
  for (int c0 = lane * 16; c0 < end; c0 += 512 * U) {
    uint4 wv[U][C][2], xv[U][MR];
    float s[U][MR][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + 512 * u;
#pragma unroll
      for (int q = 0; q < C; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          wv[u][q][h] = c < K && j0 + q < I ? __ldcs(reinterpret_cast<const uint4*>(w + (int64_t)n[q][h] * K + c))
                                            : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + 512 * u, b = c / kFp8Block;
      const bool in = c < K;
      const float g = in ? sg[b] : 0.0f, v = in ? su[b] : 0.0f;
#pragma unroll
      for (int m = 0; m < MR; ++m) {
        const bool on = in && r0 + m < a.M;
        xv[u][m] = on ? *reinterpret_cast<const uint4*>(a.x + (r0 + m) * K + c) : make_uint4(0, 0, 0, 0);
        const float sx = on ? a.x_scale[(r0 + m) * KB + b] : 0.0f;
        s[u][m][0] = sx * g, s[u][m][1] = sx * v;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int q = 0; q < C; ++q)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float d = dot4(xv[u][m].x, wv[u][q][h].x, 0.0f);
            d = dot4(xv[u][m].y, wv[u][q][h].y, d);
            d = dot4(xv[u][m].z, wv[u][q][h].z, d);
            d = dot4(xv[u][m].w, wv[u][q][h].w, d);
            tot[m][q][h] = fmaf(d, s[u][m][h], tot[m][q][h]);
          }
  }
  float h[MR][C];
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    float largest = 0.0f;
#pragma unroll
    for (int q = 0; q < C; ++q) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        tot[m][q][0] += __shfl_xor_sync(0xffffffffu, tot[m][q][0], o);
        tot[m][q][1] += __shfl_xor_sync(0xffffffffu, tot[m][q][1], o);
      }
      const float g = tot[m][q][0], u = tot[m][q][1];
      h[m][q] = g * sigmoid(g) * u;
      if (j0 + q < I) largest = fmaxf(largest, finite_abs(h[m][q]));
      if (lane == 0 && j0 + q < I && r0 + m < a.M) {
        const int64_t at = (r0 + m) * I + j0 + q, at_g = (r0 + m) * a.N + n[q][0], at_u = (r0 + m) * a.N + n[q][1];
        if (a.out_dtype == kDtF32) {
          if (a.out != nullptr) static_cast<float*>(a.out)[at] = h[m][q];
          if (a.gate_up != nullptr) static_cast<float*>(a.gate_up)[at_g] = g, static_cast<float*>(a.gate_up)[at_u] = u;
        } else {
          if (a.out != nullptr) static_cast<uint16_t*>(a.out)[at] = (uint16_t)out_pair(h[m][q], 0.0f, a.out_dtype);
          if (a.gate_up != nullptr) {
            static_cast<uint16_t*>(a.gate_up)[at_g] = (uint16_t)out_pair(g, 0.0f, a.out_dtype);
            static_cast<uint16_t*>(a.gate_up)[at_u] = (uint16_t)out_pair(u, 0.0f, a.out_dtype);
          }
        }
      }
    }
    if (CODES && lane == 0) warp_max[m][warp] = largest;
  }
  if (!CODES) return;
  __syncthreads();
  cluster_wait();
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x < MR * kCluster) {  // this block's maximum of row m, to block `to` of the cluster
    const int m = threadIdx.x / kCluster, to = threadIdx.x % kCluster;
    float v = warp_max[m][0];
#pragma unroll
    for (int i = 1; i < kGsWarps; ++i) v = fmaxf(v, warp_max[m][i]);
    st_shared_cluster_f32(mapa_shared(smem_u32(&block_max[m][rank]), (uint32_t)to), v);
  }
  __syncwarp();
  cluster_sync();
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    float v = block_max[m][lane % kCluster];
#pragma unroll
    for (int o = kCluster / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    const BlockScale sc = computed_scale(v);
    if (lane != 0 || r0 + m >= a.M) continue;
#pragma unroll
    for (int q = 0; q < C; ++q) {
      uint32_t w[1];
      encode_computed<1>(&h[m][q], sc.mult, fabsf(h[m][q]) > 3.402823466e38f, w);
      if (j0 + q < I) a.codes[(r0 + m) * I + j0 + q] = (uint8_t)w[0];
    }
    if (j0 < I && j0 % kFp8Block == 0)
      a.scales[(r0 + m) * ((I + kFp8Block - 1) / kFp8Block) + j0 / kFp8Block] = sc.scale;
  }
}

template <int MR, int U, int C, bool CODES>
cudaError_t launch_rows(const GemmBlockArgs& a, cudaStream_t s) {
  constexpr int kCluster = kFp8Block / (kGsWarps * C);
  const int I = a.N / 2, per = CODES ? kFp8Block : kGsWarps * C;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((I + per - 1) / per * (per / (kGsWarps * C))), (unsigned)((a.M + MR - 1) / MR));
  cfg.blockDim = dim3(kGsThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  if (CODES) {
    if (kCluster > 8) {
      static std::atomic<int> ready[64];  // per device: clusters of 16 are allowed
      int dev = 0;
      cudaError_t err = cudaGetDevice(&dev);
      if (err != cudaSuccess) return err;
      if (dev >= 64) return cudaErrorInvalidDevice;
      if (!ready[dev].load(std::memory_order_acquire)) {
        err = cudaFuncSetAttribute(gemv_swiglu_kernel<MR, U, C, CODES>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (err != cudaSuccess) return err;
        ready[dev].store(1, std::memory_order_release);
      }
    }
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, gemv_swiglu_kernel<MR, U, C, CODES>, a);
}

// Two columns of h a warp make the clusters 8 blocks: faster from three grouped rows on (a cluster a row and 128
// columns), slower below (I = 1152, K = 5120, rows of 64 experts, one / two columns, us: 1 7.3 / 9.8, 2 9.3 / 10.6, 3
// 14.1 / 11.3, 4 16.2 / 12.5; dense, one row 5.5 / 5.7; values, one column: 3 rows 9.1, 4 13.2).
template <bool CODES>
cudaError_t launch(const GemmBlockArgs& a, cudaStream_t s) {
  if (CODES && a.offsets != nullptr && a.M > 2) return launch_rows<1, 5, 2, CODES>(a, s);
  if (a.offsets != nullptr || a.M == 1) return launch_rows<1, 5, 1, CODES>(a, s);
  if (a.M == 2) return launch_rows<2, 4, 1, CODES>(a, s);
  return launch_rows<4, 2, 1, CODES>(a, s);
}

}  // namespace

// As use_gemv; with codes the clusters and their barrier cost 1 to 5 us more, and the tiles with a split reduction
// take over earlier.  Vector form / tiles, us, dense rows to codes: I = 512, K = 2048: 1 3.4 / 8.4, 2 3.8 / 8.5, 4 5.6 /
// 8.8; I = 1152, K = 5120: 1 5.5 / 10.3, 2 8.1 / 10.2, 3 11.4 / 10.4, 4 11.8 / 10.3; I = 2048, K = 7168: 1 10.6 / 13.9,
// 2 16.4 / 14.1.
bool use_gemv_swiglu(const GemmBlockArgs& a) {
  if (!use_gemv(a)) return false;
  if (a.codes == nullptr || a.offsets != nullptr || a.M == 1) return true;
  return (int64_t)a.N * a.K <= (int64_t)1 << (a.M == 2 ? 24 : 23);
}

cudaError_t launch_gemv_swiglu(const GemmBlockArgs& a, cudaStream_t s) {
  return a.codes != nullptr ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace moe
