// gemv_swiglu.cu -- the gated FP8 product for a few rows (a token through a shared expert or a dense gated block):
//   h[r, j] = silu(g) u,  g = <x_r, gate row j>,  u = <x_r, up row j>  with the blocks' scales.
//
// As gemv_block.cu: one pass over the weights with plain 16-byte loads, no tensor core.  A warp owns the gate and the
// up row of one column of h, so both sums end in the same warp.  For codes the 128 columns of a block are a cluster
// of 16 blocks of 8 warps, whose row maxima meet in every block's shared memory: the grid stays as wide as without
// codes, where one block for 128 columns would leave most SMs idle.
#include <atomic>

#include "fp8_block_device.cuh"
#include "gemm_block_common.cuh"
#include "ptx.cuh"
#include "swiglu_device.cuh"

namespace moe {
namespace {

constexpr int kGsThreads = 256;
constexpr int kGsWarps = kGsThreads / 32;             // columns of h of a block
constexpr int kGsCluster = kFp8Block / kGsWarps;      // blocks of a scale block

// MR rows of x a pass (one expert: they share the weights), U column chunks in flight.
template <int MR, int U, bool CODES>
__global__ void __launch_bounds__(kGsThreads) gemv_swiglu_kernel(const __grid_constant__ GemmBlockArgs a) {
  __shared__ float warp_max[MR][kGsWarps], block_max[MR][kGsCluster];
  __shared__ int group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 8)
    a.status[threadIdx.x] = threadIdx.x == kFormWord ? kFormVector : 0;
  const int I = a.N / 2, j = blockIdx.x * kGsWarps + warp;
  const int64_t r0 = (int64_t)blockIdx.y * MR;
  int e = 0;
  if (a.offsets != nullptr) {  // the group that holds row r0
    if (threadIdx.x == 0) group = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < a.E; i += kGsThreads)
      if (r0 >= group_start(a.offsets, i, a.M) && r0 < group_start(a.offsets, i + 1, a.M)) group = i;
    __syncthreads();
    e = group;
    if (e < 0) return;  // the whole cluster has this row
  }
  const int K = a.K, KB = (K + kFp8Block - 1) / kFp8Block, NB = (a.N + kFp8Block - 1) / kFp8Block;
  const int ng = a.stacked ? j : 2 * j, nu = a.stacked ? I + j : 2 * j + 1;
  const uint8_t* wg = a.w + ((int64_t)e * a.N + ng) * K;
  const uint8_t* wu = a.w + ((int64_t)e * a.N + nu) * K;
  const float* sg = a.w_scale + ((int64_t)e * NB + ng / kFp8Block) * KB;
  const float* su = a.w_scale + ((int64_t)e * NB + nu / kFp8Block) * KB;
  const int end = j < I ? K : 0;
  float tot[MR][2] = {};
  for (int c0 = lane * 16; c0 < end; c0 += 512 * U) {
    uint4 wv[U][2], xv[U][MR];
    float s[U][MR][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + 512 * u;
      const bool in = c < K;
      wv[u][0] = in ? __ldcs(reinterpret_cast<const uint4*>(wg + c)) : make_uint4(0, 0, 0, 0);
      wv[u][1] = in ? __ldcs(reinterpret_cast<const uint4*>(wu + c)) : make_uint4(0, 0, 0, 0);
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
        for (int i = 0; i < 2; ++i) {
          float d = dot4(xv[u][m].x, wv[u][i].x, 0.0f);
          d = dot4(xv[u][m].y, wv[u][i].y, d);
          d = dot4(xv[u][m].z, wv[u][i].z, d);
          d = dot4(xv[u][m].w, wv[u][i].w, d);
          tot[m][i] = fmaf(d, s[u][m][i], tot[m][i]);
        }
  }
  float h[MR];
#pragma unroll
  for (int m = 0; m < MR; ++m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      tot[m][0] += __shfl_xor_sync(0xffffffffu, tot[m][0], o);
      tot[m][1] += __shfl_xor_sync(0xffffffffu, tot[m][1], o);
    }
    const float g = tot[m][0], u = tot[m][1];
    h[m] = g * sigmoid(g) * u;
    if (lane == 0 && j < I && r0 + m < a.M) {
      const int64_t row = r0 + m;
      if (a.out_dtype == kDtF32) {
        if (a.out != nullptr) static_cast<float*>(a.out)[row * I + j] = h[m];
        if (a.gate_up != nullptr) {
          static_cast<float*>(a.gate_up)[row * a.N + ng] = g;
          static_cast<float*>(a.gate_up)[row * a.N + nu] = u;
        }
      } else {
        if (a.out != nullptr) static_cast<uint16_t*>(a.out)[row * I + j] = (uint16_t)out_pair(h[m], 0.0f, a.out_dtype);
        if (a.gate_up != nullptr) {
          static_cast<uint16_t*>(a.gate_up)[row * a.N + ng] = (uint16_t)out_pair(g, 0.0f, a.out_dtype);
          static_cast<uint16_t*>(a.gate_up)[row * a.N + nu] = (uint16_t)out_pair(u, 0.0f, a.out_dtype);
        }
      }
    }
    if (CODES && lane == 0) warp_max[m][warp] = j < I ? finite_abs(h[m]) : 0.0f;
  }
  if (!CODES) return;
  __syncthreads();
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x < MR * kGsCluster) {  // this block's maximum of row m, to block `to` of the cluster
    const int m = threadIdx.x / kGsCluster, to = threadIdx.x % kGsCluster;
    float v = warp_max[m][0];
#pragma unroll
    for (int w = 1; w < kGsWarps; ++w) v = fmaxf(v, warp_max[m][w]);
    st_shared_cluster_f32(mapa_shared(smem_u32(&block_max[m][rank]), (uint32_t)to), v);
  }
  __syncwarp();
  cluster_sync();
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    float v = block_max[m][lane % kGsCluster];
#pragma unroll
    for (int o = kGsCluster / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    const BlockScale sc = computed_scale(v);
    if (lane != 0 || j >= I || r0 + m >= a.M) continue;
    a.codes[(r0 + m) * I + j] = (uint8_t)encode2(h[m], 0.0f, sc.mult);
    if (j % kFp8Block == 0) a.scales[(r0 + m) * ((I + kFp8Block - 1) / kFp8Block) + j / kFp8Block] = sc.scale;
  }
}

template <int MR, int U, bool CODES>
cudaError_t launch_rows(const GemmBlockArgs& a, cudaStream_t s) {
  const int I = a.N / 2, per = CODES ? kFp8Block : kGsWarps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((I + per - 1) / per * (per / kGsWarps)), (unsigned)((a.M + MR - 1) / MR));
  cfg.blockDim = dim3(kGsThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  if (CODES) {
    static std::atomic<int> ready[64];  // per device: clusters of 16 are allowed
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_acquire)) {
      err = cudaFuncSetAttribute(gemv_swiglu_kernel<MR, U, CODES>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (err != cudaSuccess) return err;
      ready[dev].store(1, std::memory_order_release);
    }
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kGsCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, gemv_swiglu_kernel<MR, U, CODES>, a);
}

template <bool CODES>
cudaError_t launch(const GemmBlockArgs& a, cudaStream_t s) {
  if (a.offsets != nullptr || a.M == 1) return launch_rows<1, 5, CODES>(a, s);
  if (a.M == 2) return launch_rows<2, 4, CODES>(a, s);
  return launch_rows<4, 2, CODES>(a, s);
}

}  // namespace

cudaError_t launch_gemv_swiglu(const GemmBlockArgs& a, cudaStream_t s) {
  return a.codes != nullptr ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace moe
