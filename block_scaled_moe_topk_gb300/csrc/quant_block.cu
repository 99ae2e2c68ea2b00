// quant_block.cu -- rows to E4M3 codes with one fp32 scale per block of 128 columns (1x128, for
// activations) or of 128 rows by 128 columns (for weights).
//
// For a block with largest finite magnitude m: scale = m / 448, code = the E4M3 value nearest to
// 448 x / m, ties to the even code.  m < 2^-100 gives scale 0 and signed-zero codes; a non-finite
// x becomes the NaN code and leaves the block's scale to the finite elements.
//
// The quotient is formed as q = x * (448 / m), at most 2^-23 (relative) off.  A 16-bit x and m have
// at most 11 significant bits, so 448 x / m either is a tie between two codes or lies 2^-16
// (relative) or more away from every tie; ties are frequent (about one element in 300 of bf16
// data).  Rounding q to 20 significant bits first (tie_snap: three fp32 operations) puts it back
// on the tie, so the codes are those of the exact quotient at a fifth of an IEEE division's
// instructions.  For fp32 x a quotient within 2^-20 of a tie may take either neighbour.
//
// HBM-bound: 8 lanes form a block of 128 columns, 16 columns each (two 16-byte loads of 16-bit x),
// agree on m with three shuffles, and write 16 codes a lane to each of the row's destinations, one
// destination after the other.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "expert_internal.h"

namespace moe {
namespace {

constexpr int kQbThreads = 256;
constexpr float kMaxE4m3 = 448.0f;

// q rounded to 20 significant bits (Veltkamp's splitting; the _rn forms are never fused).
__device__ __forceinline__ float tie_snap(float q) {
  const float c = __fmul_rn(q, 17.0f);
  return __fsub_rn(c, __fsub_rn(c, q));
}

struct BlockScale {
  float scale, mult;
};
__device__ __forceinline__ BlockScale block_scale(float m) {
  if (m < 7.888609052210118e-31f) return {0.0f, 0.0f};  // 2^-100
  return {__fdiv_rn(m, kMaxE4m3), __fdiv_rn(kMaxE4m3, m)};
}

__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a <= 3.402823466e38f ? a : 0.0f;  // false for NaN and infinities
}

// 16 values -> 16 E4M3 bytes, element 0 in the lowest byte.  The conversion saturates, so an
// infinity is turned into a NaN first (inf - inf) and NaN stays NaN.
__device__ __forceinline__ uint4 encode16(const float (&v)[16], float mult) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float q[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float x = v[2 * i + h];
      q[h] = tie_snap(__fmul_rn(x, mult));
      if (!(fabsf(x) <= 3.402823466e38f)) q[h] = __int_as_float(0x7fffffff);
    }
    w[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16));
}

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if (DT == kDtBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  if (DT == kDtF16) return __half2float(static_cast<const __half*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

// Columns [c, c + 16) of a row of n columns starting at element `base`; columns past n read as 0.
// VEC: the row start is 16-byte aligned and n a multiple of 16.
template <int DT, bool VEC>
__device__ __forceinline__ void load16(const void* x, int64_t base, int c, int n, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  if (c >= n) return;
  if (VEC && DT == kDtF32) {
    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(x) + base + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = src[i];
      v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
    }
  } else if (VEC) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + base + c);
    const uint4 r0 = src[0], r1 = src[1];
    const uint32_t u[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (DT == kDtBf16) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c + i < n) v[i] = load1<DT>(x, base + c + i);
  }
}

template <bool VEC>
__device__ __forceinline__ void store16(uint8_t* row, int c, int n, uint4 q) {
  if (c >= n) return;
  if (VEC) {
    *reinterpret_cast<uint4*>(row + c) = q;
  } else {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c + i < n) row[c + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

struct QuantRowsParams {
  QuantBlockArgs a;
  int groups;  // 16-column groups of a row, padded to whole blocks
  int lg;      // log2 of the threads a row gets (at least 8)
};

// 1x128 blocks.  A row gets 2^lg threads of a block; thread i owns column groups i, i + 2^lg, ...
// (U of them, all loaded before the first is used).
template <int DT, bool VEC, int U>
__global__ void __launch_bounds__(kQbThreads) quant_rows_block_kernel(const __grid_constant__ QuantRowsParams p) {
  const QuantBlockArgs& a = p.a;
  const int tpr = 1 << p.lg, K = a.K;
  const int64_t row = (int64_t)blockIdx.x * (kQbThreads >> p.lg) + (threadIdx.x >> p.lg);
  const int g0 = blockIdx.y * (tpr * U) + (threadIdx.x & (tpr - 1));
  const bool on = row < a.rows;
  const int KB = (K + kFp8Block - 1) / kFp8Block;
  float v[U][16];
#pragma unroll
  for (int u = 0; u < U; ++u) load16<DT, VEC>(a.x, row * a.x_stride, on ? (g0 + u * tpr) * 16 : K, K, v[u]);
  int64_t dst[kMaxTopK];
  const int n = a.inv != nullptr ? a.k : 1;
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    dst[j] = -1;
    if (on && j < n) {
      const int64_t r = a.inv != nullptr ? (int64_t)a.inv[row * n + j] : row;
      if (r >= 0 && r < a.R) dst[j] = r;
    }
  }
  uint4 q[U];
  float scale[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, finite_abs(v[u][i]));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const BlockScale sc = block_scale(m);
    q[u] = encode16(v[u], sc.mult);
    scale[u] = sc.scale;
  }
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    if (dst[j] < 0) continue;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + u * tpr;
      store16<VEC>(a.codes + dst[j] * K, g * 16, K, q[u]);
      if ((g & 7) == 0 && g * 16 < K) a.scales[dst[j] * KB + g / 8] = scale[u];
    }
  }
}

// 128x128 blocks: one CTA per block, 32 rows at a time, values kept in registers.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kQbThreads) quant_tiles_kernel(QuantBlockArgs a) {
  __shared__ float part[kQbThreads / 32];
  const int64_t rb = blockIdx.x;
  const int cb = blockIdx.y, KB = gridDim.y;
  const int c = cb * kFp8Block + (threadIdx.x & 7) * 16;
  const int64_t r0 = rb * kFp8Block + (threadIdx.x >> 3);
  float v[4][16], m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 32 * i;
    load16<DT, VEC>(a.x, r * a.x_stride, r < a.rows ? c : a.K, a.K, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 16; ++h) m = fmaxf(m, finite_abs(v[i][h]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQbThreads / 32; ++i) m = fmaxf(m, part[i]);
  const BlockScale sc = block_scale(m);
  if (threadIdx.x == 0) a.scales[rb * KB + cb] = sc.scale;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 32 * i;
    if (r < a.rows) store16<VEC>(a.codes + r * a.K, c, a.K, encode16(v[i], sc.mult));
  }
}

// Two column groups a thread keep more loads in flight (T = 8192, K = 7168, k = 6: 79.8 against 83.9
// us, 0.89 of the copy rate); below four blocks of single groups an SM, spreading them over more SMs
// counts more (T = 64, K = 5120: 3.8 against 3.0 us).
constexpr int64_t kSpreadGroups = 152 * 4 * kQbThreads;

template <int DT, bool VEC, int U>
cudaError_t launch_rows_u(const QuantBlockArgs& a, int groups, cudaStream_t s) {
  QuantRowsParams p{a, groups, 3};
  while (p.lg < 8 && (U << p.lg) < p.groups) ++p.lg;
  const int64_t per = kQbThreads >> p.lg;
  const dim3 grid((unsigned)((a.rows + per - 1) / per), (unsigned)((p.groups + (U << p.lg) - 1) / (U << p.lg)));
  quant_rows_block_kernel<DT, VEC, U><<<grid, kQbThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int DT, bool VEC>
cudaError_t launch_typed(const QuantBlockArgs& a, cudaStream_t s) {
  if (a.block_rows == kFp8Block) {
    const dim3 grid((unsigned)((a.rows + kFp8Block - 1) / kFp8Block), (unsigned)((a.K + kFp8Block - 1) / kFp8Block));
    quant_tiles_kernel<DT, VEC><<<grid, kQbThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  const int groups = (a.K + kFp8Block - 1) / kFp8Block * (kFp8Block / 16);
  return a.rows * groups < kSpreadGroups ? launch_rows_u<DT, VEC, 1>(a, groups, s) : launch_rows_u<DT, VEC, 2>(a, groups, s);
}

}  // namespace

cudaError_t launch_quant_block(const QuantBlockArgs& a, cudaStream_t s) {
  if (a.rows == 0 || (a.inv != nullptr && a.R == 0)) return cudaSuccess;
  const int es = dtype_bytes(a.dtype);
  const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (a.x_stride * es) % 16 == 0 && a.K % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.codes) % 16 == 0;
  if (a.dtype == kDtBf16) return vec ? launch_typed<kDtBf16, true>(a, s) : launch_typed<kDtBf16, false>(a, s);
  if (a.dtype == kDtF16) return vec ? launch_typed<kDtF16, true>(a, s) : launch_typed<kDtF16, false>(a, s);
  return vec ? launch_typed<kDtF32, true>(a, s) : launch_typed<kDtF32, false>(a, s);
}

}  // namespace moe
