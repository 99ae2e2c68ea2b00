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
// HBM-bound: 16 lanes form a block of 128 columns, 8 columns each (one 16-byte load of 16-bit x),
// agree on m with four shuffles, and write 8 codes a lane to each of the row's destinations.
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

// Eight values -> eight E4M3 bytes, element 0 in the lowest byte.  The conversion saturates, so an
// infinity is turned into a NaN first (inf - inf) and NaN stays NaN.
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float mult) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float q[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float x = v[2 * i + h];
      q[h] = tie_snap(__fmul_rn(x, mult));
      if (!(fabsf(x) <= 3.402823466e38f)) q[h] = __int_as_float(0x7fffffff);
    }
    w[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if (DT == kDtBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  if (DT == kDtF16) return __half2float(static_cast<const __half*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

// Columns [c, c + 8) of a row of n columns starting at element `base`; columns past n read as 0.
// VEC: the row start is 16-byte aligned and n a multiple of 8.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* x, int64_t base, int c, int n, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  if (c >= n) return;
  if (VEC) {
    if (DT == kDtF32) {
      const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(x) + base + c);
      const float4 a = src[0], b = src[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + base + c);
      const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (DT == kDtBf16) {
          v[2 * i] = __uint_as_float(u[i] << 16);
          v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
          v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) v[i] = load1<DT>(x, base + c + i);
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(uint8_t* row, int c, int n, uint2 q) {
  if (c >= n) return;
  if (VEC) {
    *reinterpret_cast<uint2*>(row + c) = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
  }
}

struct QuantRowsParams {
  QuantBlockArgs a;
  int groups;  // 8-column groups of a row, padded to whole blocks
  int lg;      // log2 of the threads a row gets (at least 16)
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
  float v[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) load8<DT, VEC>(a.x, row * a.x_stride, on ? (g0 + u * tpr) * 8 : K, K, v[u]);
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
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int g = g0 + u * tpr;
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_abs(v[u][i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));  // the block's 16 lanes
    const BlockScale sc = block_scale(m);
    const uint2 q = encode8(v[u], sc.mult);
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
      if (dst[j] < 0) continue;
      store8<VEC>(a.codes + dst[j] * K, g * 8, K, q);
      if ((g & 15) == 0 && g * 8 < K) a.scales[dst[j] * KB + g / 16] = sc.scale;
    }
  }
}

// 128x128 blocks: one CTA per block, 16 rows at a time, values kept in registers.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kQbThreads) quant_tiles_kernel(QuantBlockArgs a) {
  __shared__ float part[kQbThreads / 32];
  const int64_t rb = blockIdx.x;
  const int cb = blockIdx.y, KB = gridDim.y;
  const int c = cb * kFp8Block + (threadIdx.x & 15) * 8;
  const int64_t r0 = rb * kFp8Block + (threadIdx.x >> 4);
  float v[8][8], m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    load8<DT, VEC>(a.x, r * a.x_stride, r < a.rows ? c : a.K, a.K, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int h = 0; h < 8; ++h) m = fmaxf(m, finite_abs(v[i][h]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQbThreads / 32; ++i) m = fmaxf(m, part[i]);
  const BlockScale sc = block_scale(m);
  if (threadIdx.x == 0) a.scales[rb * KB + cb] = sc.scale;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < a.rows) store8<VEC>(a.codes + r * a.K, c, a.K, encode8(v[i], sc.mult));
  }
}

template <int DT, bool VEC>
cudaError_t launch_typed(const QuantBlockArgs& a, cudaStream_t s) {
  if (a.block_rows == kFp8Block) {
    const dim3 grid((unsigned)((a.rows + kFp8Block - 1) / kFp8Block), (unsigned)((a.K + kFp8Block - 1) / kFp8Block));
    quant_tiles_kernel<DT, VEC><<<grid, kQbThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  constexpr int U = 2;
  QuantRowsParams p{a, (a.K + kFp8Block - 1) / kFp8Block * (kFp8Block / 8), 4};
  while (p.lg < 8 && (U << p.lg) < p.groups) ++p.lg;
  const int64_t per = kQbThreads >> p.lg;
  const dim3 grid((unsigned)((a.rows + per - 1) / per), (unsigned)((p.groups + (U << p.lg) - 1) / (U << p.lg)));
  quant_rows_block_kernel<DT, VEC, U><<<grid, kQbThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant_block(const QuantBlockArgs& a, cudaStream_t s) {
  if (a.rows == 0 || (a.inv != nullptr && a.R == 0)) return cudaSuccess;
  const int es = dtype_bytes(a.dtype);
  const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (a.x_stride * es) % 16 == 0 && a.K % 8 == 0 &&
                   reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
  if (a.dtype == kDtBf16) return vec ? launch_typed<kDtBf16, true>(a, s) : launch_typed<kDtBf16, false>(a, s);
  if (a.dtype == kDtF16) return vec ? launch_typed<kDtF16, true>(a, s) : launch_typed<kDtF16, false>(a, s);
  return vec ? launch_typed<kDtF32, true>(a, s) : launch_typed<kDtF32, false>(a, s);
}

}  // namespace moe
