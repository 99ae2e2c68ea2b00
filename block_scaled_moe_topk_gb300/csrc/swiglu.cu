// swiglu.cu -- gradient of the gated activation h = silu(g) u between the two products of a gated block:
//   du = dh silu(g),   dg = dh u sig(g) (1 + g (1 - sig(g)))
// for rows whose 2I columns hold gate and up in turn (2j gate, 2j + 1 up) or one after the other, leaving as
// FP8 codes with one fp32 scale per 1x128 block (of the 2I columns, as the next product's reduction reads
// them), as values, or both.  Elementwise but for the blocks' maxima, bound by HBM: 7 bytes in and out per
// h of 16-bit rows with codes.
//
// A thread owns 8 columns of h and their 16 of gate and up: on 16-byte boundaries 8 consecutive ones, so
// that 8 lanes (in turn) or 16 (one after the other) hold a block.  Otherwise a warp owns spans of 256
// columns of h, element j of a lane at column 32 j + lane.
#include <algorithm>

#include "norm_device.cuh"
#include "swiglu_device.cuh"

namespace moe {
namespace {

constexpr int kSwThreads = 256;

// 16 columns of gate and up in turn -> codes; c: the first, of N.
__device__ __forceinline__ void put_pairs(const SwigluBackwardArgs& a, int64_t row, int c, bool on, const float (&dg)[8],
                                          const float (&du)[8]) {
  const int N = 2 * a.I, NB = (N + kFp8Block - 1) / kFp8Block;
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(finite_abs(dg[j]), finite_abs(du[j])));
  const BlockScale sc = block_scale(lanes_max(m, 8));
  if (!on || c >= N) return;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = encode2(dg[2 * i], du[2 * i], sc.mult) | (encode2(dg[2 * i + 1], du[2 * i + 1], sc.mult) << 16);
  *reinterpret_cast<uint4*>(a.codes + row * N + c) = make_uint4(w[0], w[1], w[2], w[3]);
  if ((c & (kFp8Block - 1)) == 0) a.scales[row * NB + c / kFp8Block] = sc.scale;
}

// The same for single elements: pair j of a lane at column 2 (c + 32 j); two j's are a block.
__device__ __forceinline__ void put_pairs_single(const SwigluBackwardArgs& a, int64_t row, int c, bool on,
                                                 const float (&dg)[8], const float (&du)[8]) {
  const int N = 2 * a.I, NB = (N + kFp8Block - 1) / kFp8Block;
#pragma unroll
  for (int j0 = 0; j0 < 8; j0 += 2) {
    float m = 0.0f;
#pragma unroll
    for (int j = j0; j < j0 + 2; ++j) m = fmaxf(m, fmaxf(finite_abs(dg[j]), finite_abs(du[j])));
    const BlockScale sc = block_scale(lanes_max(m, 32));
#pragma unroll
    for (int j = j0; j < j0 + 2; ++j) {
      const int cj = 2 * (c + 32 * j);
      if (!on || cj >= N) continue;
      const uint32_t two = encode2(dg[j], du[j], sc.mult);
      a.codes[row * N + cj] = (uint8_t)two;
      a.codes[row * N + cj + 1] = (uint8_t)(two >> 8);
    }
    const int c0 = 2 * (c + 32 * j0);
    if (on && c0 < N && (c0 & (kFp8Block - 1)) == 0) a.scales[row * NB + c0 / kFp8Block] = sc.scale;
  }
}

// Codes of the gate's or the up projection's half of the row (I a multiple of 128).
template <bool VEC>
__device__ __forceinline__ void put_half(const SwigluBackwardArgs& a, int64_t row, int c, int half, bool on,
                                         const float (&v)[8]) {
  const int I = a.I;
  // rows of I codes and I / 128 scales: row 2 r + half of the halves
  put_fp8<VEC>(a.codes, a.scales, 2 * row + half, I, c, on, v);
}

template <int DT, bool VEC, bool STACKED, bool CODES>
__global__ void __launch_bounds__(kSwThreads) swiglu_backward_kernel(const __grid_constant__ SwigluBackwardArgs a, int tpr) {
  const int I = a.I;
  const int64_t row = (int64_t)blockIdx.x * (kSwThreads / tpr) + threadIdx.x / tpr;
  const bool on = row < a.R;
  const ColumnMap<VEC> map(blockIdx.y * tpr + threadIdx.x % tpr, 0);
  const int c = map.col(0), n = on ? I : 0;
  float g[8], u[8], dh[8];
  const int64_t base = row * a.gate_up_stride;
  load8<DT, VEC>(a.dh, row * a.dh_stride, c, n, dh);
  if (STACKED) {
    load8<DT, VEC>(a.gate_up, base, c, n, g);
    load8<DT, VEC>(a.gate_up, base + I, c, n, u);
  } else if (VEC) {
    float p[2][8];
    load8<DT, true>(a.gate_up, base, 2 * c, 2 * n, p[0]);
    load8<DT, true>(a.gate_up, base, 2 * c + 8, 2 * n, p[1]);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = p[j >> 2][2 * (j & 3)], u[j] = p[j >> 2][2 * (j & 3) + 1];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = c + 32 * j < n;
      g[j] = in ? load1<DT>(a.gate_up, base + 2 * (c + 32 * j)) : 0.0f;
      u[j] = in ? load1<DT>(a.gate_up, base + 2 * (c + 32 * j) + 1) : 0.0f;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float sig = sigmoid(g[j]);
    const float du = dh[j] * g[j] * sig;
    g[j] = dh[j] * u[j] * sig * (1.0f + g[j] * (1.0f - sig));
    u[j] = du;
  }
  if (a.d_gate_up != nullptr) {
    const int64_t dbase = row * a.d_gate_up_stride;
    if (STACKED) {
      store8<DT, VEC>(a.d_gate_up, dbase, c, n, g);
      store8<DT, VEC>(a.d_gate_up, dbase + I, c, n, u);
    } else if (VEC) {
      const float lo[8] = {g[0], u[0], g[1], u[1], g[2], u[2], g[3], u[3]};
      const float hi[8] = {g[4], u[4], g[5], u[5], g[6], u[6], g[7], u[7]};
      store8<DT, true>(a.d_gate_up, dbase, 2 * c, 2 * n, lo);
      store8<DT, true>(a.d_gate_up, dbase, 2 * c + 8, 2 * n, hi);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (c + 32 * j >= n) continue;
        const int64_t o = dbase + 2 * (c + 32 * j);
        if (DT == kDtF32) {
          static_cast<float*>(a.d_gate_up)[o] = g[j];
          static_cast<float*>(a.d_gate_up)[o + 1] = u[j];
        } else {
          const uint32_t two = pack2<DT>(g[j], u[j]);
          static_cast<uint16_t*>(a.d_gate_up)[o] = (uint16_t)two;
          static_cast<uint16_t*>(a.d_gate_up)[o + 1] = (uint16_t)(two >> 16);
        }
      }
    }
  }
  if (CODES) {
    if (STACKED) {
      put_half<VEC>(a, row, c, 0, on, g);
      put_half<VEC>(a, row, c, 1, on, u);
    } else if (VEC) {
      put_pairs(a, row, 2 * c, on, g, u);
    } else {
      put_pairs_single(a, row, c, on, g, u);
    }
  }
}

template <int DT, bool VEC, bool STACKED>
cudaError_t launch_layout(const SwigluBackwardArgs& a, cudaStream_t s) {
  const int groups = VEC ? (a.I + 7) / 8 : (a.I + 255) / 256 * 32;
  int tpr = 32;  // whole warps: a block of 128 never crosses one
  while (tpr < kSwThreads && tpr < groups) tpr *= 2;
  const int rows = kSwThreads / tpr;
  const dim3 grid((unsigned)((a.R + rows - 1) / rows), (unsigned)((groups + tpr - 1) / tpr));
  if (a.codes != nullptr) swiglu_backward_kernel<DT, VEC, STACKED, true><<<grid, kSwThreads, 0, s>>>(a, tpr);
  else swiglu_backward_kernel<DT, VEC, STACKED, false><<<grid, kSwThreads, 0, s>>>(a, tpr);
  return cudaGetLastError();
}

template <int DT>
cudaError_t launch_typed(const SwigluBackwardArgs& a, bool vec, cudaStream_t s) {
  if (a.stacked) return vec ? launch_layout<DT, true, true>(a, s) : launch_layout<DT, false, true>(a, s);
  return vec ? launch_layout<DT, true, false>(a, s) : launch_layout<DT, false, false>(a, s);
}

}  // namespace

cudaError_t launch_swiglu_backward(const SwigluBackwardArgs& a, cudaStream_t s) {
  if (a.R == 0) return cudaSuccess;
  const int64_t es = dtype_bytes(a.dtype);
  auto grid16 = [&](const void* q, int64_t stride) {
    return q == nullptr || (reinterpret_cast<uintptr_t>(q) % 16 == 0 && (a.R == 1 || stride * es % 16 == 0));
  };
  const bool vec = a.I % 8 == 0 && grid16(a.gate_up, a.gate_up_stride) && grid16(a.dh, a.dh_stride) &&
                   grid16(a.d_gate_up, a.d_gate_up_stride) && reinterpret_cast<uintptr_t>(a.codes) % 16 == 0;
  if (a.dtype == kDtBf16) return launch_typed<kDtBf16>(a, vec, s);
  if (a.dtype == kDtF16) return launch_typed<kDtF16>(a, vec, s);
  return launch_typed<kDtF32>(a, vec, s);
}

}  // namespace moe
