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
#include <cstdlib>

#include "norm_device.cuh"
#include "swiglu_device.cuh"

namespace moe {
namespace {

constexpr int kSwThreads = 256;

// du and dg of 8 columns, in place of u and g.
__device__ __forceinline__ void gradient8(const float (&dh)[8], float (&g)[8], float (&u)[8]) {
  const uint64_t one = two(1.0f, 1.0f), minus = two(-1.0f, -1.0f);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const uint64_t G = two(g[j], g[j + 1]), S = two(sigmoid(g[j]), sigmoid(g[j + 1]));
    const uint64_t a = mul2(two(dh[j], dh[j + 1]), S);
    const uint64_t bracket = fma2(G, fma2(S, minus, one), one);
    apart(mul2(mul2(a, two(u[j], u[j + 1])), bracket), g[j], g[j + 1]);
    apart(mul2(a, G), u[j], u[j + 1]);
  }
}

// Gate and up in turn -> codes; c: the first of a thread's 16 columns, of 2I.
__device__ __forceinline__ void put_pairs(const SwigluBackwardArgs& a, int64_t row, int c, bool on, const float (&dg)[8],
                                          const float (&du)[8]) {
  const int N = 2 * a.I, NB = (N + kFp8Block - 1) / kFp8Block;
  float v[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[2 * j] = dg[j], v[2 * j + 1] = du[j];
  bool infinite;
  const BlockScale sc = computed_scale(lanes_max(finite_max<16>(v, infinite), 8));
  uint32_t w[4];
  encode_computed<16>(v, sc.mult, infinite, w);
  if (!on || c >= N) return;
  *reinterpret_cast<uint4*>(a.codes + row * N + c) = make_uint4(w[0], w[1], w[2], w[3]);
  if ((c & (kFp8Block - 1)) == 0) a.scales[row * NB + c / kFp8Block] = sc.scale;
}

// The same for single elements: pair j of a lane at column 2 (c + 32 j); two j's are a block.
__device__ __forceinline__ void put_pairs_single(const SwigluBackwardArgs& a, int64_t row, int c, bool on,
                                                 const float (&dg)[8], const float (&du)[8]) {
  const int N = 2 * a.I, NB = (N + kFp8Block - 1) / kFp8Block;
#pragma unroll
  for (int j0 = 0; j0 < 8; j0 += 2) {
    const float v[4] = {dg[j0], du[j0], dg[j0 + 1], du[j0 + 1]};
    bool infinite;
    const BlockScale sc = computed_scale(lanes_max(finite_max<4>(v, infinite), 32));
    uint32_t w[1];
    encode_computed<4>(v, sc.mult, infinite, w);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int cj = 2 * (c + 32 * (j0 + j));
      if (!on || cj >= N) continue;
      a.codes[row * N + cj] = (uint8_t)(w[0] >> (16 * j));
      a.codes[row * N + cj + 1] = (uint8_t)(w[0] >> (16 * j + 8));
    }
    const int c0 = 2 * (c + 32 * j0);
    if (on && c0 < N && (c0 & (kFp8Block - 1)) == 0) a.scales[row * NB + c0 / kFp8Block] = sc.scale;
  }
}

// U groups of 8 columns of h a thread, all loaded before the first is used.
template <int DT, bool VEC, bool STACKED, int U>
__global__ void __launch_bounds__(kSwThreads, 1) swiglu_backward_kernel(const __grid_constant__ SwigluBackwardArgs a, int tpr) {
  const int I = a.I;
  const int64_t row = (int64_t)blockIdx.x * (kSwThreads / tpr) + threadIdx.x / tpr;
  const bool on = row < a.R;
  const ColumnMap<VEC> map(blockIdx.y * tpr * U + threadIdx.x % tpr, tpr);
  const int n = on ? I : 0;
  const int64_t base = row * a.gate_up_stride, dbase = row * a.d_gate_up_stride;
  float g[U][8], u[U][8], dh[U][8];
#pragma unroll
  for (int q = 0; q < U; ++q) {
    const int c = map.col(q);
    load8<DT, VEC>(a.dh, row * a.dh_stride, c, n, dh[q]);
    if (STACKED) {
      load8<DT, VEC>(a.gate_up, base, c, n, g[q]);
      load8<DT, VEC>(a.gate_up, base + I, c, n, u[q]);
    } else if (VEC) {
      float p[2][8];
      load8<DT, true>(a.gate_up, base, 2 * c, 2 * n, p[0]);
      load8<DT, true>(a.gate_up, base, 2 * c + 8, 2 * n, p[1]);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[q][j] = p[j >> 2][2 * (j & 3)], u[q][j] = p[j >> 2][2 * (j & 3) + 1];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = c + 32 * j < n;
        g[q][j] = in ? load1<DT>(a.gate_up, base + 2 * (c + 32 * j)) : 0.0f;
        u[q][j] = in ? load1<DT>(a.gate_up, base + 2 * (c + 32 * j) + 1) : 0.0f;
      }
    }
  }
#pragma unroll
  for (int q = 0; q < U; ++q) {
    const int c = map.col(q);
    gradient8(dh[q], g[q], u[q]);
    if (a.d_gate_up != nullptr) {
      if (STACKED) {
        store8<DT, VEC>(a.d_gate_up, dbase, c, n, g[q]);
        store8<DT, VEC>(a.d_gate_up, dbase + I, c, n, u[q]);
      } else if (VEC) {
        const float lo[8] = {g[q][0], u[q][0], g[q][1], u[q][1], g[q][2], u[q][2], g[q][3], u[q][3]};
        const float hi[8] = {g[q][4], u[q][4], g[q][5], u[q][5], g[q][6], u[q][6], g[q][7], u[q][7]};
        store8<DT, true>(a.d_gate_up, dbase, 2 * c, 2 * n, lo);
        store8<DT, true>(a.d_gate_up, dbase, 2 * c + 8, 2 * n, hi);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (c + 32 * j >= n) continue;
          const int64_t o = dbase + 2 * (c + 32 * j);
          if (DT == kDtF32) {
            static_cast<float*>(a.d_gate_up)[o] = g[q][j];
            static_cast<float*>(a.d_gate_up)[o + 1] = u[q][j];
          } else {
            const uint32_t pair = pack2<DT>(g[q][j], u[q][j]);
            static_cast<uint16_t*>(a.d_gate_up)[o] = (uint16_t)pair;
            static_cast<uint16_t*>(a.d_gate_up)[o + 1] = (uint16_t)(pair >> 16);
          }
        }
      }
    }
    if (a.codes == nullptr) continue;
    if (STACKED) {  // rows of I codes and I / 128 scales: row 2 r gate, 2 r + 1 up
      put_fp8<VEC>(a.codes, a.scales, 2 * row, I, c, on, g[q]);
      put_fp8<VEC>(a.codes, a.scales, 2 * row + 1, I, c, on, u[q]);
    } else if (VEC) {
      put_pairs(a, row, 2 * c, on, g[q], u[q]);
    } else {
      put_pairs_single(a, row, c, on, g[q], u[q]);
    }
  }
}

template <int DT, bool VEC, bool STACKED, int U>
cudaError_t launch_groups(const SwigluBackwardArgs& a, cudaStream_t s) {
  const int groups = VEC ? (a.I + 7) / 8 : (a.I + 255) / 256 * 32;
  int tpr = 32;  // whole warps: a block of 128 never crosses one
  while (tpr < kSwThreads && tpr * U < groups) tpr *= 2;
  const int rows = kSwThreads / tpr;
  const dim3 grid((unsigned)((a.R + rows - 1) / rows), (unsigned)((groups + tpr * U - 1) / (tpr * U)));
  swiglu_backward_kernel<DT, VEC, STACKED, U><<<grid, kSwThreads, 0, s>>>(a, tpr);
  return cudaGetLastError();
}

template <int DT, bool VEC, bool STACKED>
cudaError_t launch_layout(const SwigluBackwardArgs& a, cudaStream_t s) {
  if (getenv("X_U") && atoi(getenv("X_U")) == 1) return launch_groups<DT, VEC, STACKED, 1>(a, s);
  return launch_groups<DT, VEC, STACKED, 2>(a, s);
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
