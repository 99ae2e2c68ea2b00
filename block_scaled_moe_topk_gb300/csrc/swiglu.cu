// swiglu.cu -- gradient of the gated activation h = silu(g) u between the two products of a gated block:
//   du = dh silu(g),   dg = dh u sig(g) (1 + g (1 - sig(g)))
// for rows whose 2I columns hold gate and up in turn (2j gate, 2j + 1 up) or one after the other, leaving as
// FP8 codes with one fp32 scale per 1x128 block (of the 2I columns, as the next product's reduction reads
// them), as values, or both.  Elementwise but for the blocks' maxima, bound by HBM: 8 bytes in and out per h of 16-bit
// rows with codes (49152 x 2048: 127-128 us, 0.95 of the copy rate), with the issue slots 70 % used.
//
// A thread owns 8 columns of h and their 16 of gate and up: on 16-byte boundaries 8 consecutive ones, so
// that 8 lanes (in turn) or 16 (one after the other) hold a block.  Otherwise a warp owns spans of 256
// columns of h, element j of a lane at column 32 j + lane.
#include "norm_device.cuh"
#include "swiglu_device.cuh"

namespace moe {
namespace {

constexpr int kSwThreads = 256;
constexpr int64_t kSpreadGroups = 152 * 2 * kSwThreads;  // below, two groups a thread leave SMs idle

// dg and du of two columns.
__device__ __forceinline__ void gradient2(const float (&dh)[2], const float (&g)[2], const float (&u)[2], float* dg, float* du) {
  const uint64_t one = two(1.0f, 1.0f), minus = two(-1.0f, -1.0f);
  const uint64_t G = two(g[0], g[1]), S = two(sigmoid(g[0]), sigmoid(g[1]));
  const uint64_t a = mul2(two(dh[0], dh[1]), S);
  const uint64_t bracket = fma2(G, fma2(S, minus, one), one);
  apart(mul2(mul2(a, two(u[0], u[1])), bracket), dg[0], dg[1]);
  apart(mul2(a, G), du[0], du[1]);
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
template <int DT, bool VEC, bool STACKED, int U, int MINB>
__global__ void __launch_bounds__(kSwThreads, MINB) swiglu_backward_kernel(const __grid_constant__ SwigluBackwardArgs a, int tpr) {
  const int I = a.I;
  const int64_t row = (int64_t)blockIdx.x * (kSwThreads / tpr) + threadIdx.x / tpr;
  const bool on = row < a.R;
  const ColumnMap<VEC> map(blockIdx.y * tpr * U + threadIdx.x % tpr, tpr);
  const int n = on ? I : 0;
  const int64_t base = row * a.gate_up_stride, dbase = row * a.d_gate_up_stride;
  // VEC: dh, then gate and up one after the other, or their 16 columns in turn, as they lie in memory
  Raw8<DT> raw[U][3];
  float single[VEC ? 1 : U][3][8];
#pragma unroll
  for (int q = 0; q < U; ++q) {
    const int c = map.col(q);
    if constexpr (VEC) {
      raw[q][0] = raw8<DT>(a.dh, row * a.dh_stride, c, n);
      raw[q][1] = STACKED ? raw8<DT>(a.gate_up, base, c, n) : raw8<DT>(a.gate_up, base, 2 * c, 2 * n);
      raw[q][2] = STACKED ? raw8<DT>(a.gate_up, base + I, c, n) : raw8<DT>(a.gate_up, base + 8, 2 * c, 2 * n);
    } else {
      load8<DT, false>(a.dh, row * a.dh_stride, c, n, single[q][0]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = c + 32 * j < n;
        const int64_t o = STACKED ? base + c + 32 * j : base + 2 * (c + 32 * j);
        single[q][1][j] = in ? load1<DT>(a.gate_up, o) : 0.0f;
        single[q][2][j] = in ? load1<DT>(a.gate_up, o + (STACKED ? I : 1)) : 0.0f;
      }
    }
  }
#pragma unroll
  for (int q = 0; q < U; ++q) {
    const int c = map.col(q);
    float g[8], u[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float dh[2], gj[2], uj[2];
      if constexpr (VEC) {
        raw_pair<DT>(raw[q][0], j / 2, dh[0], dh[1]);
        if (STACKED) {
          raw_pair<DT>(raw[q][1], j / 2, gj[0], gj[1]);
          raw_pair<DT>(raw[q][2], j / 2, uj[0], uj[1]);
        } else {
          raw_pair<DT>(raw[q][1 + j / 4], j & 3, gj[0], uj[0]);
          raw_pair<DT>(raw[q][1 + j / 4], (j & 3) + 1, gj[1], uj[1]);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) dh[h] = single[q][0][j + h], gj[h] = single[q][1][j + h], uj[h] = single[q][2][j + h];
      }
      gradient2(dh, gj, uj, &g[j], &u[j]);
    }
    if (a.d_gate_up != nullptr) {
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
            const uint32_t pair = pack2<DT>(g[j], u[j]);
            static_cast<uint16_t*>(a.d_gate_up)[o] = (uint16_t)pair;
            static_cast<uint16_t*>(a.d_gate_up)[o + 1] = (uint16_t)(pair >> 16);
          }
        }
      }
    }
    if (a.codes == nullptr) continue;
    if (STACKED) {  // rows of I codes and I / 128 scales: row 2 r gate, 2 r + 1 up
      put_fp8<VEC>(a.codes, a.scales, 2 * row, I, c, on, g);
      put_fp8<VEC>(a.codes, a.scales, 2 * row + 1, I, c, on, u);
    } else if (VEC) {
      put_pairs(a, row, 2 * c, on, g, u);
    } else {
      put_pairs_single(a, row, c, on, g, u);
    }
  }
}

template <int DT, bool VEC, bool STACKED, int U, int MINB>
cudaError_t launch_groups(const SwigluBackwardArgs& a, cudaStream_t s) {
  const int groups = VEC ? (a.I + 7) / 8 : (a.I + 255) / 256 * 32;
  int tpr = 32;  // whole warps: a block of 128 never crosses one
  while (tpr < kSwThreads && tpr * U < groups) tpr *= 2;
  const int rows = kSwThreads / tpr;
  const dim3 grid((unsigned)((a.R + rows - 1) / rows), (unsigned)((groups + tpr * U - 1) / (tpr * U)));
  swiglu_backward_kernel<DT, VEC, STACKED, U, MINB><<<grid, kSwThreads, 0, s>>>(a, tpr);
  return cudaGetLastError();
}

template <int DT, bool VEC, bool STACKED>
cudaError_t launch_layout(const SwigluBackwardArgs& a, cudaStream_t s) {
  // Blocks an SM that the registers have to leave room for, and groups a thread.  bf16, codes, us (U = 1 with 4, 6, 8
  // blocks; U = 2 with 4, 5, 6): 49152 x 2048 142, 134, 130; 127, 125, 156; 12288 x 1152 31.0, 28.9, 28.3; 28.1, 26.5,
  // 28.7; 384 x 1152 2.8, 2.8, 2.7; 2.9, 3.1, 3.3.  fp32, 24576 x 2048 98, 100, 101; 101, 136, 169.
  // Single elements, 24576 x 2047 105, 101, 102; 166...
  constexpr int kBlocks = DT == kDtF32 ? 4 : VEC ? 8 : 6;
  if constexpr (VEC && DT != kDtF32) {
    if (a.R * ((a.I + 7) / 8) >= kSpreadGroups) return launch_groups<DT, VEC, STACKED, 2, 5>(a, s);
  }
  return launch_groups<DT, VEC, STACKED, 1, kBlocks>(a, s);
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
