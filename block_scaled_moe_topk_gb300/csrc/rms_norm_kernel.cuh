// rms_norm_kernel.cuh -- root-mean-square norm of rows with the residual's addition, leaving as it is (rms_norm.cu),
// as FP8 codes with a scale per 1x128 block (rms_norm_fp8.cu) or as MX codes (rms_norm_mx.cu), or as both:
//   s = x + r,   rstd = 1 / sqrt(mean(s^2) + eps),   y = s rstd w
// and its gradients (rms_norm_backward.cu).  One pass: a row's sums stay in registers from the load to
// the output, so x and r are read once and s, y, the codes and the scales written once; it is bound by
// HBM for many rows and by launch latency for a few.
//
// The norm and the codes are those of the unrounded fp32 sum x + r; only what is written is rounded
// (s and y to the rows' type, y to codes straight from fp32).  The sum of squares is fp32.
//
// A row belongs to `tpr` threads of a block.  With rows on 16-byte boundaries a thread owns chunks of 8
// columns (one 16-byte access of 16-bit elements), so 16 lanes hold a 1x128 block and 4 lanes an MX
// block of 32.  Otherwise (VEC = false) a warp owns spans of 256 columns, element j of a lane at
// column 32 j + lane: single elements, but consecutive ones for consecutive lanes.
#pragma once
#include <algorithm>

#include "norm_device.cuh"

namespace moe {
namespace {

constexpr int kNormThreads = 256;  // of a block that holds several rows

struct NormParams {
  NormArgs a;
  int tpr;  // threads of a row: a power of two up to 32, or whole warps
  int rpb;  // rows of a block
};

// Rows on 16-byte boundaries: NCH chunks of 8 columns a thread; QF: how y is quantised.  Values are kept and multiplied
// in pairs (mul.f32x2 and its like): beside the quantiser the issue slots bound it as much as HBM does.
template <int DT, int NCH, int QF, bool RES, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) rms_norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int es = DT == kDtF32 ? 4 : 2;
  const NormArgs& a = p.a;
  const int H = a.H, tpr = p.tpr;
  const int rb = tpr >= (int)blockDim.x ? 0 : threadIdx.x / tpr;
  const int first = 8 * (threadIdx.x - rb * tpr), step = 8 * tpr;  // this thread's first column, its chunks' distance
  const int64_t row = (int64_t)blockIdx.x * p.rpb + rb;
  const bool on = rb < p.rpb && row < a.T;  // half a warp may be left over
  const int n = on ? H - first : 0;         // columns from the first on
  auto at = [&](const void* q, int64_t stride) {
    return static_cast<const uint8_t*>(q) + (on ? row * stride + first : 0) * es;
  };
  Raw8<DT> xr[NCH], rr[RES ? NCH : 1], wr[NCH];
  const uint8_t* xp = at(a.x, a.x_stride);
#pragma unroll
  for (int c = 0; c < NCH; ++c) xr[c] = raw8<DT>(xp, 0, c * step, n);
  if (RES) {
    const uint8_t* rp = at(a.residual, a.residual_stride);
#pragma unroll
    for (int c = 0; c < NCH; ++c) rr[RES ? c : 0] = raw8<DT>(rp, 0, c * step, n);
  }
  const bool same = DT == kDtF32 || a.weight_dtype == DT;  // an fp32 weight of 16-bit rows is loaded where it is used
  if (same) {
    const uint8_t* wp = static_cast<const uint8_t*>(a.weight) + (n > 0 ? first : 0) * es;
#pragma unroll
    for (int c = 0; c < NCH; ++c) wr[c] = raw8<DT>(wp, 0, c * step, n);
  }
  uint64_t v[NCH][4], sq = two(0.0f, 0.0f);
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[c][j] = raw_two<DT>(xr[c], j);
      if (RES) v[c][j] = add2(v[c][j], raw_two<DT>(rr[RES ? c : 0], j));
      sq = fma2(v[c][j], v[c][j], sq);
    }
  if (a.residual_out != nullptr) {
    uint8_t* sp = const_cast<uint8_t*>(at(a.residual_out, a.residual_out_stride));
#pragma unroll
    for (int c = 0; c < NCH; ++c) put8<DT>(sp, c * step, n, v[c]);
  }
  float s0, s1;
  apart(sq, s0, s1);
  const float rstd = __frsqrt_rn(row_sum(s0 + s1, tpr, rb) / (float)H + a.eps);
  if (a.rstd != nullptr && on && first == 0) a.rstd[row] = rstd;
  const uint64_t rstd2 = two(rstd, rstd);
  uint8_t* op = const_cast<uint8_t*>(at(a.out, a.out_stride));
  const int64_t code = on ? row * H + first : 0;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    if (same) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[c][j] = mul2(mul2(v[c][j], rstd2), raw_two<DT>(wr[c], j));
    } else {
      const Raw8<kDtF32> w = raw8<kDtF32>(a.weight, first, c * step, n);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[c][j] = mul2(mul2(v[c][j], rstd2), raw_two<kDtF32>(w, j));
    }
    if (a.out != nullptr) put8<DT>(op, c * step, n, v[c]);
    if constexpr (QF != kQuantNone) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) apart(v[c][j], y[2 * j], y[2 * j + 1]);
      if (QF == kQuantFp8Block)
        put_fp8_chunk(a.codes + code, static_cast<float*>(a.scales) + (on ? row : 0) * ((H + kFp8Block - 1) / kFp8Block),
                      first, c * step, n, y);
      else if (a.mx_fmt == 0) put_mx_chunk<0>(a.codes, static_cast<uint8_t*>(a.scales), code + c * step, c * step < n, y);
      else put_mx_chunk<1>(a.codes, static_cast<uint8_t*>(a.scales), code + c * step, c * step < n, y);
    }
  }
}

// Any other rows, element by element.
template <int DT, int NCH, int QF, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) rms_norm_single_kernel(const __grid_constant__ NormParams p) {
  const NormArgs& a = p.a;
  const int H = a.H, tpr = p.tpr;
  const int rb = tpr >= (int)blockDim.x ? 0 : threadIdx.x / tpr;
  const int i = threadIdx.x - rb * tpr;  // this thread among the row's
  const int64_t row = (int64_t)blockIdx.x * p.rpb + rb;
  const bool on = rb < p.rpb && row < a.T;
  const ColumnMap<false> map(i, tpr);
  float v[NCH][8];
  float sq = 0.0f;
#pragma unroll
  for (int c = 0; c < NCH; ++c) load8<DT, false>(a.x, row * a.x_stride, map.col(c), on ? H : 0, v[c]);
  if (a.residual != nullptr) {
    float r[NCH][8];
#pragma unroll
    for (int c = 0; c < NCH; ++c) load8<DT, false>(a.residual, row * a.residual_stride, map.col(c), on ? H : 0, r[c]);
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] += r[c][j];
  }
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) sq = fmaf(v[c][j], v[c][j], sq);
  if (a.residual_out != nullptr) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
      store8<DT, false>(a.residual_out, row * a.residual_out_stride, map.col(c), on ? H : 0, v[c]);
  }
  sq = row_sum(sq, tpr, rb);
  const float rstd = __frsqrt_rn(sq / (float)H + a.eps);
  if (a.rstd != nullptr && on && i == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    float w[8];
    const int col = map.col(c);
    if (a.weight_dtype == DT) load8<DT, false>(a.weight, 0, col, H, w);
    else load8<kDtF32, false>(a.weight, 0, col, H, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[c][j] = v[c][j] * rstd * w[j];
    if (a.out != nullptr) store8<DT, false>(a.out, row * a.out_stride, col, on ? H : 0, v[c]);
    if (QF == kQuantFp8Block) put_fp8<false>(a.codes, static_cast<float*>(a.scales), row, H, col, on, v[c]);
    else if (QF == kQuantMx && a.mx_fmt == 0) put_mx_single<0>(a.codes, static_cast<uint8_t*>(a.scales), row, H, col, on, v[c]);
    else if (QF == kQuantMx) put_mx_single<1>(a.codes, static_cast<uint8_t*>(a.scales), row, H, col, on, v[c]);
  }
}

// One chunk a thread while the rows leave SMs idle (more threads in flight, less work behind the last
// load); else four (fewer threads to bring together a row), eight where four do not hold the row.
template <int DT, bool VEC, int QF, bool RES>
cudaError_t launch_rows(const NormArgs& a, cudaStream_t s) {
  const int chunks = VEC ? (a.H + 7) / 8 : (a.H + 255) / 256 * 32;
  NormParams p{a, 0, 1};
  const int nch = chunks <= 32 || (a.T <= kSpreadRows && chunks <= 1024) ? 1 : chunks <= 4 * 512 ? 4 : 8;
  p.tpr = (chunks + nch - 1) / nch;
  if (VEC && p.tpr <= 16) p.tpr = 16;
  else p.tpr = (p.tpr + 31) / 32 * 32;
  p.rpb = std::max(1, kNormThreads / p.tpr);
  if (p.rpb > a.T) p.rpb = (int)a.T;
  const int threads = (p.tpr * p.rpb + 31) / 32 * 32;
  const unsigned grid = (unsigned)((a.T + p.rpb - 1) / p.rpb);
  if constexpr (VEC) {
    // Blocks an SM that the registers leave room for, 16-bit rows of up to 7168 columns; 8192 x 7168 bf16, us, with 1,
    // 4, 5, 6 blocks asked for: with residual 69.4, 69.0, 74, 117; to codes 69.9, 62.8, 75, 115; without residual
    // 45.9, 40.6, 38.0, 48; to codes 54, 47, 45, 60.  fp32, 4096 x 7168 with residual: 70.8, 93.
    constexpr int kBlocks = DT == kDtF32 ? 1 : RES || QF != kQuantNone ? 4 : 5;
    if constexpr (kBlocks > 1) {
      if (nch == 4 && threads <= 224) {
        rms_norm_kernel<DT, 4, QF, RES, 224, kBlocks><<<grid, threads, 0, s>>>(p);
        return cudaGetLastError();
      }
    }
    if (nch == 1) rms_norm_kernel<DT, 1, QF, RES, 1024, 1><<<grid, threads, 0, s>>>(p);
    else if (nch == 4) rms_norm_kernel<DT, 4, QF, RES, 512, 1><<<grid, threads, 0, s>>>(p);
    else rms_norm_kernel<DT, 8, QF, RES, 512, 1><<<grid, threads, 0, s>>>(p);
  } else {
    if (nch == 1) rms_norm_single_kernel<DT, 1, QF, 1024><<<grid, threads, 0, s>>>(p);
    else if (nch == 4) rms_norm_single_kernel<DT, 4, QF, 512><<<grid, threads, 0, s>>>(p);
    else rms_norm_single_kernel<DT, 8, QF, 512><<<grid, threads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

template <int DT, int QF>
cudaError_t launch_typed(const NormArgs& a, bool vec, cudaStream_t s) {
  if (!vec) return launch_rows<DT, false, QF, false>(a, s);
  return a.residual != nullptr ? launch_rows<DT, true, QF, true>(a, s) : launch_rows<DT, true, QF, false>(a, s);
}

template <int QF>
cudaError_t launch_quant(const NormArgs& a, cudaStream_t s) {
  const int64_t es = dtype_bytes(a.dtype);
  auto grid16 = [&](const void* q, int64_t stride) {
    return q == nullptr || (reinterpret_cast<uintptr_t>(q) % 16 == 0 && (a.T == 1 || stride * es % 16 == 0));
  };
  const bool vec = a.H % 8 == 0 && grid16(a.x, a.x_stride) && grid16(a.residual, a.residual_stride) &&
                   grid16(a.residual_out, a.residual_out_stride) && grid16(a.out, a.out_stride) &&
                   reinterpret_cast<uintptr_t>(a.weight) % 16 == 0 && reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
  if (a.dtype == kDtBf16) return launch_typed<kDtBf16, QF>(a, vec, s);
  if (a.dtype == kDtF16) return launch_typed<kDtF16, QF>(a, vec, s);
  return launch_typed<kDtF32, QF>(a, vec, s);
}

}  // namespace
}  // namespace moe
