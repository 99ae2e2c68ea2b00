// rms_norm.cu -- root-mean-square norm of rows with the residual's addition, leaving as it is, as FP8
// codes with a scale per block, or both:
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

// NCH chunks of 8 columns a thread; QF: how y is quantised.
template <int DT, bool VEC, int NCH, int QF, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) rms_norm_kernel(const __grid_constant__ NormParams p) {
  const NormArgs& a = p.a;
  const int H = a.H, tpr = p.tpr;
  const int rb = tpr >= (int)blockDim.x ? 0 : threadIdx.x / tpr;
  const int i = threadIdx.x - rb * tpr;  // this thread among the row's
  const int64_t row = (int64_t)blockIdx.x * p.rpb + rb;
  const bool on = rb < p.rpb && row < a.T;  // half a warp may be left over
  const ColumnMap<VEC> map(i, tpr);
  float v[NCH][8];
  float sq = 0.0f;
#pragma unroll
  for (int c = 0; c < NCH; ++c) load8<DT, VEC>(a.x, row * a.x_stride, map.col(c), on ? H : 0, v[c]);
  if (a.residual != nullptr) {
    float r[NCH][8];
#pragma unroll
    for (int c = 0; c < NCH; ++c) load8<DT, VEC>(a.residual, row * a.residual_stride, map.col(c), on ? H : 0, r[c]);
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
      store8<DT, VEC>(a.residual_out, row * a.residual_out_stride, map.col(c), on ? H : 0, v[c]);
  }
  sq = row_sum(sq, tpr, rb);
  const float rstd = __frsqrt_rn(sq / (float)H + a.eps);
  if (a.rstd != nullptr && on && i == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    float w[8];
    const int col = map.col(c);
    if (a.weight_dtype == DT) load8<DT, VEC>(a.weight, 0, col, H, w);
    else load8<kDtF32, VEC>(a.weight, 0, col, H, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[c][j] = v[c][j] * rstd * w[j];
    if (a.out != nullptr) store8<DT, VEC>(a.out, row * a.out_stride, col, on ? H : 0, v[c]);
    if (QF == kQuantFp8Block) put_fp8<VEC>(a.codes, static_cast<float*>(a.scales), row, H, col, on, v[c]);
    else if (QF == kQuantMx && a.mx_fmt == 0) put_mx<VEC, 0>(a.codes, static_cast<uint8_t*>(a.scales), row, H, col, on, v[c]);
    else if (QF == kQuantMx) put_mx<VEC, 1>(a.codes, static_cast<uint8_t*>(a.scales), row, H, col, on, v[c]);
  }
}

// One chunk a thread while the rows leave SMs idle (more threads in flight, less work behind the last
// load); else four (fewer threads to bring together a row), eight where four do not hold the row.
template <int DT, bool VEC, int QF>
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
  if (nch == 1) rms_norm_kernel<DT, VEC, 1, QF, 1024><<<grid, threads, 0, s>>>(p);
  else if (nch == 4) rms_norm_kernel<DT, VEC, 4, QF, 512><<<grid, threads, 0, s>>>(p);
  else rms_norm_kernel<DT, VEC, 8, QF, 512><<<grid, threads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int DT, int QF>
cudaError_t launch_quant(const NormArgs& a, bool vec, cudaStream_t s) {
  return vec ? launch_rows<DT, true, QF>(a, s) : launch_rows<DT, false, QF>(a, s);
}

template <int DT>
cudaError_t launch_typed(const NormArgs& a, bool vec, cudaStream_t s) {
  if (a.quant == kQuantNone) return launch_quant<DT, kQuantNone>(a, vec, s);
  if (a.quant == kQuantFp8Block) return launch_quant<DT, kQuantFp8Block>(a, vec, s);
  return launch_quant<DT, kQuantMx>(a, vec, s);
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const int64_t es = dtype_bytes(a.dtype);
  auto grid16 = [&](const void* q, int64_t stride) {
    return q == nullptr || (reinterpret_cast<uintptr_t>(q) % 16 == 0 && (a.T == 1 || stride * es % 16 == 0));
  };
  const bool vec = a.H % 8 == 0 && grid16(a.x, a.x_stride) && grid16(a.residual, a.residual_stride) &&
                   grid16(a.residual_out, a.residual_out_stride) && grid16(a.out, a.out_stride) &&
                   reinterpret_cast<uintptr_t>(a.weight) % 16 == 0 && reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
  if (a.dtype == kDtBf16) return launch_typed<kDtBf16>(a, vec, s);
  if (a.dtype == kDtF16) return launch_typed<kDtF16>(a, vec, s);
  return launch_typed<kDtF32>(a, vec, s);
}

}  // namespace moe
