// rms_norm_kernel.cuh -- root-mean-square norm of rows with the residual's addition, leaving as it is (rms_norm.cu),
// as FP8 codes with a scale per 1x128 block (rms_norm_fp8.cu) or as MX codes (rms_norm_mx.cu), or as both:
//   s = x + r,   rstd = 1 / sqrt(mean(s^2) + eps),   y = s rstd w
// and its gradients (rms_norm_backward.cu).  One pass: a row's sums stay in registers from the load to
// the output, so x and r are read once and s, y, the codes and the scales written once; it is bound by
// HBM for many rows (8192 x 7168 bf16 with residual 70 us, to rows and MXFP8 codes 79, MXFP4 75: 0.99-1.00 of the copy
// rate) and by launch latency for a few (one row of 5120 2.5 us).  To codes alone without a residual (47 us, 0.57) 19
// instructions an element use 66 % of the issue slots, with 28 warps an SM that wait for loads, sums and conversions.
//
// The norm and the codes are those of the unrounded fp32 sum x + r; only what is written is rounded
// (s and y to the rows' type, y to codes straight from fp32).  The sum of squares is fp32.
//
// A row belongs to `tpr` threads of a block.  With rows on 16-byte boundaries a thread owns chunks of 8
// columns (one 16-byte access of 16-bit elements), so 16 lanes hold a 1x128 block and 4 lanes an MX
// block of 32.  Long 16-bit rows with a residual that start off those boundaries, all matrices' alike (contiguous ones of an
// odd width), are read and written the same way from the boundary below (SHIFT: a thread's columns then begin up to 7
// earlier, and the weight's are moved up to them in registers); for codes y passes through shared memory.  Other rows
// go element by element, a warp owning spans of 256 columns, element j of a lane at column 32 j + lane.
#pragma once
#include <algorithm>
#include <utility>

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
template <int DT, int NCH, int QF, bool RES, bool SHIFT, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) rms_norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int es = DT == kDtF32 ? 4 : 2, EP = 16 / es;
  const NormArgs& a = p.a;
  extern __shared__ float rows_y[];  // SHIFT with codes: y of the block's rows
  const int H = a.H, tpr = p.tpr;
  const int rb = tpr >= (int)blockDim.x ? 0 : threadIdx.x / tpr;
  const int64_t row = (int64_t)blockIdx.x * p.rpb + rb;
  const int shift = SHIFT ? (int)(row * a.x_stride % EP) : 0;  // elements from the 16-byte boundary to the row's first
  const int first = 8 * (int)(threadIdx.x - rb * tpr) - shift, step = 8 * tpr;  // first column, distance of the chunks
  const bool on = rb < p.rpb && row < a.T;  // half a warp may be left over
  const int n = on ? H - first : 0;         // columns from the first on, and how many of them are not the row's
  const int skip = SHIFT ? max(-first, 0) : 0;
  const int room = SHIFT && on ? n + (int)min((a.T - 1 - row) * H, (int64_t)8) : n;
  auto at = [&](const void* q, int64_t stride) {
    return static_cast<const uint8_t*>(q) + (on ? row * stride + first : 0) * es;
  };
  Raw8<DT> xr[NCH], rr[RES ? NCH : 1], wr[NCH];
  const uint8_t* xp = at(a.x, a.x_stride);
#pragma unroll
  for (int c = 0; c < NCH; ++c) xr[c] = row_chunk<DT, SHIFT>(xp, c * step, n, room);
  if (RES) {
    const uint8_t* rp = at(a.residual, a.residual_stride);
#pragma unroll
    for (int c = 0; c < NCH; ++c) rr[RES ? c : 0] = row_chunk<DT, SHIFT>(rp, c * step, n, room);
  }
  const bool same = DT == kDtF32 || a.weight_dtype == DT;  // an fp32 weight of 16-bit rows is loaded where it is used
  if (same) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) wr[c] = weight_chunk<DT, SHIFT>(a.weight, first + c * step, on ? H : 0, shift);
  }
  if constexpr (SHIFT) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
      if ((c == 0 && skip > 0) || c * step + 8 > n) {
        trim<DT>(xr[c], c == 0 ? skip : 0, n - c * step);
        if (RES) trim<DT>(rr[RES ? c : 0], c == 0 ? skip : 0, n - c * step);
      }
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
    for (int c = 0; c < NCH; ++c) put_chunk<DT, SHIFT>(sp, c * step, n, c == 0 ? skip : 0, v[c]);
  }
  float s0, s1;
  apart(sq, s0, s1);
  const float rstd = __frsqrt_rn(row_sum(s0 + s1, tpr, rb) / (float)H + a.eps);
  if (a.rstd != nullptr && on && first == -shift) a.rstd[row] = rstd;
  const uint64_t rstd2 = two(rstd, rstd);
  uint8_t* op = const_cast<uint8_t*>(at(a.out, a.out_stride));
  const int64_t code = on ? row * H + first : 0;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    if (same) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[c][j] = mul2(mul2(v[c][j], rstd2), raw_two<DT>(wr[c], j));
    } else {
      const Raw8<kDtF32> w = weight_chunk<kDtF32, SHIFT>(a.weight, first + c * step, on ? H : 0, shift);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[c][j] = mul2(mul2(v[c][j], rstd2), raw_two<kDtF32>(w, j));
    }
    if (a.out != nullptr) put_chunk<DT, SHIFT>(op, c * step, n, c == 0 ? skip : 0, v[c]);
    if constexpr (QF != kQuantNone && SHIFT) {  // the blocks of 128 columns do not begin where a thread does
      float* mine = rows_y + rb * H;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float lo, hi;
        apart(v[c][j / 2], lo, hi);
        const int col = first + c * step + j;
        if (on && col >= 0 && col < H) mine[col] = j & 1 ? hi : lo;
      }
    } else if constexpr (QF != kQuantNone) {
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
  if constexpr (QF != kQuantNone && SHIFT) {
    __syncthreads();
    // whole warps a row (tpr is a multiple of 32 here), 256 columns a time, element j of a lane at 32 j + lane
    const ColumnMap<false> map(threadIdx.x - rb * tpr, tpr);
    for (int c = map.col(0); c - (int)(threadIdx.x & 31) < H; c += step) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = on && c + 32 * j < H ? rows_y[rb * H + c + 32 * j] : 0.0f;
      put_fp8<false>(a.codes, static_cast<float*>(a.scales), row, H, c, on, y);
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

constexpr int kRowsBytes = 48 * 1024 - 32 * 4;  // of y in shared memory: a block's default limit less row_sum's 32 words
// Element by element, 20 M elements of bf16, four / one chunks a thread, us: without residual H = 499 42 / 29, 1501 34 /
// 29, 3001 34 / 32, 6001 33 / 49; to codes with residual 499 89 / 50, 1501 69 / 50, 3001 69 / 54, 6001 69 / 77.
constexpr int kSingleOnes = 512;  // chunks: 4096 columns

// One chunk a thread up to `ones` chunks a row, and while the rows leave SMs idle (more threads in flight, less work behind
// the last load); else four (fewer threads to bring together a row), eight where four do not hold the row.
NormParams shape_of(const NormArgs& a, int chunks, int ones, bool whole_warps, int* nch, int* threads, unsigned* grid) {
  NormParams p{a, 0, 1};
  *nch = chunks <= ones || (a.T <= kSpreadRows && chunks <= 1024) ? 1 : chunks <= 4 * 512 ? 4 : 8;
  p.tpr = (chunks + *nch - 1) / *nch;
  if (!whole_warps && p.tpr <= 16) p.tpr = 16;
  else p.tpr = (p.tpr + 31) / 32 * 32;
  p.rpb = std::max(1, kNormThreads / p.tpr);
  if (p.rpb > a.T) p.rpb = (int)a.T;
  *threads = (p.tpr * p.rpb + 31) / 32 * 32;
  *grid = (unsigned)((a.T + p.rpb - 1) / p.rpb);
  return p;
}

template <int DT, int QF, bool RES, bool SHIFT>
cudaError_t launch_chunks(const NormArgs& a, cudaStream_t s) {
  int nch, threads;
  unsigned grid;
  const bool rows = SHIFT && QF != kQuantNone;
  const NormParams p = shape_of(a, (a.H + (SHIFT ? 16 / dtype_bytes(DT) - 1 : 0) + 7) / 8, 32, rows, &nch, &threads, &grid);
  const size_t smem = rows ? (size_t)p.rpb * a.H * 4 : 0;
  // Blocks an SM that the registers leave room for, where a block has up to 224 threads (16-bit rows of 4097 to 7168
  // columns; narrower ones mostly fill 256 threads with several rows); 8192 x 7168 bf16, us, with 1, 4, 5, 6 blocks
  // asked for: with residual 69.4, 69.0, 74, 117; to codes 69.9, 62.8, 75, 115; without residual 45.9, 40.6, 38.0, 48;
  // to codes 54, 47, 45, 60.  fp32, 4096 x 7168 with residual: 70.8, 93.  Blocks of 256 threads and more run with one
  // asked for: 8192 x 4096 41 us with residual (0.97 of the copy rate), 27 without (0.73), 8192 x 8192 78 and 75 to codes.
  constexpr int kBlocks = DT == kDtF32 ? 1 : SHIFT ? 3 : RES || QF != kQuantNone ? 4 : 5;
  if constexpr (kBlocks > 1) {
    if (nch == 4 && threads <= 224) {
      rms_norm_kernel<DT, 4, QF, RES, SHIFT, 224, kBlocks><<<grid, threads, smem, s>>>(p);
      return cudaGetLastError();
    }
  }
  if (nch == 1) rms_norm_kernel<DT, 1, QF, RES, SHIFT, 1024, 1><<<grid, threads, smem, s>>>(p);
  else if (nch == 4) rms_norm_kernel<DT, 4, QF, RES, SHIFT, 512, 1><<<grid, threads, smem, s>>>(p);
  else if constexpr (!SHIFT) rms_norm_kernel<DT, 8, QF, RES, SHIFT, 512, 1><<<grid, threads, smem, s>>>(p);
  return cudaGetLastError();
}

template <int DT, int QF>
cudaError_t launch_single(const NormArgs& a, cudaStream_t s) {
  int nch, threads;
  unsigned grid;
  const NormParams p = shape_of(a, (a.H + 255) / 256 * 32, kSingleOnes, true, &nch, &threads, &grid);
  if (nch == 1) rms_norm_single_kernel<DT, 1, QF, 1024><<<grid, threads, 0, s>>>(p);
  else if (nch == 4) rms_norm_single_kernel<DT, 4, QF, 512><<<grid, threads, 0, s>>>(p);
  else rms_norm_single_kernel<DT, 8, QF, 512><<<grid, threads, 0, s>>>(p);
  return cudaGetLastError();
}

// `vec`: rows of whole chunks on 16-byte boundaries; `shifted`: their boundaries are passed at the same elements.
template <int DT, int QF>
cudaError_t launch_typed(const NormArgs& a, bool vec, bool shifted, cudaStream_t s) {
  const bool res = a.residual != nullptr;
  if (vec) return res ? launch_chunks<DT, QF, true, false>(a, s) : launch_chunks<DT, QF, false, false>(a, s);
  // bf16, shifted / element by element, us: with residual 8192 x 7167 110 / 123, 20 M elements of H = 1501 51 / 42, 3001 35 /
  // 45, 6001 34 / 52; to codes 3001 62 / 54, 6001 62 / 69; without residual 8192 x 7166 85 / 74; fp32 is no faster
  if constexpr (QF != kQuantMx && DT != kDtF32) {
    if (shifted && res && a.H > (QF == kQuantNone ? 2048 : 4096)) return launch_chunks<DT, QF, true, true>(a, s);
  }
  return launch_single<DT, QF>(a, s);
}

template <int QF>
cudaError_t launch_quant(const NormArgs& a, cudaStream_t s) {
  const int64_t EP = 16 / dtype_bytes(a.dtype);
  bool bases = reinterpret_cast<uintptr_t>(a.weight) % 16 == 0, same = true, whole = a.H % 8 == 0;
  for (const auto& m : {std::pair<const void*, int64_t>(a.x, a.x_stride), {a.residual, a.residual_stride},
                        {a.residual_out, a.residual_out_stride}, {a.out, a.out_stride}}) {
    if (m.first == nullptr) continue;
    bases = bases && reinterpret_cast<uintptr_t>(m.first) % 16 == 0;
    same = same && (a.T == 1 || m.second % EP == a.x_stride % EP);
    whole = whole && (a.T == 1 || m.second % EP == 0);
  }
  const bool vec = bases && whole && reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
  const bool shifted = bases && same && a.H <= 4 * 512 * 8 - 8 &&  // four chunks a thread
                       (QF == kQuantNone || a.H * 4 <= kRowsBytes);
  if (a.dtype == kDtBf16) return launch_typed<kDtBf16, QF>(a, vec, shifted, s);
  if (a.dtype == kDtF16) return launch_typed<kDtF16, QF>(a, vec, shifted, s);
  return launch_typed<kDtF32, QF>(a, vec, shifted, s);
}

}  // namespace
}  // namespace moe
