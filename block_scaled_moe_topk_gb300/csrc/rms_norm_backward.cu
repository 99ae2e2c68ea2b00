// rms_norm_backward.cu -- gradients of the root-mean-square norm.  With xh = x rstd and g = w dy:
//   dx = rstd (g - xh mean(g xh)) + dres,   dw = sum over rows of dy xh
// One pass over dy, x and dres.  Blocks stay and walk the rows, so a thread keeps its columns' sums of dw in
// registers; each block leaves its sums in the workspace and a second kernel adds them up, in the same
// order every time (no atomics).
//
// A row's rstd is known, so one sum (of g xh) stands between its loads and its dx.  To keep HBM busy
// meanwhile, rows on 16-byte boundaries come through shared memory by asynchronous 16-byte copies, a few
// rows ahead; a thread copies what it will read itself, so no barrier guards the ring.  Rows off those
// boundaries, and rows too long for the ring, are read directly, twice (the second time from L1 or L2).
#include <algorithm>
#include <atomic>

#include "norm_device.cuh"

namespace moe {
namespace {

constexpr int kNbThreads = 256;     // of a block that holds several rows
constexpr int kNbMaxThreads = 512;
constexpr int kNbMaxStages = 4;
constexpr int kNbRingBytes = 108 * 1024;  // a block's share of an SM that holds two
constexpr int kNbMaxRing = 216 * 1024;

struct NormBackwardParams {
  NormBackwardArgs a;
  int tpr, rpb;  // as in rms_norm.cu
  int stages;    // rows of the ring per row group
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sum over a row's threads, as row_sum, but callable again and again: two buffers in turn, so that one barrier a
// call is enough.
__device__ __forceinline__ float row_sum_again(float v, int tpr, int rb, int turn) {
  __shared__ float part[2][32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < tpr) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (tpr <= 32) return v;
  const int nw = tpr >> 5, lane = threadIdx.x & 31;
  if (lane == 0) part[turn][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < nw ? part[turn][rb * nw + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The block's sums of dw: the row groups' own sums meet in shared memory, in the groups' order.
template <bool VEC, int NCH>
__device__ __forceinline__ void leave_dw(const NormBackwardParams& p, const ColumnMap<VEC>& map, int rb, float* sums,
                                         const float (&dw)[NCH][8]) {
  const int H = p.a.H;
  float* out = p.a.partial + (int64_t)blockIdx.x * H;
  for (int g = 0; g < p.rpb; ++g) {
    if (p.rpb > 1) __syncthreads();
    if (g != rb) continue;
    const bool last = g == p.rpb - 1;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = map.col(c) + (VEC ? j : 32 * j);
        if (col >= H) continue;
        float v = dw[c][j];
        if (g > 0) v += sums[col];
        if (last) out[col] = v;
        else sums[col] = v;
      }
  }
}

template <int DT, bool VEC>
__device__ __forceinline__ void load_weight(const NormBackwardArgs& a, int col, float (&w)[8]) {
  if (a.weight_dtype == DT) load8<DT, VEC>(a.weight, 0, col, a.H, w);
  else load8<kDtF32, VEC>(a.weight, 0, col, a.H, w);
}

// Rows through the ring.  Shared memory: [stage][array][chunk half][thread] of 16 bytes.
template <int DT, bool DRES>
__global__ void __launch_bounds__(kNbMaxThreads, 1) norm_backward_ring_kernel(const __grid_constant__ NormBackwardParams p) {
  constexpr int NCH = 4, kParts = DT == kDtF32 ? 2 : 1, kArrays = DRES ? 3 : 2;
  extern __shared__ __align__(16) uint8_t ring[];
  const NormBackwardArgs& a = p.a;
  const int H = a.H, tpr = p.tpr, es = DT == kDtF32 ? 4 : 2;
  const int rb = p.rpb == 1 ? 0 : threadIdx.x / tpr;
  const int i = threadIdx.x - rb * tpr;
  const ColumnMap<true> map(i, tpr);
  const uint32_t ring0 = (uint32_t)__cvta_generic_to_shared(ring);
  const int64_t step = (int64_t)gridDim.x * p.rpb;
  const int64_t first = (int64_t)blockIdx.x * p.rpb;  // of the block; every row group makes the same rounds
  const uint32_t slot_bytes = kArrays * NCH * kParts * blockDim.x * 16;
  auto at = [&](int array, int c, int h) { return (uint32_t)(((array * NCH + c) * kParts + h) * blockDim.x + threadIdx.x) * 16u; };
  auto fetch = [&](int64_t base, int slot) {
    const int64_t row = base + rb;
    const bool on = base < a.T && rb < p.rpb && row < a.T;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int h = 0; h < kParts; ++h) {
        const int col = map.col(c) + 4 * h;
        const bool in = on && col < H;
        const uint32_t dst = ring0 + slot * slot_bytes;
        const int64_t o = in ? col : 0, r = in ? row : 0;
        copy16(dst + at(0, c, h), static_cast<const uint8_t*>(a.dy) + (r * a.dy_stride + o) * es, in);
        copy16(dst + at(1, c, h), static_cast<const uint8_t*>(a.x) + (r * a.x_stride + o) * es, in);
        if (DRES) copy16(dst + at(2, c, h), static_cast<const uint8_t*>(a.dres) + (r * a.dres_stride + o) * es, in);
      }
    copy_commit();
  };
  auto read = [&](int slot, int array, int c, float (&v)[8]) {
    const uint8_t* src = ring + slot * slot_bytes;
    const uint4 u = *reinterpret_cast<const uint4*>(src + at(array, c, 0));
    if (DT == kDtF32) {
      const uint4 t = *reinterpret_cast<const uint4*>(src + at(array, c, kParts - 1));
      v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y), v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
      v[4] = __uint_as_float(t.x), v[5] = __uint_as_float(t.y), v[6] = __uint_as_float(t.z), v[7] = __uint_as_float(t.w);
    } else {
      unpack8<DT>(u, v);
    }
  };
  float dw[NCH][8] = {};
  for (int s = 0; s < p.stages; ++s) fetch(first + s * step, s);
  int slot = 0, turn = 0;
  for (int64_t base = first; base < a.T; base += step) {
    const int64_t row = base + rb;
    const bool on = rb < p.rpb && row < a.T;
    const float rstd = on ? a.rstd[row] : 0.0f;
    // one group of copies a round, in the rows' order: this round's is complete when at most stages - 1 are not
    if (p.stages == 4) copy_wait<3>();
    else if (p.stages == 3) copy_wait<2>();
    else copy_wait<1>();
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      float w[8], dy[8], x[8];
      load_weight<DT, true>(a, map.col(c), w);
      read(slot, 0, c, dy);
      read(slot, 1, c, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = dy[j] * (x[j] * rstd);
        dw[c][j] += t;
        dot = fmaf(w[j], t, dot);
      }
    }
    dot = row_sum_again(dot, tpr, rb, turn) / (float)H;
    turn ^= 1;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      float w[8], dy[8], x[8], dres[8];
      load_weight<DT, true>(a, map.col(c), w);
      read(slot, 0, c, dy);
      read(slot, 1, c, x);
      if (DRES) read(slot, 2, c, dres);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dy[j] = rstd * (w[j] * dy[j] - x[j] * rstd * dot);
        if (DRES) dy[j] += dres[j];
      }
      store8<DT, true>(a.dx, row * a.dx_stride, map.col(c), on ? H : 0, dy);
    }
    fetch(base + p.stages * step, slot);
    if (++slot == p.stages) slot = 0;
  }
  copy_wait<0>();
  if (a.dw == nullptr) return;
  __syncthreads();  // the ring is free
  leave_dw<true, NCH>(p, map, rb, reinterpret_cast<float*>(ring), dw);
}

// Rows read directly.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kNbMaxThreads, 1) norm_backward_kernel(const __grid_constant__ NormBackwardParams p) {
  constexpr int NCH = 8;
  extern __shared__ __align__(16) uint8_t ring[];
  const NormBackwardArgs& a = p.a;
  const int H = a.H, tpr = p.tpr;
  const int rb = p.rpb == 1 ? 0 : threadIdx.x / tpr;
  const int i = threadIdx.x - rb * tpr;
  const ColumnMap<VEC> map(i, tpr);
  float dw[NCH][8] = {};
  int turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * p.rpb; base < a.T; base += (int64_t)gridDim.x * p.rpb) {
    const int64_t row = base + rb;
    const bool on = rb < p.rpb && row < a.T;
    const int n = on ? H : 0;
    const float rstd = on ? a.rstd[row] : 0.0f;
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = map.col(c);
      if (col >= H) break;
      float w[8], dy[8], x[8];
      load_weight<DT, VEC>(a, col, w);
      load8<DT, VEC>(a.dy, row * a.dy_stride, col, n, dy);
      load8<DT, VEC>(a.x, row * a.x_stride, col, n, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = dy[j] * (x[j] * rstd);
        dw[c][j] += t;
        dot = fmaf(w[j], t, dot);
      }
    }
    dot = row_sum_again(dot, tpr, rb, turn) / (float)H;
    turn ^= 1;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = map.col(c);
      if (col >= H) break;
      float w[8], dy[8], x[8], dres[8];
      load_weight<DT, VEC>(a, col, w);
      load8<DT, VEC>(a.dy, row * a.dy_stride, col, n, dy);
      load8<DT, VEC>(a.x, row * a.x_stride, col, n, x);
      if (a.dres != nullptr) load8<DT, VEC>(a.dres, row * a.dres_stride, col, n, dres);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dy[j] = rstd * (w[j] * dy[j] - x[j] * rstd * dot);
        if (a.dres != nullptr) dy[j] += dres[j];
      }
      store8<DT, VEC>(a.dx, row * a.dx_stride, col, n, dy);
    }
  }
  if (a.dw == nullptr) return;
  leave_dw<VEC, NCH>(p, map, rb, reinterpret_cast<float*>(ring), dw);
}

// dw[c] = the blocks' sums of column c.  32 columns a block, 16 threads a column.
constexpr int kSumWays = 16;
__global__ void __launch_bounds__(32 * kSumWays) norm_weight_sum_kernel(const float* partial, int parts, int H, float* dw) {
  __shared__ float sums[kSumWays][32];
  const int lane = threadIdx.x & 31, way = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (col < H)
    for (int q = way; q < parts; q += kSumWays) v += partial[(int64_t)q * H + col];
  sums[way][lane] = v;
  __syncthreads();
  if (way > 0 || col >= H) return;
#pragma unroll
  for (int q = 1; q < kSumWays; ++q) v += sums[q][lane];
  dw[col] = v;
}

struct Shape {
  int tpr, rpb;
};
Shape shape_of(int chunks, int nch, bool vec, int64_t T) {
  Shape s{(chunks + nch - 1) / nch, 1};
  if (vec && s.tpr <= 16) {
    int t = 1;
    while (t < s.tpr) t *= 2;
    s.tpr = t;
  } else {
    s.tpr = (s.tpr + 31) / 32 * 32;
  }
  s.rpb = (int)std::min<int64_t>(std::max(1, kNbThreads / s.tpr), T);
  return s;
}

template <typename K>
cudaError_t allow_smem(K kernel, std::atomic<int> (&ready)[64]) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (ready[dev].load(std::memory_order_acquire)) return cudaSuccess;
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNbMaxRing);
  if (err == cudaSuccess) ready[dev].store(1, std::memory_order_release);
  return err;
}

template <int DT, bool DRES>
cudaError_t launch_ring(const NormBackwardParams& p, int grid, int threads, int64_t smem, cudaStream_t s) {
  static std::atomic<int> ready[64];
  const cudaError_t err = allow_smem(norm_backward_ring_kernel<DT, DRES>, ready);
  if (err != cudaSuccess) return err;
  norm_backward_ring_kernel<DT, DRES><<<grid, threads, smem, s>>>(p);
  return cudaGetLastError();
}

template <int DT>
cudaError_t launch_typed(const NormBackwardArgs& a, bool vec, cudaStream_t s) {
  NormBackwardParams p{a, 0, 1, 0};
  const int chunks = vec ? (a.H + 7) / 8 : (a.H + 255) / 256 * 32;
  const int64_t es = DT == kDtF32 ? 4 : 2, arrays = a.dres != nullptr ? 3 : 2;
  Shape sh = shape_of(chunks, 4, vec, a.T);
  int threads = (sh.tpr * sh.rpb + 31) / 32 * 32;
  const int64_t stage = arrays * 4 * 8 * es * threads;
  p.stages = (int)std::min<int64_t>(kNbMaxStages, kNbRingBytes / stage);
  if (p.stages < 2) p.stages = (int)std::min<int64_t>(kNbMaxStages, kNbMaxRing / stage);
  cudaError_t err;
  if (vec && sh.tpr <= kNbMaxThreads && p.stages >= 2) {
    p.tpr = sh.tpr;
    p.rpb = sh.rpb;
    const int grid = (int)std::min<int64_t>(norm_backward_parts(a.T, a.H), (a.T + sh.rpb - 1) / sh.rpb);
    const int64_t smem = std::max<int64_t>(p.stages * stage, sh.rpb > 1 ? 4 * (int64_t)a.H : 0);
    err = a.dres != nullptr ? launch_ring<DT, true>(p, grid, threads, smem, s)
                            : launch_ring<DT, false>(p, grid, threads, smem, s);
    p.stages = grid;
  } else {
    sh = shape_of(chunks, 8, vec, a.T);
    p.tpr = sh.tpr;
    p.rpb = sh.rpb;
    threads = (sh.tpr * sh.rpb + 31) / 32 * 32;
    const int grid = (int)std::min<int64_t>(norm_backward_parts(a.T, a.H), (a.T + sh.rpb - 1) / sh.rpb);
    const int64_t smem = sh.rpb > 1 ? 4 * (int64_t)a.H : 0;  // rows of at most 8 K columns share a block
    if (vec) norm_backward_kernel<DT, true><<<grid, threads, smem, s>>>(p);
    else norm_backward_kernel<DT, false><<<grid, threads, smem, s>>>(p);
    err = cudaGetLastError();
    p.stages = grid;
  }
  if (err != cudaSuccess || a.dw == nullptr) return err;
  norm_weight_sum_kernel<<<(a.H + 31) / 32, 32 * kSumWays, 0, s>>>(a.partial, p.stages, a.H, a.dw);
  return cudaGetLastError();
}

}  // namespace

// Two blocks an SM of the 152, fewer for fewer rows.
int norm_backward_parts(int64_t T, int) { return (int)std::min<int64_t>(T, 2 * 152); }

cudaError_t launch_rms_norm_backward(const NormBackwardArgs& a, cudaStream_t s) {
  if (a.T == 0) return a.dw != nullptr ? cudaMemsetAsync(a.dw, 0, (size_t)a.H * 4, s) : cudaSuccess;
  const int64_t es = dtype_bytes(a.dtype);
  auto grid16 = [&](const void* q, int64_t stride) {
    return q == nullptr || (reinterpret_cast<uintptr_t>(q) % 16 == 0 && (a.T == 1 || stride * es % 16 == 0));
  };
  const bool vec = a.H % 8 == 0 && grid16(a.dy, a.dy_stride) && grid16(a.x, a.x_stride) &&
                   grid16(a.dres, a.dres_stride) && grid16(a.dx, a.dx_stride) &&
                   reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
  if (a.dtype == kDtBf16) return launch_typed<kDtBf16>(a, vec, s);
  if (a.dtype == kDtF16) return launch_typed<kDtF16>(a, vec, s);
  return launch_typed<kDtF32>(a, vec, s);
}

}  // namespace moe
