// rms_norm_backward.cu -- gradients of the root-mean-square norm.  With xh = x rstd and g = w dy:
//   dx = rstd (g - xh mean(g xh)) + dres,   dw = sum over rows of dy xh
// One pass over dy, x and dres.  Blocks stay and walk the rows, so a thread keeps its columns' sums of dw in
// registers; each block leaves its sums in the workspace and a second kernel adds them up, in the same
// order every time (no atomics).  8192 x 7168 bf16 with d_residual 83 us (0.85 of the copy rate; 75 without dw), 4095 x
// 5120 fp32 51 (0.74); 37 x 266 7.6.  Two blocks an SM wait for their rows' sums in turn (72 registers a thread, with
// which the fp32 instances spill 32-68 bytes); one block with a ring of five rows took 111 us.
//
// A row's rstd is known, so one sum (of g xh) stands between its loads and its dx.  To keep HBM busy
// meanwhile, rows come through shared memory by asynchronous 16-byte copies, a few rows ahead; a thread copies
// what it will read itself, so no barrier guards the ring.  Rows that start off the 16-byte boundaries are
// copied from the boundary below: a thread's columns then begin `shift` elements earlier.  The shift repeats
// every 2 to 8 rows, and a block takes rows of one shift only, so that its columns of dw stay its own
// (37401 x 1570 bf16 with d_residual 317 us element by element, 130 so; 8192 x 7167 88-90 against 83 of 7168).
// Rows of matrices that disagree on the shift, and rows too long for the ring, are read directly, twice (the
// second time from L1 or L2).
#include <algorithm>
#include <atomic>
#include <utility>

#include "norm_device.cuh"

namespace moe {
namespace {

constexpr int kNbThreads = 256;     // of a block that holds several rows
constexpr int kNbMaxThreads = 512;
constexpr int kNbHeldThreads = 448;  // with the weight in registers, two blocks an SM
constexpr int kNbMaxStages = 4;
constexpr int kNbMaxRing = 216 * 1024;  // of an SM

struct NormBackwardParams {
  NormBackwardArgs a;
  int tpr, rpb;  // as in rms_norm_kernel.cuh
  int stages;    // rows of the ring per row group
  int classes;   // rows r and r + classes start at the same place between two 16-byte boundaries
};

// `bytes` of 16 from a 16-byte boundary, the rest zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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

// The block's sums of dw, N values a thread.  `first` is the place of the thread's first one, `shift` places before which is
// column 0; the others follow in pieces of EP, 8 tpr apart (EP = 1: 32 apart, eight of them).  Rows that share a warp
// meet by shuffles; the warps (or groups of warps) of different rows lay theirs side by side in shared memory, where each
// column is added up in the groups' order and leaves in the columns' order.  A call, once a block: inlined, it costs
// the loop in front of it registers (8192 x 7168 82 -> 94 us, 37401 x 1570 128 -> 211).
template <int N, int EP>
__device__ __noinline__ void leave_dw(float* out, int H, int tpr, int first, int shift, float* sums, float* values) {
  const int lane = threadIdx.x & 31;
  float dw[N];
#pragma unroll
  for (int q = 0; q < N; ++q) dw[q] = values[q];
  auto col = [&](int q) {
    return EP == 1 ? first + (q / 8) * 8 * tpr + 32 * (q % 8) : first + (q / EP) * tpr * EP + q % EP;
  };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o >= tpr) {
#pragma unroll
      for (int q = 0; q < N; ++q) dw[q] += __shfl_xor_sync(0xffffffffu, dw[q], o);
    }
  const int per = max(tpr, 32), groups = (blockDim.x + per - 1) / per, slots = tpr * N;
  float* mine = sums + (threadIdx.x / per) * slots;
  if (tpr >= 32 || lane < tpr) {
#pragma unroll
    for (int q = 0; q < N; q += EP >= 4 ? 4 : 1) {
      if (EP >= 4) *reinterpret_cast<float4*>(mine + col(q)) = make_float4(dw[q], dw[(q + 1) % N], dw[(q + 2) % N], dw[(q + 3) % N]);
      else mine[col(q)] = dw[q];
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < H; c += blockDim.x) {
    float v = sums[c + shift];
    for (int g = 1; g < groups; ++g) v += sums[g * slots + c + shift];
    out[c] = v;
  }
}

template <int DT, bool VEC>
__device__ __forceinline__ void load_weight(const NormBackwardArgs& a, int col, float (&w)[8]) {
  if (a.weight_dtype == DT) load8<DT, VEC>(a.weight, 0, col, a.H, w);
  else load8<kDtF32, VEC>(a.weight, 0, col, a.H, w);
}

// Rows through the ring.  A thread owns pieces of 16 bytes (8 columns of 16-bit rows, 4 of fp32 ones), neighbouring
// threads neighbouring pieces.  Shared memory: [stage][array][piece][thread] of 16 bytes.
template <int DT, bool DRES, bool SHIFT, int NCH, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) norm_backward_ring_kernel(const __grid_constant__ NormBackwardParams p) {
  constexpr int kArrays = DRES ? 3 : 2, es = DT == kDtF32 ? 4 : 2, EP = 16 / es, NP = NCH * 8 / EP;
  constexpr bool kHoldWeight = NCH <= 2 || SHIFT;  // in registers; else from L1 every time
  extern __shared__ __align__(16) uint8_t ring[];
  const NormBackwardArgs& a = p.a;
  const int H = a.H, tpr = p.tpr;
  const int rb = tpr >= (int)blockDim.x ? 0 : threadIdx.x / tpr;
  // this block's rows: cls, cls + classes, ...; they start `shift` elements behind a 16-byte boundary
  const int classes = SHIFT ? p.classes : 1, cls = SHIFT ? (int)blockIdx.x % classes : 0;
  const int lanes = SHIFT ? max((int)gridDim.x / classes, 1) : gridDim.x;
  const int shift = SHIFT ? (int)((cls * a.x_stride) % EP) : 0;
  const int first = (int)(threadIdx.x - rb * tpr) * EP - shift;
  auto col = [&](int q) { return first + q * tpr * EP; };
  const uint32_t ring0 = (uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * 16u;
  const int64_t step = (int64_t)classes * lanes * p.rpb, row0 = cls + (int64_t)classes * (SHIFT ? blockIdx.x / classes : blockIdx.x) * p.rpb;
  const uint32_t piece = blockDim.x * 16u, array = NP * piece, slot_bytes = kArrays * array;
  int64_t ahead = row0 + classes * rb;  // the next row to fetch; every row group makes the same rounds
  const bool group = rb < p.rpb;
  auto fetch = [&](uint32_t dst) {
    const bool on = group && ahead < a.T;
    const int64_t r = on ? ahead : 0;
    const uint8_t* dy = static_cast<const uint8_t*>(a.dy) + r * a.dy_stride * es;
    const uint8_t* x = static_cast<const uint8_t*>(a.x) + r * a.x_stride * es;
    const uint8_t* dres = DRES ? static_cast<const uint8_t*>(a.dres) + r * a.dres_stride * es : nullptr;
    const int below = SHIFT && on ? -shift * es : 0;  // the boundary below the row (r = 0 lies on one itself)
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      const int c = col(q);
      const int bytes = !on || c >= H ? 0 : SHIFT ? min((H - c) * es, 16) : 16;  // nothing behind the row's end
      const int o = bytes > 0 ? c * es : below;  // a copy of nothing has to name a 16-byte boundary too
      const uint32_t at = dst + (uint32_t)q * piece;
      copy16(at, dy + o, bytes);
      copy16(at + array, x + o, bytes);
      if (DRES) copy16(at + 2 * array, dres + o, bytes);
    }
    copy_commit();
    ahead += step;
  };
  auto read = [&](uint32_t src, int which, int q) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(src + which * array + (uint32_t)q * piece) : "memory");
    if (SHIFT && q == 0 && first < 0) {  // the row before's last elements
      uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (DT == kDtF32) u[k] = k < shift ? 0u : u[k];
        else u[k] = 2 * k + 1 < shift ? 0u : 2 * k < shift ? u[k] & 0xFFFF0000u : u[k];
      }
      v = make_uint4(u[0], u[1], u[2], u[3]);
    }
    return v;
  };
  // elements 2j and 2j + 1 of a piece
  auto pair = [&](const uint4& v, int j) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    if (DT == kDtF32) return two(__uint_as_float(u[(2 * j) & 3]), __uint_as_float(u[(2 * j + 1) & 3]));
    if (DT == kDtBf16) return two(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xFFFF0000u));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
    return two(f.x, f.y);
  };
  float w[NP][EP];
  auto weight = [&](int q) {
    const int c = col(q);
#pragma unroll
    for (int j = 0; j < EP; ++j) w[q][j] = 0.0f;
    const bool same = DT != kDtF32 && a.weight_dtype == DT;
    if (SHIFT) {  // element by element, all loads on their way at once: a test each would wait for each
      auto elements = [&](auto load) {
        float f[EP];
#pragma unroll
        for (int j = 0; j < EP; ++j) f[j] = load(min(max(c + j, 0), H - 1));
#pragma unroll
        for (int j = 0; j < EP; ++j) w[q][j] = c + j >= 0 && c + j < H ? f[j] : 0.0f;
      };
      if (same) elements([&](int k) { return load1<DT>(a.weight, k); });
      else elements([&](int k) { return load1<kDtF32>(a.weight, k); });
      return;
    }
    if (c >= H) return;
    const uint8_t* at = static_cast<const uint8_t*>(a.weight) + (int64_t)c * (same ? 2 : 4);
    if (same) {
      const uint4 v = *reinterpret_cast<const uint4*>(at);
#pragma unroll
      for (int j = 0; j < EP / 2; ++j) apart(pair(v, j), w[q][2 * j], w[q][2 * j + 1]);
    } else {
#pragma unroll
      for (int j = 0; j < EP; j += 4) {
        const float4 v = *reinterpret_cast<const float4*>(at + 4 * j);
        w[q][j] = v.x, w[q][j + 1] = v.y, w[q][j + 2] = v.z, w[q][j + 3] = v.w;
      }
    }
  };
  auto weight_pair = [&](int q, int j) { return two(w[q][2 * j], w[q][2 * j + 1]); };
  if (kHoldWeight) {
#pragma unroll
    for (int q = 0; q < NP; ++q) weight(q);
  }
  uint64_t dw[NP][EP / 2] = {};
  for (int s = 0; s < p.stages; ++s) fetch(ring0 + s * slot_bytes);
  int slot = 0, turn = 0;
  const float inv_h = 1.0f / (float)H;
  int64_t row = row0 + classes * rb;
  float next = group && row < a.T ? a.rstd[row] : 0.0f;  // the next round's rstd
  for (int64_t base = row0; base < a.T; base += step, row += step) {
    const bool on = group && row < a.T;
    const float rstd = next;
    next = group && row + step < a.T ? a.rstd[row + step] : 0.0f;
    // one group of copies a round, in the rows' order: this round's is complete when at most stages - 1 are not
    if (p.stages == 4) copy_wait<3>();
    else if (p.stages == 3) copy_wait<2>();
    else copy_wait<1>();
    const uint32_t src = ring0 + slot * slot_bytes;
    const uint64_t rstd2 = two(rstd, rstd);
    uint64_t dot2 = two(0.0f, 0.0f);
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      if (!kHoldWeight) weight(q);
      const uint4 dy = read(src, 0, q), x = read(src, 1, q);
#pragma unroll
      for (int j = 0; j < EP / 2; ++j) {
        const uint64_t t = mul2(pair(dy, j), mul2(pair(x, j), rstd2));
        dw[q][j] = add2(dw[q][j], t);
        dot2 = fma2(weight_pair(q, j), t, dot2);
      }
    }
    float lo, hi;
    apart(dot2, lo, hi);
    const float dot = row_sum_again(lo + hi, tpr, rb, turn) * inv_h;
    turn ^= 1;
    const float k = -(rstd * rstd) * dot;
    const uint64_t k2 = two(k, k);
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      if (!kHoldWeight) weight(q);
      const uint4 dy = read(src, 0, q), x = read(src, 1, q);
      uint4 dres = dy;
      if (DRES) dres = read(src, 2, q);
      float v[EP];
#pragma unroll
      for (int j = 0; j < EP / 2; ++j) {
        uint64_t t = mul2(pair(x, j), k2);
        if (DRES) t = add2(t, pair(dres, j));
        apart(fma2(mul2(weight_pair(q, j), pair(dy, j)), rstd2, t), v[2 * j], v[2 * j + 1]);
      }
      const int c = col(q);
      if (SHIFT && on && (c < 0 || c + EP > H)) {
#pragma unroll
        for (int j = 0; j < EP; ++j) {
          if (c + j < 0 || c + j >= H) continue;
          const int64_t o = row * a.dx_stride + c + j;
          if (DT == kDtF32) static_cast<float*>(a.dx)[o] = v[j];
          else static_cast<uint16_t*>(a.dx)[o] = (uint16_t)pack2<DT>(v[j], 0.0f);
        }
      } else if (on && (SHIFT || c < H)) {
        uint4 r;
        if constexpr (DT == kDtF32)
          r = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        else
          r = make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7]));
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.dx) + (row * a.dx_stride + c) * es) = r;
      }
    }
    fetch(src);
    if (++slot == p.stages) slot = 0;
  }
  copy_wait<0>();
  if (a.dw == nullptr) return;
  __syncthreads();  // the ring is free
  float sums[NP * EP];
#pragma unroll
  for (int q = 0; q < NP; ++q)
#pragma unroll
    for (int j = 0; j < EP / 2; ++j) apart(dw[q][j], sums[q * EP + 2 * j], sums[q * EP + 2 * j + 1]);
  leave_dw<NP * EP, EP>(a.partial + (int64_t)blockIdx.x * H, H, tpr, first + shift, shift, reinterpret_cast<float*>(ring), sums);
}

// Rows read directly.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kNbMaxThreads, 1) norm_backward_kernel(const __grid_constant__ NormBackwardParams p) {
  constexpr int NCH = 8;
  extern __shared__ __align__(16) uint8_t ring[];
  const NormBackwardArgs& a = p.a;
  const int H = a.H, tpr = p.tpr;
  const int rb = tpr >= (int)blockDim.x ? 0 : threadIdx.x / tpr;
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
  float sums[NCH * 8];
#pragma unroll
  for (int q = 0; q < NCH * 8; ++q) sums[q] = dw[q / 8][q % 8];
  leave_dw<NCH * 8, VEC ? 8 : 1>(a.partial + (int64_t)blockIdx.x * H, H, tpr, map.col(0), 0, reinterpret_cast<float*>(ring), sums);
}

// dw[c] = the blocks' sums of column c.  32 columns a block, 16 threads a column, each with all its loads in flight.
constexpr int kSumWays = 16;
constexpr int kNbParts = 3 * 152;  // the most blocks
__global__ void __launch_bounds__(32 * kSumWays, 1) norm_weight_sum_kernel(const float* partial, int parts, int H, float* dw) {
  __shared__ float sums[kSumWays][32];
  const int lane = threadIdx.x & 31, way = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  constexpr int kEach = (kNbParts + kSumWays - 1) / kSumWays;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float v[kEach], sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int q = way + i * kSumWays;
    v[i] = col < H && q < parts ? partial[(int64_t)q * H + col] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) sum += v[i];
  sums[way][lane] = sum;
  __syncthreads();
  if (way > 0 || col >= H) return;
#pragma unroll
  for (int q = 1; q < kSumWays; ++q) sum += sums[q][lane];
  dw[col] = sum;
}

// Two blocks an SM, three of 16-bit rows that take 256 threads or fewer (37401 x 1570 bf16 140 against 129 us; two rows
// ahead of fp32 do not fit three times).
int blocks_an_sm(int H, int es) { return H <= 2 * 8 * kNbThreads && es == 2 ? 3 : 2; }

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

// What leave_dw lays out.
int64_t sums_bytes(const Shape& s, int threads, int nch) {
  const int per = std::max(s.tpr, 32);
  return (int64_t)((threads + per - 1) / per) * s.tpr * nch * 8 * 4;
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

template <int DT, bool DRES, bool SHIFT, int NCH, int THREADS, int BLOCKS>
cudaError_t launch_kernel(const NormBackwardParams& p, int grid, int threads, int64_t smem, cudaStream_t s) {
  static std::atomic<int> ready[64];
  const cudaError_t err = allow_smem(norm_backward_ring_kernel<DT, DRES, SHIFT, NCH, THREADS, BLOCKS>, ready);
  if (err != cudaSuccess) return err;
  norm_backward_ring_kernel<DT, DRES, SHIFT, NCH, THREADS, BLOCKS><<<grid, threads, smem, s>>>(p);
  return cudaGetLastError();
}

template <int DT, int NCH, int THREADS, int BLOCKS>
cudaError_t launch_ring(const NormBackwardParams& p, bool shift, int grid, int threads, int64_t smem, cudaStream_t s) {
  const bool dres = p.a.dres != nullptr;
  if (shift)
    return dres ? launch_kernel<DT, true, true, NCH, THREADS, BLOCKS>(p, grid, threads, smem, s)
                : launch_kernel<DT, false, true, NCH, THREADS, BLOCKS>(p, grid, threads, smem, s);
  return dres ? launch_kernel<DT, true, false, NCH, THREADS, BLOCKS>(p, grid, threads, smem, s)
              : launch_kernel<DT, false, false, NCH, THREADS, BLOCKS>(p, grid, threads, smem, s);
}

// `vec`: rows of whole chunks on 16-byte boundaries; `classes`: how often their shift repeats, or 0 where the matrices'
// rows do not share one.
template <int DT>
cudaError_t launch_typed(const NormBackwardArgs& a, bool vec, int classes, cudaStream_t s) {
  NormBackwardParams p{a, 0, 1, 0, classes};
  constexpr int EP = DT == kDtF32 ? 4 : 8;
  const int64_t es = DT == kDtF32 ? 4 : 2, arrays = a.dres != nullptr ? 3 : 2;
  const int chunks = (a.H + (classes > 1 ? EP - 1 : 0) + 7) / 8;
  const int nch = chunks <= 2 * kNbHeldThreads ? 2 : 4;
  Shape sh = shape_of(chunks, nch, true, (a.T + std::max(classes, 1) - 1) / std::max(classes, 1));
  int threads = (sh.tpr * sh.rpb + 31) / 32 * 32;
  const int64_t stage = arrays * nch * 8 * es * threads;
  p.stages = (int)std::min<int64_t>(kNbMaxStages, kNbMaxRing / blocks_an_sm(a.H, es) / stage);
  if (p.stages < 2) p.stages = (int)std::min<int64_t>(kNbMaxStages, kNbMaxRing / stage);
  cudaError_t err;
  if (classes > 0 && sh.tpr <= kNbMaxThreads && p.stages >= 2) {
    p.tpr = sh.tpr;
    p.rpb = sh.rpb;
    int64_t grid = std::min<int64_t>(152 * blocks_an_sm(a.H, es), (a.T + sh.rpb - 1) / sh.rpb);
    // the same number of blocks for every class, or one for each of fewer rows than classes
    grid = std::max<int64_t>(grid / classes * classes, std::min<int64_t>(classes, a.T));
    const int64_t smem = std::max<int64_t>(p.stages * stage, sums_bytes(sh, threads, nch));
    // a weight off the 16-byte boundaries is read as under a shift
    const bool shift = classes > 1 || a.H % EP != 0 || reinterpret_cast<uintptr_t>(a.weight) % 16 != 0;
    err = nch == 2 ? launch_ring<DT, 2, kNbHeldThreads, 2>(p, shift, (int)grid, threads, smem, s)
                   : launch_ring<DT, 4, kNbMaxThreads, 1>(p, shift, (int)grid, threads, smem, s);
    p.stages = (int)grid;
  } else {
    sh = shape_of(vec ? (a.H + 7) / 8 : (a.H + 255) / 256 * 32, 8, vec, a.T);
    p.tpr = sh.tpr;
    p.rpb = sh.rpb;
    threads = (sh.tpr * sh.rpb + 31) / 32 * 32;
    const int grid = (int)std::min<int64_t>(norm_backward_parts(a.T, a.H), (a.T + sh.rpb - 1) / sh.rpb);
    const int64_t smem = sums_bytes(sh, threads, 8);
    static std::atomic<int> ready[2][64];
    err = vec ? allow_smem(norm_backward_kernel<DT, true>, ready[0]) : allow_smem(norm_backward_kernel<DT, false>, ready[1]);
    if (err != cudaSuccess) return err;
    if (vec) norm_backward_kernel<DT, true><<<grid, threads, smem, s>>>(p);
    else norm_backward_kernel<DT, false><<<grid, threads, smem, s>>>(p);
    err = cudaGetLastError();
    p.stages = grid;
  }
  if (err != cudaSuccess || a.dw == nullptr) return err;
  // Its launch is prepared under the first kernel, which gives no signal: its blocks start when the first's have left, and
  // wait for what those wrote.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.H + 31) / 32));
  cfg.blockDim = dim3(32 * kSumWays);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_weight_sum_kernel, (const float*)a.partial, p.stages, a.H, a.dw);
}

}  // namespace

// The most blocks that are launched, for either size of elements.
int norm_backward_parts(int64_t T, int H) { return (int)std::min<int64_t>(T, 152 * blocks_an_sm(H, 2)); }

cudaError_t launch_rms_norm_backward(const NormBackwardArgs& a, cudaStream_t s) {
  if (a.T == 0) return a.dw != nullptr ? cudaMemsetAsync(a.dw, 0, (size_t)a.H * 4, s) : cudaSuccess;
  const int64_t es = dtype_bytes(a.dtype);
  const int64_t EP = 16 / es;
  bool bases = true, strides = true, whole = a.H % 8 == 0;
  for (const auto& m : {std::pair<const void*, int64_t>(a.dy, a.dy_stride), {a.x, a.x_stride}, {a.dres, a.dres_stride},
                        {a.dx, a.dx_stride}}) {
    if (m.first == nullptr) continue;
    bases = bases && reinterpret_cast<uintptr_t>(m.first) % 16 == 0;
    strides = strides && (a.T == 1 || m.second % EP == a.x_stride % EP);
    whole = whole && (a.T == 1 || m.second % EP == 0);
  }
  const int64_t off = a.T == 1 ? 0 : a.x_stride % EP;
  const int classes = !bases || !strides ? 0 : off == 0 ? 1 : off % 4 == 0 ? (int)(EP / 4) : off % 2 == 0 ? (int)(EP / 2) : (int)EP;
  const bool vec = bases && whole && reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
  if (a.dtype == kDtBf16) return launch_typed<kDtBf16>(a, vec, classes, s);
  if (a.dtype == kDtF16) return launch_typed<kDtF16>(a, vec, classes, s);
  return launch_typed<kDtF32>(a, vec, classes, s);
}

}  // namespace moe
