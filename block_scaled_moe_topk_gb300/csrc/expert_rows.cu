// expert_rows.cu -- token rows to expert rows and back, their gradients, and the gradient of the
// routing weights.  With r(t, j) = inv[t*k + j] the row of token t's slot j:
//   permute            rows[r(t, j)] = x[t]
//   permute backward   dx[t] = sum_j drows[r(t, j)]
//   unpermute          out[t] = sum_j w[t, j] rows[r(t, j)]
//   unpermute backward drows[r(t, j)] = w[t, j] dout[t];  dw[t, j] = <dout[t], rows[r(t, j)]>
//   route backward     w = softmax over the k selected logits, so with g_j = w_j (dw_j - sum_i w_i dw_i)
//                      dlogits[t, ids[t, j]] = g_j and 0 in the other columns
// All sums run in fp32 in slot order and are rounded once; a pair whose row lies outside [0, R) is
// dropped: it is neither read nor written, and its dw is 0.
//
// Every kernel moves each byte once and is bound by HBM, so work is split by token: a token's row
// is read once and its k expert rows are touched by the same threads, with all loads of a thread
// issued before the first use.  A thread's access is the widest power of two (16 bytes at most)
// that divides the addresses, strides and row length.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "expert_internal.h"

namespace moe {
namespace {

constexpr int kRowThreads = 256;
constexpr int64_t kFewTokens = 152;  // a row's threads are then spread wider: latency counts

template <int VB>
struct Raw;
template <>
struct Raw<16> { using T = uint4; };
template <>
struct Raw<8> { using T = uint2; };
template <>
struct Raw<4> { using T = uint32_t; };
template <>
struct Raw<2> { using T = uint16_t; };
template <>
struct Raw<1> { using T = uint8_t; };

template <int DT>
struct Elem;
template <>
struct Elem<kDtBf16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float to(T v) { return __bfloat162float(v); }
  static __device__ __forceinline__ T from(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<kDtF16> {
  using T = __half;
  static __device__ __forceinline__ float to(T v) { return __half2float(v); }
  static __device__ __forceinline__ T from(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<kDtF32> {
  using T = float;
  static __device__ __forceinline__ float to(T v) { return v; }
  static __device__ __forceinline__ T from(float v) { return v; }
};

// VB bytes as the elements they hold.
template <int DT, int VB>
union Chunk {
  using E = typename Elem<DT>::T;
  static constexpr int kN = VB / (int)sizeof(E);
  typename Raw<VB>::T raw;
  E e[kN];
  __device__ __forceinline__ Chunk() {}
};

struct RowsParams {
  RowsArgs a;
  int chunks;    // VB-byte chunks of a row
  int lg;        // log2 of the threads a row gets
  int elem;      // bytes of an element
  int slices;    // blocks that share a row
};

// The k expert rows of token t; -1 for a dropped pair.
template <int KM>
__device__ __forceinline__ void load_rows(const RowsArgs& a, int64_t t, int (&r)[KM]) {
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    r[j] = -1;
    if (j < a.k) {
      const int v = a.inv[t * a.k + j];
      if (v >= 0 && v < a.R) r[j] = v;
    }
  }
}

// The first of a thread's U chunks, `step` apart: a warp's rounds are neighbours in the row, so that the
// sectors that two rounds share are fetched and written while they are at hand (permute at H = 7166,
// bf16, T = 8192, k = 6: 183 us with the rounds a block apart, 126 us so).
template <int U>
__device__ __forceinline__ int first_chunk(int in_row, int step) {
  return (in_row & ~(step - 1)) * U + (in_row & (step - 1));
}

// A thread copies U chunks of a token's row to each of its k rows.  Blocks of a row are neighbours in
// launch order: with the rows in the order of one slice after the other, H = 7167 took 220 against 180
// us (T = 8192, k = 6, bf16; with adjacent rounds 151, and H = 7168: 124, 0.98 of the copy rate).
template <int VB, int U>
__global__ void __launch_bounds__(kRowThreads) permute_kernel(const __grid_constant__ RowsParams p) {
  using V = typename Raw<VB>::T;
  const RowsArgs& a = p.a;
  const int tpr = 1 << p.lg;
  const uint32_t group = blockIdx.x / (uint32_t)p.slices, slice = blockIdx.x - group * (uint32_t)p.slices;
  const int64_t t = (int64_t)group * (kRowThreads >> p.lg) + (threadIdx.x >> p.lg);
  const int step = min(tpr, 32), c0 = (int)slice * (tpr * U) + first_chunk<U>(threadIdx.x & (tpr - 1), step);
  if (t >= a.T) return;
  const uint8_t* src = static_cast<const uint8_t*>(a.tokens_in) + t * a.token_stride * p.elem;
  V v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * step;
    if (c < p.chunks) v[u] = reinterpret_cast<const V*>(src)[c];
  }
  int r[kMaxTopK];
  load_rows(a, t, r);
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    if (r[j] < 0) continue;
    V* dst = reinterpret_cast<V*>(static_cast<uint8_t*>(a.rows_out) + (int64_t)r[j] * a.rows_out_stride * p.elem);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * step;
      if (c < p.chunks) dst[c] = v[u];
    }
  }
}

// A thread sums U chunks over the k <= KM rows of a token (w null: plain sum).  Here the blocks of one
// slice of all rows come first (row by row: 139 against 131 us at T = 8192, H = 7168, k = 6, bf16, 0.92
// of the copy rate with streaming loads).  KM = 4 leaves registers for more threads an SM.  Narrow
// accesses over more slots are held to three blocks' registers, which batches their loads: H = 7167 253 -> 230 us,
// H = 7166 163 -> 156, H = 121 with T = 16384, k = 8 13.3 -> 11.8; the others are best left alone (H = 7168:
// 131 against 145 us with three, k = 3 77 against 83 with four).
template <int DT, int VB, int U, int KM>
__global__ void __launch_bounds__(kRowThreads, VB < 16 && KM > 4 ? 3 : 0)
    unpermute_kernel(const __grid_constant__ RowsParams p) {
  using C = Chunk<DT, VB>;
  const RowsArgs& a = p.a;
  const int tpr = 1 << p.lg;
  const int64_t t = (int64_t)blockIdx.x * (kRowThreads >> p.lg) + (threadIdx.x >> p.lg);
  const int step = min(tpr, 32), c0 = blockIdx.y * (tpr * U) + first_chunk<U>(threadIdx.x & (tpr - 1), step);
  if (t >= a.T) return;
  int r[KM];
  load_rows(a, t, r);
  float w[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) w[j] = j < a.k && a.w != nullptr ? a.w[t * a.k + j] : 1.0f;
  C v[U][KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    if (r[j] < 0) continue;
    const uint8_t* src = static_cast<const uint8_t*>(a.rows_in) + (int64_t)r[j] * a.rows_in_stride * p.elem;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * step;
      if (c < p.chunks) v[u][j].raw = __ldcs(reinterpret_cast<const typename Raw<VB>::T*>(src) + c);
    }
  }
  uint8_t* dst = static_cast<uint8_t*>(a.tokens_out) + t * a.token_stride * p.elem;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * step;
    if (c >= p.chunks) continue;
    C o;
#pragma unroll
    for (int i = 0; i < C::kN; ++i) {
      float acc = 0.0f;
#pragma unroll
      for (int j = 0; j < KM; ++j)
        if (r[j] >= 0) acc = fmaf(w[j], Elem<DT>::to(v[u][j].e[i]), acc);
      o.e[i] = Elem<DT>::from(acc);
    }
    reinterpret_cast<typename Raw<VB>::T*>(dst)[c] = o.raw;
  }
}

// Blocks of the kernel below that an SM is to hold: loads in flight carry it, and left alone some instances
// take up to 98 registers a thread.  us, left alone / held:
//   f32, k <= 4: T = 4096, H = 5120, k = 3 92 / 89, T = 16384, H = 512, k = 2 70 / 54; bf16 8-byte rows, H = 260, k = 3
//   60 / 51; k > 4, narrow: T = 16384, H = 1026, k = 6, bf16 147 / 122, f32 (T = 10152) 148 / 102
// Warps of their own (LG = 5) with more than four slots spill at four blocks: 54 against 48 us with three at
// T = 16384, H = 512, k = 8, bf16, and 32 against 25 us at H = 124 left alone.
// 16-bit rows of a block's threads are best left alone on 16 bytes with more than four slots (held to four: T = 16384,
// H = 768, k = 8 105 / 110, H = 7168 the same) and narrower ones with four or fewer (H = 1026, k = 4 86 / 100).
// f32 rows with more than four slots are held to four blocks (64 registers, 84 bytes of spills) while short
// and to three when long: T = 15258, H = 512, k = 8 113 with three / 106 with four, T = 6781, H = 1536, k = 6 90 / 88,
// T = 2034, H = 5120, k = 6 84 / 87, T = 1089, H = 7168, k = 8 83 / 88; hence kLongChunks.
constexpr int kLongChunks = 512;
constexpr int backward_blocks(int bytes, int vb, int lg, int km, bool long_rows) {
  if (lg > 8) return 0;
  if (lg == 5) return km > 4 ? 3 : vb == 2 ? 4 : 5;
  if (bytes == 2 && (km > 4 ? vb == 16 : vb <= 4)) return 0;
  if (km > 4) return long_rows ? 3 : 4;
  return 5;
}

// The 2^LG threads of a token walk its row, U chunks at a time: every chunk of dout is read once,
// scaled into the k rows of drows and multiplied into the k dot products, which are then summed over
// the threads (warp shuffles, then shared memory in warp order: the same bits on every call).  Rounds
// lie a block apart: adjacent ones leave a row's last warps without work (261 against 225 us at T = 8192,
// H = 7168, k = 6, bf16).  A round reads its chunks of the rows before it writes them: drows may be rows.
template <int DT, int VB, int LG, int U, int KM, bool LONG>
__global__ void __launch_bounds__(LG > 8 ? 1 << LG : kRowThreads,
                                  backward_blocks(sizeof(typename Elem<DT>::T), VB, LG, KM, LONG))
    unpermute_backward_kernel(const __grid_constant__ RowsParams p) {
  using C = Chunk<DT, VB>;
  using V = typename Raw<VB>::T;
  constexpr int kTpr = 1 << LG, kThreads = LG > 8 ? kTpr : kRowThreads;
  const RowsArgs& a = p.a;
  __shared__ float part[kThreads / 32][KM];
  const int64_t t = (int64_t)blockIdx.x * (kThreads >> LG) + (threadIdx.x >> LG);
  const bool on = t < a.T;
  int r[KM];
  float w[KM], dot[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) r[j] = -1, dot[j] = 0.0f, w[j] = 1.0f;
  if (on) {
    load_rows(a, t, r);
    if (a.w != nullptr) {
#pragma unroll
      for (int j = 0; j < KM; ++j)
        if (j < a.k) w[j] = a.w[t * a.k + j];
    }
    const V* src = reinterpret_cast<const V*>(static_cast<const uint8_t*>(a.tokens_in) + t * a.token_stride * p.elem);
    for (int c0 = threadIdx.x & (kTpr - 1); c0 < p.chunks; c0 += kTpr * U) {
      C d[U], v[U][KM];
#pragma unroll
      for (int u = 0; u < U; ++u)
        d[u].raw = U == 1 || c0 + u * kTpr < p.chunks ? src[c0 + u * kTpr] : V{};
      if (a.dw != nullptr) {
#pragma unroll
        for (int j = 0; j < KM; ++j) {
          if (r[j] < 0) continue;
          const V* row = reinterpret_cast<const V*>(static_cast<const uint8_t*>(a.rows_in) +
                                                    (int64_t)r[j] * a.rows_in_stride * p.elem);
#pragma unroll
          for (int u = 0; u < U; ++u)
            v[u][j].raw = U == 1 || c0 + u * kTpr < p.chunks ? row[c0 + u * kTpr] : V{};
        }
      }
      if (a.rows_out != nullptr) {
#pragma unroll
        for (int j = 0; j < KM; ++j) {
          if (r[j] < 0) continue;
          V* row = reinterpret_cast<V*>(static_cast<uint8_t*>(a.rows_out) + (int64_t)r[j] * a.rows_out_stride * p.elem);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            C o;
#pragma unroll
            for (int i = 0; i < C::kN; ++i) o.e[i] = Elem<DT>::from(w[j] * Elem<DT>::to(d[u].e[i]));
            if (U == 1 || c0 + u * kTpr < p.chunks) row[c0 + u * kTpr] = o.raw;
          }
        }
      }
      if (a.dw != nullptr) {
#pragma unroll
        for (int j = 0; j < KM; ++j) {
          if (r[j] < 0) continue;
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < C::kN; ++i) dot[j] = fmaf(Elem<DT>::to(d[u].e[i]), Elem<DT>::to(v[u][j].e[i]), dot[j]);
        }
      }
    }
  }
  if (a.dw == nullptr) return;
#pragma unroll
  for (int j = 0; j < KM; ++j) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (LG == 5) {
    if (on && lane == 0) {
#pragma unroll
      for (int j = 0; j < KM; ++j)
        if (j < a.k) a.dw[t * a.k + j] = dot[j];
    }
    return;
  }
  if (lane == 0) {
#pragma unroll
    for (int j = 0; j < KM; ++j) part[warp][j] = dot[j];
  }
  __syncthreads();
  if (on && threadIdx.x < a.k) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) sum += part[i][threadIdx.x];
    a.dw[t * a.k + threadIdx.x] = sum;
  }
}

// One warp per token: every lane forms the k gradients and writes whole vectors of the row, each
// column the sum of the slots that selected it (a column no slot selected gets 0).
template <int V>
__global__ void __launch_bounds__(kRowThreads) route_backward_kernel(RouteBackwardArgs a) {
  const int64_t t = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  float w[kMaxTopK], g[kMaxTopK];
  int id[kMaxTopK];
  float mean = 0.0f;
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    id[j] = -1;
    w[j] = g[j] = 0.0f;
    if (j < a.k) {
      id[j] = a.ids[t * a.k + j];
      w[j] = a.w[t * a.k + j];
      g[j] = a.dw[t * a.k + j];
      mean = fmaf(w[j], g[j], mean);
    }
  }
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) g[j] = w[j] * (g[j] - mean);
  float* row = a.dlogits + t * a.E;
  for (int c = (threadIdx.x & 31) * V; c < a.E; c += 32 * V) {
    float o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      o[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < kMaxTopK; ++j)
        if (id[j] == c + i) o[i] += g[j];
    }
    if (V == 4) *reinterpret_cast<float4*>(row + c) = make_float4(o[0], o[1 % V], o[2 % V], o[3 % V]);
    else row[c] = o[0];
  }
}

// The widest access: the largest power of two up to 16 dividing every address, stride and the row.
int access_bytes(const RowsArgs& a) {
  const int64_t es = dtype_bytes(a.dtype);
  uint64_t bits = 16 | (uint64_t)(a.H * es);
  const auto with = [&](const void* ptr, int64_t stride) {
    if (ptr != nullptr) bits |= reinterpret_cast<uintptr_t>(ptr) | (uint64_t)(stride * es);
  };
  with(a.tokens_in, a.token_stride);
  with(a.tokens_out, a.token_stride);
  with(a.rows_in, a.rows_in_stride);
  with(a.rows_out, a.rows_out_stride);
  return (int)(bits & (~bits + 1));
}

// Threads per row: the power of two that leaves each thread about U chunks, at most a block.
int row_threads_log2(int chunks, int U) {
  int lg = 0;
  while (lg < 8 && (U << lg) < chunks) ++lg;
  return lg;
}

// Bytes that the threads of a row cover, U chunks of VB bytes each: the row's own and those past its end.
template <int VB, int U>
int64_t covered_bytes(const RowsArgs& a) {
  const int chunks = (int)((int64_t)a.H * dtype_bytes(a.dtype) / VB), span = U << row_threads_log2(chunks, U);
  return (int64_t)((chunks + span - 1) / span) * span * VB;
}

// The parameters of a kernel whose threads own U chunks each, and its grid.
template <int VB, int U>
RowsParams row_params(const RowsArgs& a, unsigned* blocks) {
  RowsParams p{a, a.H * dtype_bytes(a.dtype) / VB, 0, dtype_bytes(a.dtype), 1};
  p.lg = row_threads_log2(p.chunks, U);
  p.slices = (p.chunks + (U << p.lg) - 1) / (U << p.lg);
  const int64_t per = kRowThreads >> p.lg;
  *blocks = (unsigned)((a.T + per - 1) / per * p.slices);  // T <= 2^24 and 256 slices or fewer
  return p;
}

template <int VB, int U>
cudaError_t permute_vb(const RowsArgs& a, cudaStream_t s) {
  unsigned blocks = 0;
  const RowsParams p = row_params<VB, U>(a, &blocks);
  permute_kernel<VB, U><<<blocks, kRowThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int DT, int VB, int KM>
cudaError_t unpermute_vb(const RowsArgs& a, cudaStream_t s) {
  constexpr int U = VB == 16 ? 1 : 4;
  unsigned blocks = 0;
  const RowsParams p = row_params<VB, U>(a, &blocks);
  const dim3 grid(blocks / (unsigned)p.slices, (unsigned)p.slices);
  unpermute_kernel<DT, VB, U, KM><<<grid, kRowThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int DT, int VB, int KM>
cudaError_t backward_vb(const RowsArgs& a, cudaStream_t s) {
  constexpr int U = VB >= 8 ? 1 : 4;
  const RowsParams p{a, a.H * dtype_bytes(a.dtype) / VB, 0, dtype_bytes(a.dtype), 1};
  if (p.chunks <= 64 * U) {  // short rows: a warp each
    const unsigned blocks = (unsigned)((a.T + kRowThreads / 32 - 1) / (kRowThreads / 32));
    unpermute_backward_kernel<DT, VB, 5, U, KM, false><<<blocks, kRowThreads, 0, s>>>(p);
  } else if (p.chunks > 256 * U && a.T <= kFewTokens) {  // few long rows: a block of 1024 threads each
    unpermute_backward_kernel<DT, VB, 10, U, KM, false><<<(unsigned)a.T, 1024, 0, s>>>(p);
  } else {
    constexpr bool kByLength = DT == kDtF32 && VB == 16 && KM > 4;
    if (kByLength && p.chunks >= kLongChunks)
      unpermute_backward_kernel<DT, VB, 8, U, KM, kByLength><<<(unsigned)a.T, kRowThreads, 0, s>>>(p);
    else
      unpermute_backward_kernel<DT, VB, 8, U, KM, false><<<(unsigned)a.T, kRowThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

// The instance of unpermute (or its gradient) for the access width and k.
template <int DT, int VB>
cudaError_t gather_vb(const RowsArgs& a, bool backward, cudaStream_t s) {
  if (a.k <= 4) return backward ? backward_vb<DT, VB, 4>(a, s) : unpermute_vb<DT, VB, 4>(a, s);
  return backward ? backward_vb<DT, VB, kMaxTopK>(a, s) : unpermute_vb<DT, VB, kMaxTopK>(a, s);
}

template <int DT>
cudaError_t gather_typed(const RowsArgs& a, bool backward, cudaStream_t s) {
  // Rows on the 8-byte grid.  The sums take four 8-byte accesses a thread (us, 4 / 8 bytes: T = 8192, bf16, H =
  // 7164: k = 6 156 / 135, k = 3 87 / 83; T = 16384, H = 1028: k = 5 60 / 48, k = 4 38 / 34; f32, T = 7614, H = 1026,
  // k = 8 69 / 57) but for: rows that leave more of their threads' accesses unused that way (T = 12197, bf16, H = 5124, 17
  // and 37 % unused, k = 2 80 / 94), one slot of long rows (T = 16384, f32, H = 3586 107 / 125, H = 514 25 / 23) and
  // eight slots of 16-bit rows (T = 16384, H = 252 15 / 17, T = 3049, H = 5124 52 / 61; H = 1028 66 / 64).  Over 486
  // timed rows this costs 0.6 % against the faster of both, 4 bytes always 7.6.
  // The gradients take four 4-byte accesses with more than four slots (T = 16384, H = 260, bf16, k = 6 34 against
  // 173 us with one 8-byte access), and one of 8 bytes otherwise (T = 8192, H = 7164, bf16, k = 3 146 against 156).
  constexpr int kBytes = sizeof(typename Elem<DT>::T);
  switch (access_bytes(a)) {
    case 16: return gather_vb<DT, 16>(a, backward, s);
    case 8:
      if (backward) return a.k <= 4 ? backward_vb<DT, 8, 4>(a, s) : backward_vb<DT, 4, kMaxTopK>(a, s);
      if (covered_bytes<8, 4>(a) > covered_bytes<4, 4>(a) || (a.k == 1 && a.H > 2048 / kBytes) ||
          (a.k > 6 && kBytes == 2))
        return gather_vb<DT, 4>(a, backward, s);
      return a.k <= 4 ? unpermute_vb<DT, 8, 4>(a, s) : unpermute_vb<DT, 8, kMaxTopK>(a, s);
    case 4: return gather_vb<DT, 4>(a, backward, s);
    default: return gather_vb<DT, kBytes>(a, backward, s);
  }
}

cudaError_t gather(const RowsArgs& a, bool backward, cudaStream_t s) {
  if (a.dtype == kDtBf16) return gather_typed<kDtBf16>(a, backward, s);
  if (a.dtype == kDtF16) return gather_typed<kDtF16>(a, backward, s);
  return gather_typed<kDtF32>(a, backward, s);
}

}  // namespace

cudaError_t launch_permute(const RowsArgs& a, cudaStream_t s) {
  if (a.T == 0 || a.R == 0) return cudaSuccess;
  switch (access_bytes(a)) {
    case 16: return permute_vb<16, 4>(a, s);
    case 8: return permute_vb<8, 4>(a, s);
    case 4: return permute_vb<4, 8>(a, s);
    case 2: return permute_vb<2, 8>(a, s);
    default: return permute_vb<1, 8>(a, s);
  }
}

cudaError_t launch_unpermute(const RowsArgs& a, cudaStream_t s) {
  return a.T == 0 ? cudaSuccess : gather(a, false, s);
}

cudaError_t launch_unpermute_backward(const RowsArgs& a, cudaStream_t s) {
  return a.T == 0 || (a.rows_out == nullptr && a.dw == nullptr) ? cudaSuccess : gather(a, true, s);
}

cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const unsigned blocks = (unsigned)((a.T + kRowThreads / 32 - 1) / (kRowThreads / 32));
  if (a.E % 4 == 0 && reinterpret_cast<uintptr_t>(a.dlogits) % 16 == 0)
    route_backward_kernel<4><<<blocks, kRowThreads, 0, s>>>(a);
  else
    route_backward_kernel<1><<<blocks, kRowThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
