// norm_device.cuh -- what the norm's and the gated block's row kernels share: 8 elements of a row at a time,
// which columns a thread owns, the sum of a row over its threads, and the quantisation of 8 elements.
#pragma once
#include "fp8_block_device.cuh"
#include "mx_device.cuh"

namespace moe {
namespace {

// The columns of a thread's chunk c.  VEC: 8 consecutive ones; else element j is 32 j further.
template <bool VEC>
struct ColumnMap {
  int first, step;
  __device__ __forceinline__ ColumnMap(int i, int tpr)
      : first(VEC ? 8 * i : (i >> 5) * 256 + (i & 31)), step(8 * tpr) {}
  __device__ __forceinline__ int col(int c) const { return first + c * step; }
};

// 16 bytes of 16-bit elements as 8 fp32 values.
template <int DT>
__device__ __forceinline__ void unpack8(uint4 r, float (&v)[8]) {
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

// The 8 elements of a chunk at column c of the row that starts at element `base`; columns from n on read as 0.
// VEC: the row starts on a 16-byte boundary and n is a multiple of 8.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* x, int64_t base, int c, int n, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  if (!VEC) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + 32 * j < n) v[j] = load1<DT>(x, base + c + 32 * j);
  } else if (c < n) {
    if (DT == kDtF32) {
      const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(x) + base + c);
      const float4 f0 = src[0], f1 = src[1];
      v[0] = f0.x, v[1] = f0.y, v[2] = f0.z, v[3] = f0.w;
      v[4] = f1.x, v[5] = f1.y, v[6] = f1.z, v[7] = f1.w;
    } else {
      unpack8<DT>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + base + c), v);
    }
  }
}

// The same as they lie in memory, 16 bytes of 16-bit elements in four registers, for kernels that hold several chunks.
template <int DT>
struct Raw8 {
  uint32_t w[DT == kDtF32 ? 8 : 4];
};
template <int DT>
__device__ __forceinline__ Raw8<DT> raw8(const void* x, int64_t base, int c, int n) {
  Raw8<DT> r;
#pragma unroll
  for (int i = 0; i < (DT == kDtF32 ? 2 : 1); ++i) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (c < n) v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) + (base + c) * (DT == kDtF32 ? 4 : 2))[i];
    r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
  }
  return r;
}
// Elements 2i and 2i + 1.
template <int DT>
__device__ __forceinline__ void raw_pair(const Raw8<DT>& r, int i, float& lo, float& hi) {
  if (DT == kDtF32) {
    lo = __uint_as_float(r.w[(2 * i) & (DT == kDtF32 ? 7 : 3)]), hi = __uint_as_float(r.w[(2 * i + 1) & (DT == kDtF32 ? 7 : 3)]);
  } else if (DT == kDtBf16) {
    lo = __uint_as_float(r.w[i] << 16), hi = __uint_as_float(r.w[i] & 0xFFFF0000u);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
    lo = f.x, hi = f.y;
  }
}

template <int DT>
__device__ __forceinline__ uint64_t raw_two(const Raw8<DT>& r, int i) {
  float lo, hi;
  raw_pair<DT>(r, i, lo, hi);
  return two(lo, hi);
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (DT == kDtBf16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int DT, bool VEC>
__device__ __forceinline__ void store8(void* x, int64_t base, int c, int n, const float (&v)[8]) {
  if (!VEC) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (c + 32 * j >= n) continue;
      if (DT == kDtF32) static_cast<float*>(x)[base + c + 32 * j] = v[j];
      else static_cast<uint16_t*>(x)[base + c + 32 * j] = (uint16_t)pack2<DT>(v[j], 0.0f);
    }
  } else if (c < n) {
    if (DT == kDtF32) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(x) + base + c);
      dst[0] = make_float4(v[0], v[1], v[2], v[3]);
      dst[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(x) + base + c) =
          make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7]));
    }
  }
}

// The chunk at column c of a row, n columns from the thread's first on; the chunk starts on a 16-byte boundary.  SHIFT
// (16-bit rows, and the weight, which may be fp32): the row may begin and end inside it; what else it holds is memory's around the row, of which `room` columns from the
// thread's first on belong to the matrix, and is trimmed where the chunk is used: a test of what was loaded would wait
// for it before the next load is on its way.
template <int DT, bool SHIFT>
__device__ __forceinline__ Raw8<DT> row_chunk(const uint8_t* row, int c, int n, int room) {
  constexpr int es = DT == kDtF32 ? 4 : 2, W = DT == kDtF32 ? 8 : 4;
  if (!SHIFT || c + 8 <= room || c >= n) return raw8<DT>(row, 0, c, n);
  Raw8<DT> r;  // the matrix's last chunk
#pragma unroll
  for (int k = 0; k < W; ++k) r.w[k] = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (c + j < 0 || c + j >= n) continue;
    if (DT == kDtF32) r.w[j & (W - 1)] = *reinterpret_cast<const uint32_t*>(row + (c + j) * es);
    else r.w[(j / 2) & (W - 1)] |= (uint32_t)*reinterpret_cast<const uint16_t*>(row + (c + j) * es) << (16 * (j & 1));
  }
  return r;
}

// Zeros in place of the first `skip` of 8 16-bit elements and of those from `left` on.
template <int DT>
__device__ __forceinline__ void trim(Raw8<DT>& r, int skip, int left) {
  static_assert(DT != kDtF32, "shifted rows are 16-bit rows");
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t lo = 2 * k < skip || 2 * k >= left ? 0u : 0xFFFFu;
    const uint32_t hi = 2 * k + 1 < skip || 2 * k + 1 >= left ? 0u : 0xFFFF0000u;
    r.w[k] &= lo | hi;
  }
}

// Elements [8 - S, 16 - S) of two neighbouring chunks.
template <int DT, int S>
__device__ __forceinline__ Raw8<DT> moved_up(const Raw8<DT>& lo, const Raw8<DT>& hi) {
  constexpr int W = DT == kDtF32 ? 8 : 4, up = 8 - S, words = DT == kDtF32 ? up : up / 2;
  Raw8<DT> r;
  auto word = [&](int k) { return k < W ? lo.w[k & (W - 1)] : hi.w[k & (W - 1)]; };
#pragma unroll
  for (int k = 0; k < W; ++k)
    r.w[k] = DT != kDtF32 && (up & 1) ? __funnelshift_r(word(k + words), word(k + words + 1), 16) : word(k + words);
  return r;
}

// 8 elements of the weight [H], which starts on a 16-byte boundary, from column c = 8 i - shift on: the two chunks that
// hold them, moved up in registers (a branch that the whole row takes alike).
template <int DT, bool SHIFT>
__device__ __forceinline__ Raw8<DT> weight_chunk(const void* w, int c, int H, int shift) {
  const uint8_t* p = static_cast<const uint8_t*>(w);
  if (!SHIFT) return raw8<DT>(p, 0, c, H);
  const int i = c + shift;
  const Raw8<DT> hi = row_chunk<DT, true>(p, i, H, H);
  if (shift == 0) return hi;
  Raw8<DT> lo = hi;
  if (i >= 8) lo = row_chunk<DT, true>(p, i - 8, H, H);
  switch (shift) {
    case 1: return moved_up<DT, 1>(lo, hi);
    case 2: return moved_up<DT, 2>(lo, hi);
    case 3: return moved_up<DT, 3>(lo, hi);
    case 4: return moved_up<DT, 4>(lo, hi);
    case 5: return moved_up<DT, 5>(lo, hi);
    case 6: return moved_up<DT, 6>(lo, hi);
    default: return moved_up<DT, 7>(lo, hi);
  }
}

// 8 values in pairs to the chunk at column c of a row; nothing from column n on, nor (SHIFT) in the first `skip`.
template <int DT, bool SHIFT>
__device__ __forceinline__ void put_chunk(uint8_t* row, int c, int n, int skip, const uint64_t (&v)[4]) {
  if (c >= n) return;
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) apart(v[j], f[2 * j], f[2 * j + 1]);
  if (!SHIFT || (c + 8 <= n && skip == 0)) {
    store8<DT, true>(row, 0, c, n, f);
    return;
  }
  static_assert(!SHIFT || DT != kDtF32, "shifted rows are 16-bit rows");
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j >= skip && c + j < n) reinterpret_cast<uint16_t*>(row)[c + j] = (uint16_t)pack2<DT>(f[j], 0.0f);
}

// The sum over the tpr threads of a row (a power of two up to 32, or whole warps), the same for all of them, in an
// order that depends on tpr alone.  rb: the row's place in the block.  Every thread of the block calls it.
__device__ __forceinline__ float row_sum(float v, int tpr, int rb) {
  __shared__ float part[32];
  if (tpr <= 32) {
    for (int o = tpr >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int nw = tpr >> 5, lane = threadIdx.x & 31;
  if (lane == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < nw ? part[rb * nw + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float lanes_max(float m, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// 8 values of a row of H columns at column c as codes with one fp32 scale per 128 columns, in rows of H codes and of
// H / 128 (rounded up) scales.  Every lane of the warp calls it; values past H are 0.
template <bool VEC>
__device__ __forceinline__ void put_fp8(uint8_t* codes, float* scales, int64_t row, int H, int c, bool on,
                                        const float (&v)[8]) {
  const int HB = (H + kFp8Block - 1) / kFp8Block;
  if (VEC) {  // 16 lanes a block
    bool infinite;
    const BlockScale sc = computed_scale(lanes_max(finite_max<8>(v, infinite), 16));
    uint32_t w[2];
    encode_computed<8>(v, sc.mult, infinite, w);
    if (!on || c >= H) return;
    *reinterpret_cast<uint2*>(codes + row * H + c) = make_uint2(w[0], w[1]);
    if ((c & (kFp8Block - 1)) == 0) scales[row * HB + c / kFp8Block] = sc.scale;
    return;
  }
#pragma unroll
  for (int b = 0; b < 2; ++b) {  // four elements of every lane a block
    bool infinite;
    const BlockScale sc = computed_scale(lanes_max(finite_max<4>(v + 4 * b, infinite), 32));
    uint32_t w[1];
    encode_computed<4>(v + 4 * b, sc.mult, infinite, w);
    const int c0 = c + 128 * b;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (on && c0 + 32 * j < H) codes[row * H + c0 + 32 * j] = (uint8_t)(w[0] >> (8 * j));
    if (on && c0 < H && (c0 & (kFp8Block - 1)) == 0) scales[row * HB + c0 / kFp8Block] = sc.scale;
  }
}

// The same for a thread's chunk of a row on an 8-byte boundary: `codes` and `scales` are the row's, `first` the thread's
// first column and codes' start, n the columns from there on.
__device__ __forceinline__ void put_fp8_chunk(uint8_t* codes, float* scales, int first, int c, int n, const float (&v)[8]) {
  bool infinite;
  const BlockScale sc = computed_scale(lanes_max(finite_max<8>(v, infinite), 16));
  uint32_t w[2];
  encode_computed<8>(v, sc.mult, infinite, w);
  if (c >= n) return;
  *reinterpret_cast<uint2*>(codes + c) = make_uint2(w[0], w[1]);
  if (((first + c) & (kFp8Block - 1)) == 0) scales[(first + c) / kFp8Block] = sc.scale;
}

// 8 values as MX codes (FMT 0: E4M3, 1: E2M1, two a byte) with one E8M0 scale per 32 columns, 4 lanes: `at` is the first
// one's place in the whole matrix, whose rows are whole blocks.
template <int FMT>
__device__ __forceinline__ void put_mx_chunk(uint8_t* codes, uint8_t* scales, int64_t at, bool on, const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
  const MxScale sc = mx_scale<FMT>(lanes_max(m, 4));
  if (!on) return;
  if (FMT == 0) *reinterpret_cast<uint2*>(codes + at) = pack_e4m3x8(v, sc.mult);
  else *reinterpret_cast<uint32_t*>(codes + at / 2) = pack_e2m1x8(v, sc.mult);
  if ((at & 31) == 0) scales[at / 32] = sc.byte;
}

// The same for single elements, one of every lane a block.
template <int FMT>
__device__ __forceinline__ void put_mx_single(uint8_t* codes, uint8_t* scales, int64_t row, int H, int c, bool on,
                                              const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const MxScale sc = mx_scale<FMT>(lanes_max(fabsf(v[j]), 32));
    const int cj = c + 32 * j;
    const float next = __shfl_down_sync(0xffffffffu, v[j], 1);
    if (!on || cj >= H) continue;
    if (FMT == 0)
      codes[row * H + cj] = (uint8_t)__nv_cvt_float2_to_fp8x2(make_float2(v[j] * sc.mult, 0.0f), __NV_SATFINITE, __NV_E4M3);
    else if ((cj & 1) == 0)
      codes[(row * H + cj) / 2] =
          (uint8_t)__nv_cvt_float2_to_fp4x2(make_float2(v[j] * sc.mult, next * sc.mult), __NV_E2M1, cudaRoundNearest);
    if ((cj & 31) == 0) scales[(row * H + cj) / 32] = sc.byte;
  }
}

}  // namespace
}  // namespace moe
