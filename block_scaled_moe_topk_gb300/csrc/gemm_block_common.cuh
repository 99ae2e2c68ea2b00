// gemm_block_common.cuh -- what the kernels of the FP8 block-scaled product share: rounding to the
// output type and the clamped row ranges of the groups.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "expert_internal.h"

namespace moe {
namespace {

// Two fp32 values as the bits of two elements of a 16-bit output type.
__device__ __forceinline__ uint32_t out_pair(float lo, float hi, int dtype) {
  if (dtype == kDtBf16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// If `move`, the first S words leave (where `on`), the others move up and `at` follows.
template <int S, int WORDS>
__device__ __forceinline__ void lead_words(uint8_t*& at, uint32_t (&w)[WORDS], bool move, bool on) {
  if (on && move) {
    if (S == 1) *reinterpret_cast<uint32_t*>(at) = w[0];
    else if (S == 2) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
#pragma unroll
  for (int i = 0; i + S < WORDS; ++i) w[i] = move ? w[i + S] : w[i];
  if (move) at += 4 * S;
}

// Store WORDS - less words (WORDS a multiple of 8, less 0 or 1) at a 4-byte boundary, the body as 32-byte
// stores wherever the address lies: pieces of 1, 2 and 4 words lead up to the next 32-byte boundary, the
// words behind each piece moving up in the registers (selections: a lane's own row decides), and the
// rest trails the same way.  Every lane runs it; only lanes with `on` store.
template <int WORDS>
__device__ __forceinline__ void store_words(uint8_t* at, uint32_t (&w)[WORDS], bool on, uint32_t less = 0) {
  const uint32_t lead = (8u - (uint32_t)(reinterpret_cast<uintptr_t>(at) >> 2)) & 7u;  // words to the boundary
  if (__any_sync(0xffffffffu, lead + less != 0)) {
    lead_words<1>(at, w, (lead & 1) != 0, on);
    lead_words<2>(at, w, (lead & 2) != 0, on);
    lead_words<4>(at, w, (lead & 4) != 0, on);
  }
#pragma unroll
  for (int i = 0; i + 8 < WORDS; i += 8) {
    const uint32_t v[8] = {w[i], w[i + 1], w[i + 2], w[i + 3], w[i + 4], w[i + 5], w[i + 6], w[i + 7]};
    if (on) st_global_v8(at + 4 * i, v);
  }
  at += 4 * (WORDS - 8);
  const uint32_t rest = 8u - lead - less;  // words left: all eight when nothing led
  uint32_t t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = w[WORDS - 8 + i];
  if (on && rest == 8) {
    st_global_v8(at, t);
  } else if (on) {
    const bool four = (rest & 4) != 0, two = (rest & 2) != 0;
    if (four) *reinterpret_cast<uint4*>(at) = make_uint4(t[0], t[1], t[2], t[3]);
    const uint32_t u0 = four ? t[4] : t[0], u1 = four ? t[5] : t[1], u2 = four ? t[6] : t[2];
    if (four) at += 16;
    if (two) *reinterpret_cast<uint2*>(at) = make_uint2(u0, u1);
    if (rest & 1) *reinterpret_cast<uint32_t*>(at + (two ? 8 : 0)) = two ? u2 : u0;
  }
}

// The same for words of two 16-bit elements at any 2-byte boundary: off the 4-byte grid the first
// element and the last leave alone and the others move down by half a word.
template <int WORDS>
__device__ __forceinline__ void store_halves(uint8_t* at, uint32_t (&w)[WORDS], bool on) {
  const uint32_t odd = (uint32_t)(reinterpret_cast<uintptr_t>(at) >> 1) & 1u;
  if (__any_sync(0xffffffffu, odd != 0)) {
    if (on && odd) {
      *reinterpret_cast<uint16_t*>(at) = (uint16_t)w[0];
      *reinterpret_cast<uint16_t*>(at + 4 * WORDS - 2) = (uint16_t)(w[WORDS - 1] >> 16);
    }
#pragma unroll
    for (int i = 0; i + 1 < WORDS; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16 * odd);
  }
  store_words<WORDS>(at + 2 * odd, w, on, odd);
}

// First row of group e (e = E: the end of the last), inside [0, M] whatever the offsets hold.
// Group e has the rows from group_start(e) up to group_start(e + 1), none if that is less.
__device__ __forceinline__ int64_t group_start(const int64_t* offsets, int e, int64_t M) {
  if (offsets == nullptr) return e == 0 ? 0 : M;
  const int64_t v = offsets[e];
  return v < 0 ? 0 : (v > M ? M : v);
}

}  // namespace
}  // namespace moe
