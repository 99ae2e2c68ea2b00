// expert_internal.h -- launchers of the expert-row and FP8 block-scaled operators, shared between
// their kernel files and expert_api.cu.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "moe_internal.h"

namespace moe {

constexpr int kDtBf16 = 0, kDtF16 = 1, kDtF32 = 2, kDtU8 = 3;  // moe_dtype_t
constexpr int kFp8Block = 128;                                  // FP8 scale block (1 or 128 rows x 128)

inline int dtype_bytes(int dtype) { return dtype == kDtF32 ? 4 : dtype == kDtU8 ? 1 : 2; }

// expert_rows.cu.  Strides are in elements; inv[t*k + j] outside [0, R) marks a dropped pair.
struct RowsArgs {
  const int32_t* inv;  // [T, k]
  int64_t T, R;
  int H, k, dtype;
  const void* tokens_in;  // token rows read (permute: x, unpermute backward: d_out)
  void* tokens_out;       // token rows written (unpermute: out, permute backward: dx)
  int64_t token_stride;
  const void* rows_in;    // expert rows read (unpermute, permute backward, unpermute backward)
  int64_t rows_in_stride;
  void* rows_out;         // expert rows written (permute, unpermute backward)
  int64_t rows_out_stride;
  const float* w;         // [T, k] routing weights, or null for ones
  float* dw;              // [T, k], unpermute backward only
};
cudaError_t launch_permute(const RowsArgs& a, cudaStream_t s);
cudaError_t launch_unpermute(const RowsArgs& a, cudaStream_t s);
cudaError_t launch_unpermute_backward(const RowsArgs& a, cudaStream_t s);

struct RouteBackwardArgs {
  const int32_t* ids;  // [T, k]
  const float* w;      // [T, k]
  const float* dw;     // [T, k]
  int64_t T;
  int E, k;
  float* dlogits;      // [T, E]
};
cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t s);

// quant_block.cu
struct QuantBlockArgs {
  const void* x;
  int64_t x_stride;    // elements
  int64_t rows;
  int K, dtype;
  int block_rows;      // 1 or 128 (128 only without inv)
  uint8_t* codes;      // [rows or R, K]
  float* scales;       // [rows / block_rows (rounded up) or R, K / 128 (rounded up)]
  const int32_t* inv;  // [rows, k], or null: codes and scales of row t go to row t
  int k;
  int64_t R;
};
cudaError_t launch_quant_block(const QuantBlockArgs& a, cudaStream_t s);

// gemm_block.cu.  Forward (dgrad = 0): out[r, n] = sum_c x[r, c] w[e, n, c], reduction K, N output
// columns.  dgrad = 1: out[r, c] = sum_n x[r, n] w[e, n, c], reduction N, K output columns.
struct GemmBlockArgs {
  int dgrad;
  const uint8_t* x;       // E4M3 codes [M, reduction]
  const float* x_scale;   // [M, reduction / 128 (rounded up)]
  const uint8_t* w;       // E4M3 codes [E, N, K]
  const float* w_scale;   // [E, N / 128, K / 128 (rounded up)]
  const int64_t* offsets; // [E + 1], or null: E = 1 and all M rows
  int64_t M;
  int N, K, E;
  void* out;              // [M, N] (dgrad: [M, K])
  int out_dtype;
  uint32_t* status;       // workspace status words
  uint64_t timeout_ns;
  int num_sms;
  int test_stall;
};
cudaError_t launch_gemm_block(const GemmBlockArgs& a, cudaStream_t s);
// What ran is left in status word 7 (the other words start at 0): the choice between the forms is an
// estimate, and a test or a timing that means one of them can see that it got it.
constexpr int kFormWord = 7;
enum : uint32_t { kFormVector = 1, kFormSingle = 2, kFormPair = 3, kFormSplit = 4 };
// gemv_block.cu: the forward product of a few rows, and whether a product is one.
bool use_gemv(const GemmBlockArgs& a);
cudaError_t launch_gemv_block(const GemmBlockArgs& a, cudaStream_t s);

}  // namespace moe
