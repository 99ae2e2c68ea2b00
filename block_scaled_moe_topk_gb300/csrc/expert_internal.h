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

// rms_norm*.cu.  Strides are in elements.
enum : int { kQuantNone = 0, kQuantFp8Block = 1, kQuantMx = 2 };
constexpr int kMaxNormWidth = 32768;      // columns of a row: 512 threads of 64
constexpr int64_t kSpreadRows = 2 * 152;  // up to so many rows the SMs are not filled by rows alone
struct NormArgs {
  const void* x;
  int64_t x_stride;
  const void* residual;  // or null
  int64_t residual_stride;
  int dtype;             // of x, residual, residual_out and out
  const void* weight;    // [H]
  int weight_dtype;      // dtype or fp32
  float eps;
  int64_t T;
  int H;
  void* out;             // or null (with codes)
  int64_t out_stride;
  void* residual_out;    // or null
  int64_t residual_out_stride;
  float* rstd;           // [T] or null
  int quant;             // kQuant...
  int mx_fmt;            // kQuantMx: 0 E4M3, 1 E2M1
  uint8_t* codes;        // [T, H] (E2M1: [T, H / 2])
  void* scales;          // fp32 [T, H / 128 (rounded up)], or E8M0 [T, H / 32]
};
cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t s);
cudaError_t launch_rms_norm_fp8(const NormArgs& a, cudaStream_t s);  // rms_norm_fp8.cu
cudaError_t launch_rms_norm_mx(const NormArgs& a, cudaStream_t s);   // rms_norm_mx.cu

struct NormBackwardArgs {
  const void* dy;
  int64_t dy_stride;
  const void* x;
  int64_t x_stride;
  const void* dres;      // or null
  int64_t dres_stride;
  int dtype;             // of dy, x, dres and dx
  const void* weight;    // [H]
  int weight_dtype;      // dtype or fp32
  const float* rstd;     // [T]
  int64_t T;
  int H;
  void* dx;
  int64_t dx_stride;
  float* dw;             // [H] or null
  float* partial;        // [norm_backward_parts(T, H), H] with dw
};
// How many partial sums of the weight's gradient the kernel leaves (one a block), from the sizes alone.
int norm_backward_parts(int64_t T, int H);
cudaError_t launch_rms_norm_backward(const NormBackwardArgs& a, cudaStream_t s);

// swiglu.cu
struct SwigluBackwardArgs {
  const void* gate_up;   // [R, 2I]
  int64_t gate_up_stride;
  const void* dh;        // [R, I]
  int64_t dh_stride;
  int dtype;
  int stacked;           // columns [0, I) gate, [I, 2I) up; else 2j gate, 2j + 1 up
  int64_t R;
  int I;
  void* d_gate_up;       // [R, 2I] or null
  int64_t d_gate_up_stride;
  uint8_t* codes;        // [R, 2I] or null
  float* scales;         // [R, 2I / 128 (rounded up)]
};
cudaError_t launch_swiglu_backward(const SwigluBackwardArgs& a, cudaStream_t s);

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
  // The gated product: N = 2I weight rows, out [M, I] or null (out_dtype is gate_up's type too)
  int stacked;            // rows [0, I) gate, [I, 2I) up; else 2j gate, 2j + 1 up
  void* gate_up;          // [M, 2I] or null
  uint8_t* codes;         // [M, I] or null
  float* scales;          // [M, I / 128 (rounded up)]
};
cudaError_t launch_gemm_block(const GemmBlockArgs& a, cudaStream_t s);
cudaError_t launch_gemm_swiglu(const GemmBlockArgs& a, cudaStream_t s);  // gemm_swiglu.cu
// What ran is left in status word 7 (the other words start at 0): the choice between the forms is an
// estimate, and a test or a timing that means one of them can see that it got it.
constexpr int kFormWord = 7;
enum : uint32_t { kFormVector = 1, kFormSingle = 2, kFormPair = 3, kFormSplit = 4 };
// gemv_block.cu: the forward product of a few rows, and whether a product is one.
bool use_gemv(const GemmBlockArgs& a);
cudaError_t launch_gemv_block(const GemmBlockArgs& a, cudaStream_t s);
// gemv_swiglu.cu: the same for the gated product.
bool use_gemv_swiglu(const GemmBlockArgs& a);
cudaError_t launch_gemv_swiglu(const GemmBlockArgs& a, cudaStream_t s);

}  // namespace moe
