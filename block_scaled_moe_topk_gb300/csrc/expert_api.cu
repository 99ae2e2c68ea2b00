// expert_api.cu -- the C ABI of the expert-row and FP8 block-scaled operators: argument validation
// and one launch per call.  Nothing here allocates or synchronises.
#include <cuda_runtime.h>

#include "api_common.h"
#include "expert_internal.h"
#include "moe_topk.h"

namespace {

using moe::aligned;

constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int kMaxWidth = 65536;
constexpr size_t kGemmBlockWorkspace = 256;  // the status words

moe_status_t device_ok(int* num_sms = nullptr) {
  moe::DeviceInfo d;
  const moe_status_t st = moe::device_info(&d);
  if (st == MOE_OK && num_sms) *num_sms = d.num_sms;
  return st;
}

moe_status_t status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool float_dtype(int dtype) { return dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_F16 || dtype == MOE_DTYPE_F32; }

moe_status_t check_rows(int64_t T, int H, int k, int64_t R) {
  if (T < 0 || H <= 0 || k <= 0 || R < 0) return MOE_ERR_INVALID_ARG;
  if (T > kMaxTokens || R > kMaxRows || H > kMaxWidth || k > moe::kMaxTopK) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

// One matrix of `rows` rows: present when it has rows, a stride that holds them, element-aligned.
moe_status_t check_matrix(const void* p, int64_t rows, int64_t stride, int H, int dtype) {
  if (rows > 0 && (p == nullptr || stride < H)) return MOE_ERR_INVALID_ARG;
  if (!aligned(p, moe::dtype_bytes(dtype))) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

#define MOE_TRY(expr)                            \
  do {                                           \
    const moe_status_t st_ = (expr);             \
    if (st_ != MOE_OK) return st_;               \
  } while (0)

moe_status_t unpermute(const void* rows, int64_t rows_stride, int64_t R, moe_dtype_t dtype, const int32_t* inv,
                       const float* topk_w, int64_t T, int H, int k, void* out, int64_t out_stride, void* stream) {
  MOE_TRY(check_rows(T, H, k, R));
  if (!float_dtype(dtype)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && inv == nullptr) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_matrix(rows, T > 0 ? R : 0, rows_stride, H, dtype));
  MOE_TRY(check_matrix(out, T, out_stride, H, dtype));
  if (!aligned(inv, 4) || !aligned(topk_w, 4)) return MOE_ERR_MISALIGNED;
  if (T == 0) return MOE_OK;
  MOE_TRY(device_ok());
  moe::RowsArgs a{};
  a.inv = inv;
  a.T = T;
  a.R = R;
  a.H = H;
  a.k = k;
  a.dtype = dtype;
  a.tokens_out = out;
  a.token_stride = out_stride;
  a.rows_in = rows;
  a.rows_in_stride = rows_stride;
  a.w = topk_w;
  return status_of(moe::launch_unpermute(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t quantize(const void* x, int64_t x_stride, moe_dtype_t dtype, int64_t rows, int K, int block_rows,
                      const int32_t* inv, int k, int64_t R, uint8_t* codes, float* scales, void* stream) {
  if (rows < 0 || K <= 0 || R < 0) return MOE_ERR_INVALID_ARG;
  if (block_rows != 1 && block_rows != moe::kFp8Block) return MOE_ERR_INVALID_ARG;
  if (!float_dtype(dtype)) return MOE_ERR_INVALID_ARG;
  if (rows > kMaxRows || R > kMaxRows || K > kMaxWidth) return MOE_ERR_UNSUPPORTED_SHAPE;
  MOE_TRY(check_matrix(x, rows, x_stride, K, dtype));
  if (rows > 0 && R > 0 && (codes == nullptr || scales == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(scales, 4) || !aligned(inv, 4)) return MOE_ERR_MISALIGNED;
  if (rows == 0 || R == 0) return MOE_OK;
  MOE_TRY(device_ok());
  const moe::QuantBlockArgs a{x, x_stride, rows, K, dtype, block_rows, codes, scales, inv, k, R};
  return status_of(moe::launch_quant_block(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t check_gemm(int64_t M, int N, int K, int E) {
  if (M < 0 || N <= 0 || K <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
  if (M > kMaxRows || N > kMaxWidth || K > kMaxWidth || E > moe::kMaxExperts) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

moe_status_t gemm_block(int dgrad, const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
                        const int64_t* offsets, int64_t M, int N, int K, int E, void* out, moe_dtype_t out_dtype,
                        void* workspace, size_t workspace_bytes, void* stream) {
  MOE_TRY(check_gemm(M, N, K, E));
  if (K % 16 != 0 || (dgrad && N % 16 != 0)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!float_dtype(out_dtype)) return MOE_ERR_INVALID_ARG;
  if (offsets == nullptr && E != 1) return MOE_ERR_INVALID_ARG;
  if (!w || !w_scale || !workspace || (M > 0 && (!x || !x_scale || !out))) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(offsets, 8) ||
      !aligned(out, moe::dtype_bytes(out_dtype)) || !aligned(workspace, 256))
    return MOE_ERR_MISALIGNED;
  if (workspace_bytes < moe_gemm_fp8_block_workspace_bytes(M, N, K, E)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (M == 0) return MOE_OK;
  moe::GemmBlockArgs a{};
  MOE_TRY(device_ok(&a.num_sms));
  a.dgrad = dgrad;
  a.x = x;
  a.x_scale = x_scale;
  a.w = w;
  a.w_scale = w_scale;
  a.offsets = offsets;
  a.M = M;
  a.N = N;
  a.K = K;
  a.E = E;
  a.out = out;
  a.out_dtype = out_dtype;
  a.status = static_cast<uint32_t*>(workspace);
  a.timeout_ns = moe::wait_timeout_ns();
  a.test_stall = moe::test_stall_producer();
  return status_of(moe::launch_gemm_block(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

moe_status_t moe_permute(const void* x, int64_t x_stride, moe_dtype_t dtype, const int32_t* inv, int64_t T, int H,
                         int k, void* rows, int64_t rows_stride, int64_t R, void* stream) {
  MOE_TRY(check_rows(T, H, k, R));
  if (!float_dtype(dtype) && dtype != MOE_DTYPE_U8) return MOE_ERR_INVALID_ARG;
  if (T > 0 && inv == nullptr) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_matrix(x, T, x_stride, H, dtype));
  MOE_TRY(check_matrix(rows, T > 0 ? R : 0, rows_stride, H, dtype));
  if (!aligned(inv, 4)) return MOE_ERR_MISALIGNED;
  if (T == 0 || R == 0) return MOE_OK;
  MOE_TRY(device_ok());
  moe::RowsArgs a{};
  a.inv = inv;
  a.T = T;
  a.R = R;
  a.H = H;
  a.k = k;
  a.dtype = dtype;
  a.tokens_in = x;
  a.token_stride = x_stride;
  a.rows_out = rows;
  a.rows_out_stride = rows_stride;
  return status_of(moe::launch_permute(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_permute_backward(const void* d_rows, int64_t d_rows_stride, int64_t R, moe_dtype_t dtype,
                                  const int32_t* inv, int64_t T, int H, int k, void* d_x, int64_t d_x_stride,
                                  void* stream) {
  return unpermute(d_rows, d_rows_stride, R, dtype, inv, nullptr, T, H, k, d_x, d_x_stride, stream);
}

moe_status_t moe_unpermute(const void* rows, int64_t rows_stride, int64_t R, moe_dtype_t dtype, const int32_t* inv,
                           const float* topk_w, int64_t T, int H, int k, void* out, int64_t out_stride, void* stream) {
  if (T > 0 && topk_w == nullptr) return MOE_ERR_INVALID_ARG;
  return unpermute(rows, rows_stride, R, dtype, inv, topk_w, T, H, k, out, out_stride, stream);
}

moe_status_t moe_unpermute_backward(const void* d_out, int64_t d_out_stride, const void* rows, int64_t rows_stride,
                                    int64_t R, moe_dtype_t dtype, const int32_t* inv, const float* topk_w, int64_t T,
                                    int H, int k, void* d_rows, int64_t d_rows_stride, float* d_topk_w, void* stream) {
  MOE_TRY(check_rows(T, H, k, R));
  if (!float_dtype(dtype)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (inv == nullptr || topk_w == nullptr)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_matrix(d_out, T, d_out_stride, H, dtype));
  MOE_TRY(check_matrix(rows, T > 0 && d_topk_w ? R : 0, rows_stride, H, dtype));
  if (d_rows != nullptr) MOE_TRY(check_matrix(d_rows, R, d_rows_stride, H, dtype));
  if (!aligned(inv, 4) || !aligned(topk_w, 4) || !aligned(d_topk_w, 4)) return MOE_ERR_MISALIGNED;
  if (T == 0 || (d_rows == nullptr && d_topk_w == nullptr)) return MOE_OK;
  MOE_TRY(device_ok());
  moe::RowsArgs a{};
  a.inv = inv;
  a.T = T;
  a.R = R;
  a.H = H;
  a.k = k;
  a.dtype = dtype;
  a.tokens_in = d_out;
  a.token_stride = d_out_stride;
  if (d_topk_w != nullptr) {
    a.rows_in = rows;
    a.rows_in_stride = rows_stride;
  }
  a.rows_out = d_rows;
  a.rows_out_stride = d_rows == nullptr ? 0 : d_rows_stride;
  a.w = topk_w;
  a.dw = d_topk_w;
  return status_of(moe::launch_unpermute_backward(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_topk_route_backward(const int32_t* topk_ids, const float* topk_w, const float* d_topk_w, int64_t T,
                                     int E, int k, float* d_logits, void* stream) {
  if (T < 0 || E <= 0 || k <= 0 || k > E) return MOE_ERR_INVALID_ARG;
  if (T > kMaxTokens || E > moe::kMaxExperts || k > moe::kMaxTopK) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T > 0 && (!topk_ids || !topk_w || !d_topk_w || !d_logits)) return MOE_ERR_INVALID_ARG;
  if (!aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(d_topk_w, 4) || !aligned(d_logits, 4))
    return MOE_ERR_MISALIGNED;
  if (T == 0) return MOE_OK;
  MOE_TRY(device_ok());
  const moe::RouteBackwardArgs a{topk_ids, topk_w, d_topk_w, T, E, k, d_logits};
  return status_of(moe::launch_route_backward(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_quantize_fp8_block(const void* x, int64_t x_stride, moe_dtype_t dtype, int64_t rows, int K,
                                    int block_rows, uint8_t* codes, float* scales, void* stream) {
  return quantize(x, x_stride, dtype, rows, K, block_rows, nullptr, 1, rows, codes, scales, stream);
}

moe_status_t moe_permute_quantize_fp8_block(const void* x, int64_t x_stride, moe_dtype_t dtype, const int32_t* inv,
                                            int64_t T, int K, int k, uint8_t* codes, float* scales, int64_t R,
                                            void* stream) {
  if (k <= 0 || (T > 0 && inv == nullptr)) return MOE_ERR_INVALID_ARG;
  if (T > kMaxTokens || k > moe::kMaxTopK) return MOE_ERR_UNSUPPORTED_SHAPE;
  return quantize(x, x_stride, dtype, T, K, 1, inv, k, R, codes, scales, stream);
}

size_t moe_gemm_fp8_block_workspace_bytes(int64_t M, int N, int K, int E) {
  return check_gemm(M, N, K, E) == MOE_OK ? kGemmBlockWorkspace : 0;
}

moe_status_t moe_gemm_fp8_block(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
                                const int64_t* offsets, int64_t M, int N, int K, int E, void* out,
                                moe_dtype_t out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return gemm_block(0, x, x_scale, w, w_scale, offsets, M, N, K, E, out, out_dtype, workspace, workspace_bytes, stream);
}

moe_status_t moe_gemm_fp8_block_dgrad(const uint8_t* dy, const float* dy_scale, const uint8_t* w, const float* w_scale,
                                      const int64_t* offsets, int64_t M, int N, int K, int E, void* dx,
                                      moe_dtype_t dx_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return gemm_block(1, dy, dy_scale, w, w_scale, offsets, M, N, K, E, dx, dx_dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
