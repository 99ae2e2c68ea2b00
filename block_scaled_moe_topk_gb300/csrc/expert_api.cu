// expert_api.cu -- the C ABI of the expert-row, norm, gated and FP8 block-scaled operators: argument
// validation and the launch (two for a norm's weight gradient).  Nothing here allocates or synchronises.
#include <cuda_runtime.h>

#include <algorithm>

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

moe_status_t rms_norm(moe::NormArgs a, void* stream) {
  if (a.T < 0 || a.H <= 0) return MOE_ERR_INVALID_ARG;
  if (!float_dtype(a.dtype) || (a.weight_dtype != a.dtype && a.weight_dtype != MOE_DTYPE_F32)) return MOE_ERR_INVALID_ARG;
  if (!(a.eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
  if (a.T > kMaxRows || a.H > moe::kMaxNormWidth) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (a.quant == moe::kQuantMx && a.H % 32 != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (a.weight == nullptr) return MOE_ERR_INVALID_ARG;
  if (a.T > 0 && a.quant == moe::kQuantNone && a.out == nullptr) return MOE_ERR_INVALID_ARG;
  if (a.T > 0 && a.quant != moe::kQuantNone && (a.codes == nullptr || a.scales == nullptr)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_matrix(a.x, a.T, a.x_stride, a.H, a.dtype));
  if (a.residual != nullptr) MOE_TRY(check_matrix(a.residual, a.T, a.residual_stride, a.H, a.dtype));
  if (a.residual_out != nullptr) MOE_TRY(check_matrix(a.residual_out, a.T, a.residual_out_stride, a.H, a.dtype));
  if (a.out != nullptr) MOE_TRY(check_matrix(a.out, a.T, a.out_stride, a.H, a.dtype));
  if (!aligned(a.weight, moe::dtype_bytes(a.weight_dtype)) || !aligned(a.rstd, 4)) return MOE_ERR_MISALIGNED;
  if (a.quant == moe::kQuantFp8Block && !aligned(a.scales, 4)) return MOE_ERR_MISALIGNED;
  if (a.T == 0) return MOE_OK;
  MOE_TRY(device_ok());
  return status_of(moe::launch_rms_norm(a, static_cast<cudaStream_t>(stream)));
}

moe::NormArgs norm_args(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                        moe_dtype_t dtype, const void* weight, moe_dtype_t weight_dtype, float eps, int64_t T, int H,
                        void* out, int64_t out_stride, void* residual_out, int64_t residual_out_stride, float* rstd) {
  moe::NormArgs a{};
  a.x = x;
  a.x_stride = x_stride;
  a.residual = residual;
  a.residual_stride = residual_stride;
  a.dtype = dtype;
  a.weight = weight;
  a.weight_dtype = weight_dtype;
  a.eps = eps;
  a.T = T;
  a.H = H;
  a.out = out;
  a.out_stride = out_stride;
  a.residual_out = residual_out;
  a.residual_out_stride = residual_out_stride;
  a.rstd = rstd;
  return a;
}

moe_status_t check_gemm(int64_t M, int N, int K, int E) {
  if (M < 0 || N <= 0 || K <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
  if (M > kMaxRows || N > kMaxWidth || K > kMaxWidth || E > moe::kMaxExperts) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

// `a` holds the pointers and sizes of a product (dgrad, or gated by `gated`); checked and launched.
moe_status_t gemm_block(moe::GemmBlockArgs a, bool gated, void* workspace, size_t workspace_bytes, void* stream) {
  MOE_TRY(check_gemm(a.M, a.N, a.K, a.E));
  if (a.K % 16 != 0 || (a.dgrad && a.N % 16 != 0)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!float_dtype(a.out_dtype)) return MOE_ERR_INVALID_ARG;
  if (a.offsets == nullptr && a.E != 1) return MOE_ERR_INVALID_ARG;
  const bool result = a.out != nullptr || (gated && a.codes != nullptr);
  if (!a.w || !a.w_scale || !workspace || (a.M > 0 && (!a.x || !a.x_scale || !result))) return MOE_ERR_INVALID_ARG;
  if (!aligned(a.x, 16) || !aligned(a.w, 16) || !aligned(a.x_scale, 4) || !aligned(a.w_scale, 4) ||
      !aligned(a.offsets, 8) || !aligned(a.out, moe::dtype_bytes(a.out_dtype)) ||
      !aligned(a.gate_up, moe::dtype_bytes(a.out_dtype)) || !aligned(a.codes, 16) || !aligned(a.scales, 4) ||
      !aligned(workspace, 256))
    return MOE_ERR_MISALIGNED;
  if (workspace_bytes < moe_gemm_fp8_block_workspace_bytes(a.M, a.N, a.K, a.E)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (a.M == 0) return MOE_OK;
  MOE_TRY(device_ok(&a.num_sms));
  a.status = static_cast<uint32_t*>(workspace);
  a.timeout_ns = moe::wait_timeout_ns();
  a.test_stall = moe::test_stall_producer();
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(gated ? moe::launch_gemm_swiglu(a, s) : moe::launch_gemm_block(a, s));
}

moe::GemmBlockArgs gemm_args(int dgrad, const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
                             const int64_t* offsets, int64_t M, int N, int K, int E, void* out, moe_dtype_t out_dtype) {
  moe::GemmBlockArgs a{};
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
  return a;
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

moe_status_t moe_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                          moe_dtype_t dtype, const void* weight, moe_dtype_t weight_dtype, float eps, int64_t T, int H,
                          void* out, int64_t out_stride, void* residual_out, int64_t residual_out_stride, float* rstd,
                          void* stream) {
  return rms_norm(norm_args(x, x_stride, residual, residual_stride, dtype, weight, weight_dtype, eps, T, H, out,
                            out_stride, residual_out, residual_out_stride, rstd), stream);
}

moe_status_t moe_rms_norm_quantize_fp8_block(const void* x, int64_t x_stride, const void* residual,
                                             int64_t residual_stride, moe_dtype_t dtype, const void* weight,
                                             moe_dtype_t weight_dtype, float eps, int64_t T, int H, uint8_t* codes,
                                             float* scales, void* out, int64_t out_stride, void* residual_out,
                                             int64_t residual_out_stride, float* rstd, void* stream) {
  moe::NormArgs a = norm_args(x, x_stride, residual, residual_stride, dtype, weight, weight_dtype, eps, T, H, out,
                              out_stride, residual_out, residual_out_stride, rstd);
  a.quant = moe::kQuantFp8Block;
  a.codes = codes;
  a.scales = scales;
  return rms_norm(a, stream);
}

moe_status_t moe_rms_norm_quantize_mx(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                                      moe_dtype_t dtype, const void* weight, moe_dtype_t weight_dtype, float eps,
                                      int64_t T, int H, moe_act_fmt_t fmt, uint8_t* codes, uint8_t* scales, void* out,
                                      int64_t out_stride, void* residual_out, int64_t residual_out_stride, float* rstd,
                                      void* stream) {
  if (fmt != MOE_ACT_MXFP8 && fmt != MOE_ACT_MXFP4) return MOE_ERR_INVALID_ARG;
  moe::NormArgs a = norm_args(x, x_stride, residual, residual_stride, dtype, weight, weight_dtype, eps, T, H, out,
                              out_stride, residual_out, residual_out_stride, rstd);
  a.quant = moe::kQuantMx;
  a.mx_fmt = fmt == MOE_ACT_MXFP8 ? 0 : 1;
  a.codes = codes;
  a.scales = scales;
  return rms_norm(a, stream);
}

size_t moe_rms_norm_backward_workspace_bytes(int64_t T, int H) {
  if (T < 0 || H <= 0 || T > kMaxRows || H > moe::kMaxNormWidth) return 0;
  return (size_t)std::max(1, moe::norm_backward_parts(T, H)) * (size_t)H * 4;
}

moe_status_t moe_rms_norm_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                   const void* d_residual, int64_t d_residual_stride, moe_dtype_t dtype,
                                   const void* weight, moe_dtype_t weight_dtype, const float* rstd, int64_t T, int H,
                                   void* dx, int64_t dx_stride, float* d_weight, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  if (T < 0 || H <= 0) return MOE_ERR_INVALID_ARG;
  if (!float_dtype(dtype) || (weight_dtype != dtype && weight_dtype != MOE_DTYPE_F32)) return MOE_ERR_INVALID_ARG;
  if (T > kMaxRows || H > moe::kMaxNormWidth) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (weight == nullptr || (T > 0 && rstd == nullptr) || (d_weight != nullptr && workspace == nullptr))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_matrix(dy, T, dy_stride, H, dtype));
  MOE_TRY(check_matrix(x, T, x_stride, H, dtype));
  if (d_residual != nullptr) MOE_TRY(check_matrix(d_residual, T, d_residual_stride, H, dtype));
  MOE_TRY(check_matrix(dx, T, dx_stride, H, dtype));
  if (!aligned(weight, moe::dtype_bytes(weight_dtype)) || !aligned(rstd, 4) || !aligned(d_weight, 4) ||
      !aligned(workspace, 256))
    return MOE_ERR_MISALIGNED;
  if (d_weight != nullptr && workspace_bytes < moe_rms_norm_backward_workspace_bytes(T, H))
    return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (T == 0 && d_weight == nullptr) return MOE_OK;
  MOE_TRY(device_ok());
  moe::NormBackwardArgs a{};
  a.dy = dy;
  a.dy_stride = dy_stride;
  a.x = x;
  a.x_stride = x_stride;
  a.dres = d_residual;
  a.dres_stride = d_residual_stride;
  a.dtype = dtype;
  a.weight = weight;
  a.weight_dtype = weight_dtype;
  a.rstd = rstd;
  a.T = T;
  a.H = H;
  a.dx = dx;
  a.dx_stride = dx_stride;
  a.dw = d_weight;
  a.partial = static_cast<float*>(workspace);
  return status_of(moe::launch_rms_norm_backward(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_swiglu_backward(const void* gate_up, int64_t gate_up_stride, const void* d_h, int64_t d_h_stride,
                                 moe_dtype_t dtype, moe_gate_up_t layout, int64_t R, int I, void* d_gate_up,
                                 int64_t d_gate_up_stride, uint8_t* codes, float* scales, void* stream) {
  if (R < 0 || I <= 0 || !float_dtype(dtype)) return MOE_ERR_INVALID_ARG;
  if (layout != MOE_GATE_UP_INTERLEAVED && layout != MOE_GATE_UP_STACKED) return MOE_ERR_INVALID_ARG;
  if (R > kMaxRows || I > kMaxWidth / 2) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (layout == MOE_GATE_UP_STACKED && I % moe::kFp8Block != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (R > 0 && d_gate_up == nullptr && codes == nullptr) return MOE_ERR_INVALID_ARG;
  if ((codes == nullptr) != (scales == nullptr)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_matrix(gate_up, R, gate_up_stride, 2 * I, dtype));
  MOE_TRY(check_matrix(d_h, R, d_h_stride, I, dtype));
  if (d_gate_up != nullptr) MOE_TRY(check_matrix(d_gate_up, R, d_gate_up_stride, 2 * I, dtype));
  if (!aligned(scales, 4)) return MOE_ERR_MISALIGNED;
  if (R == 0) return MOE_OK;
  MOE_TRY(device_ok());
  const moe::SwigluBackwardArgs a{gate_up, gate_up_stride, d_h, d_h_stride, dtype, layout == MOE_GATE_UP_STACKED, R, I,
                                  d_gate_up, d_gate_up_stride, codes, scales};
  return status_of(moe::launch_swiglu_backward(a, static_cast<cudaStream_t>(stream)));
}

size_t moe_gemm_fp8_block_workspace_bytes(int64_t M, int N, int K, int E) {
  return check_gemm(M, N, K, E) == MOE_OK ? kGemmBlockWorkspace : 0;
}

moe_status_t moe_gemm_fp8_block(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
                                const int64_t* offsets, int64_t M, int N, int K, int E, void* out,
                                moe_dtype_t out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return gemm_block(gemm_args(0, x, x_scale, w, w_scale, offsets, M, N, K, E, out, out_dtype), false, workspace,
                    workspace_bytes, stream);
}

moe_status_t moe_gemm_fp8_block_dgrad(const uint8_t* dy, const float* dy_scale, const uint8_t* w, const float* w_scale,
                                      const int64_t* offsets, int64_t M, int N, int K, int E, void* dx,
                                      moe_dtype_t dx_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return gemm_block(gemm_args(1, dy, dy_scale, w, w_scale, offsets, M, N, K, E, dx, dx_dtype), false, workspace,
                    workspace_bytes, stream);
}

moe_status_t moe_gemm_fp8_block_swiglu(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
                                       moe_gate_up_t layout, const int64_t* offsets, int64_t M, int I, int K, int E,
                                       void* out, void* gate_up, moe_dtype_t dtype, uint8_t* codes, float* scales,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  if (layout != MOE_GATE_UP_INTERLEAVED && layout != MOE_GATE_UP_STACKED) return MOE_ERR_INVALID_ARG;
  if (I <= 0 || (codes == nullptr) != (scales == nullptr)) return MOE_ERR_INVALID_ARG;
  if (I > kMaxWidth / 2 || (layout == MOE_GATE_UP_STACKED && I % moe::kFp8Block != 0) || (codes && I % 16 != 0))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  moe::GemmBlockArgs a = gemm_args(0, x, x_scale, w, w_scale, offsets, M, 2 * I, K, E, out, dtype);
  a.stacked = layout == MOE_GATE_UP_STACKED;
  a.gate_up = gate_up;
  a.codes = codes;
  a.scales = scales;
  return gemm_block(a, true, workspace, workspace_bytes, stream);
}

}  // extern "C"
