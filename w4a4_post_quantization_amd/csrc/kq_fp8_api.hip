// C ABI of the 8-bit path: host-side argument validation and dispatch to the kernels.
#include <cmath>

#include "kq.h"
#include "kq_fp8.hpp"

using namespace kq;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

kq_status hip_status(hipError_t e) { return e == hipSuccess ? KQ_OK : KQ_ERR_HIP; }

// Rows of `cols` values: M and cols at least 1, cols in whole 16-byte pieces.
kq_status check_rows(int64_t M, int64_t cols) {
  if (M < 1 || cols < 16 || cols % 16 != 0) return KQ_ERR_SHAPE;
  if (M > (1LL << 30) || cols > (1LL << 20)) return KQ_ERR_UNSUPPORTED;
  return KQ_OK;
}

bool dtype_ok(int32_t dtype) { return dtype == KQ_DT_F16 || dtype == KQ_DT_BF16; }

}  // namespace

extern "C" {

int64_t kq_fp8_scale_cols(int64_t K) { return K < 1 || K > (1LL << 20) ? 0 : f8_scale_cols(K); }

kq_status kq_quantize_fp8(int32_t dtype, const void* X, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales,
                          hipStream_t stream) {
  if (!X || !codes || !scales) return KQ_ERR_NULL;
  if (!dtype_ok(dtype)) return KQ_ERR_UNSUPPORTED;
  const kq_status st = check_rows(M, K);
  if (st != KQ_OK) return st;
  if (!aligned(X, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return KQ_ERR_ALIGN;
  return hip_status(launch_f8_quantize(dtype == KQ_DT_BF16, X, M, K, codes, scales, stream));
}

kq_status kq_rmsnorm_quantize_fp8(int32_t dtype, const void* X, const void* residual, const void* gamma, float eps,
                                  int64_t M, int64_t K, uint8_t* codes, uint8_t* scales, void* residual_out,
                                  hipStream_t stream) {
  if (!X || !gamma || !codes || !scales) return KQ_ERR_NULL;
  if (residual && !residual_out) return KQ_ERR_NULL;
  if (!dtype_ok(dtype)) return KQ_ERR_UNSUPPORTED;
  const kq_status st = check_rows(M, K);
  if (st != KQ_OK) return st;
  if (K > 16384) return KQ_ERR_UNSUPPORTED;
  if (!std::isfinite(eps) || eps < 0.0f) return KQ_ERR_VALUE;
  if (!aligned(X, 16) || !aligned(residual, 16) || !aligned(gamma, 16) || !aligned(codes, 16) || !aligned(scales, 4))
    return KQ_ERR_ALIGN;
  if (residual && !aligned(residual_out, 16)) return KQ_ERR_ALIGN;
  return hip_status(launch_f8_rmsnorm(dtype == KQ_DT_BF16, X, residual, gamma, eps, M, K, codes, scales, residual_out,
                                      stream));
}

kq_status kq_fp8_linear(int32_t dtype, const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                        const uint8_t* wcodes, const uint8_t* wscales, int64_t N, const void* bias, void* Y,
                        hipStream_t stream) {
  const bool precise = dtype & KQ_FP8_PRECISE;
  dtype &= ~KQ_FP8_PRECISE;
  if (!xcodes || !xscales || !wcodes || !wscales || !Y) return KQ_ERR_NULL;
  if (!dtype_ok(dtype)) return KQ_ERR_UNSUPPORTED;
  kq_status st = check_rows(M, K);
  if (st == KQ_OK) st = check_rows(1, N);
  if (st != KQ_OK) return st;
  if (!aligned(xcodes, 16) || !aligned(wcodes, 16) || !aligned(Y, 16) || !aligned(bias, 16)) return KQ_ERR_ALIGN;
  if (!aligned(xscales, 4) || !aligned(wscales, 4)) return KQ_ERR_ALIGN;
  return hip_status(launch_f8_linear(dtype == KQ_DT_BF16, precise, xcodes, xscales, M, K, wcodes, wscales, N, bias, Y,
                                     stream));
}

size_t kq_fp8_gated_linear_workspace_bytes(int64_t M, int64_t F, int64_t K) {
  if (check_rows(M, K) != KQ_OK || check_rows(1, F) != KQ_OK || F > (1LL << 19)) return 0;
  return f8_gated_workspace_bytes(M, F, K);
}

kq_status kq_fp8_gated_linear(int32_t act, const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                              const uint8_t* wcodes, const uint8_t* wscales, int64_t F, uint8_t* codes,
                              uint8_t* scales, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const bool precise = act & KQ_FP8_PRECISE;
  act &= ~KQ_FP8_PRECISE;
  if (!xcodes || !xscales || !wcodes || !wscales || !codes || !scales) return KQ_ERR_NULL;
  if (act < KQ_ACT_SILU || act > KQ_ACT_GELU_TANH) return KQ_ERR_UNSUPPORTED;
  kq_status st = check_rows(M, K);
  if (st == KQ_OK) st = check_rows(1, F);
  if (st != KQ_OK) return st;
  if (F > (1LL << 19)) return KQ_ERR_UNSUPPORTED;
  if (!aligned(xcodes, 16) || !aligned(wcodes, 16) || !aligned(codes, 16)) return KQ_ERR_ALIGN;
  if (!aligned(xscales, 4) || !aligned(wscales, 4) || !aligned(scales, 4)) return KQ_ERR_ALIGN;
  const size_t need = f8_gated_workspace_bytes(M, F, K);
  if (need && (!workspace || workspace_bytes < need)) return KQ_ERR_WORKSPACE;
  if (need && !aligned(workspace, 256)) return KQ_ERR_ALIGN;
  return hip_status(launch_f8_gated(act, precise, xcodes, xscales, M, K, wcodes, wscales, F, codes, scales, workspace,
                                    stream));
}

}  // extern "C"
