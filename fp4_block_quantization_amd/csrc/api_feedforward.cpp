// C ABI of the feed-forward operators (RMS norm, products with an epilogue, and their
// backward passes): argument validation (before any HIP call) and kernel dispatch.  See
// include/fos.h for the contract of every entry point.
#include "../../include/fos.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "feedforward.hpp"
#include "kernels.hpp"
#include "serving.hpp"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxElems = (int64_t)1 << 40;
constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 1;   // work-items of one launch
constexpr double kMinEps = 1e-38;                         // keeps rstd finite in fp32

static_assert(FOS_ACT_NONE == fos::kActNone && FOS_ACT_RELU == fos::kActRelu &&
              FOS_ACT_GELU == fos::kActGelu && FOS_ACT_GELU_TANH == fos::kActGeluTanh &&
              FOS_ACT_SILU == fos::kActSilu, "the ABI's activations");
static_assert(FOS_RECORD_NONE == fos::kRecordNone && FOS_RECORD_NVFP4 == fos::kRecordNVFP4 &&
              FOS_RECORD_MXFP4 == fos::kRecordMXFP4, "the ABI's records");

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

fos_status status_of(hipError_t e) { return e == hipSuccess ? FOS_OK : FOS_E_HIP; }

// rows x cols of a norm.
fos_status check_norm_shape(int64_t rows, int64_t cols) {
  if (rows < 0 || rows >= kMaxDim || cols < 16 || cols > fos::kMaxNormCols || cols % 16 ||
      rows > kMaxElems / cols)
    return FOS_E_SHAPE;
  return FOS_OK;
}

// Row strides of an optional [M][N] tensor.
fos_status check_stride(const void* p, int64_t stride, int64_t M, int64_t N) {
  if (p && (stride < 0 || (M > 1 && (stride < N || stride > kMaxElems / M)))) return FOS_E_SHAPE;
  return FOS_OK;
}

fos_status check_epilogue(const fos_epilogue* e, int64_t M, int64_t N, const void* y) {
  if (!e) return FOS_E_NULL;
  if (e->struct_size != sizeof(fos_epilogue) || e->activation > FOS_ACT_SILU || e->gated > 1 ||
      (e->out_dtype != FOS_OUT_F32 && e->out_dtype != FOS_OUT_BF16) || e->reserved != 0 ||
      (e->gated && e->residual_bf16))
    return FOS_E_FLAGS;
  const fos_status st = check_stride(e->residual_bf16, e->residual_stride, M, N);
  if (st != FOS_OK) return st;
  if (!aligned(e->bias_bf16, 2) || !aligned(e->residual_bf16, 2) || !aligned(e->preact_bf16, 2) ||
      !aligned(y, e->out_dtype == FOS_OUT_F32 ? 4 : 2))
    return FOS_E_ALIGN;
  return FOS_OK;
}

fos::EpilogueArgs epilogue_args(const fos_epilogue* e, int64_t M, int64_t N, const void* y) {
  fos::EpilogueArgs a = {};
  a.bias = static_cast<const uint16_t*>(e->bias_bf16);
  a.residual = static_cast<const uint16_t*>(e->residual_bf16);
  a.residual_stride = e->residual_stride;
  a.preact = static_cast<uint16_t*>(e->preact_bf16);
  a.act = (int)e->activation;
  a.f32_out = e->out_dtype == FOS_OUT_F32;
  a.pair = N % 2 == 0 && aligned(y, 4) && aligned(e->preact_bf16, 4) &&
           (!e->residual_bf16 ||
            (aligned(e->residual_bf16, 4) && (M == 1 || e->residual_stride % 2 == 0)));
  a.quad = N % 4 == 0 && aligned(y, a.f32_out ? 16 : 8) && aligned(e->preact_bf16, 8) &&
           aligned(e->bias_bf16, 8) &&
           (!e->residual_bf16 ||
            (aligned(e->residual_bf16, 8) && (M == 1 || e->residual_stride % 4 == 0)));
  return a;
}

fos_status run_qlinear(const uint8_t* xd, const uint8_t* xs, const float* xt, const uint8_t* wd,
                       const uint8_t* ws, const float* wt, bool mx, int64_t M, int64_t N,
                       int64_t K, const fos_epilogue* e, void* y, void* stream) {
  const int64_t step = mx ? 256 : 64;
  if (M < 1 || N < 1 || K < step || K % step || M >= kMaxDim || N >= kMaxDim || K >= kMaxDim)
    return FOS_E_SHAPE;
  fos_status st = check_epilogue(e, M, N, y);
  if (st != FOS_OK) return st;
  const int64_t W = e->gated ? 2 * N : N;   // weight rows
  if (N > fos::kMaxEpilogueCols || (e->residual_bf16 && e->residual_stride > fos::kMaxResidualStride))
    return FOS_E_SHAPE;
  if (W > kMaxElems / M || K > kMaxElems / M || K > kMaxElems / W) return FOS_E_SHAPE;
  // each packed operand is addressed through one buffer resource (< 4 GiB)
  if ((M + 256) * (K / 2) >= ((int64_t)1 << 32) || (W + 256) * (K / 2) >= ((int64_t)1 << 32))
    return FOS_E_SHAPE;
  fos::QLinearArgs a = {xd, xs, wd, ws, xt, wt, M, N, K, y, e->gated != 0, {}};
  if ((mx ? fos::mx_epilogue_grid(a) : fos::qlinear_epilogue_grid(a)) > fos::kMaxGrid)
    return FOS_E_SHAPE;
  if (!xd || !xs || !wd || !ws || !y || (!mx && (!xt || !wt))) return FOS_E_NULL;
  if (!aligned(xd, 16) || !aligned(wd, 16) || !aligned(xs, 4) || !aligned(ws, 4) ||
      !aligned(xt, 4) || !aligned(wt, 4))
    return FOS_E_ALIGN;
  a.e = epilogue_args(e, M, N, y);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return status_of(mx ? fos::launch_mx_epilogue(a, s) : fos::launch_qlinear_epilogue(a, s));
}

fos_status run_wlinear(const void* x, int64_t x_stride, const uint8_t* wd, const uint8_t* ws,
                       const float* wt, bool mx, int64_t M, int64_t N, int64_t K,
                       const fos_epilogue* e, void* y, void* stream) {
  const int64_t block = mx ? 32 : 16;
  if (M < 0 || N < 1 || K < block || K % block || M >= kMaxDim || N >= kMaxDim || K >= kMaxDim)
    return FOS_E_SHAPE;
  fos_status st = check_epilogue(e, M, N, y);
  if (st != FOS_OK) return st;
  const int64_t W = e->gated ? 2 * N : N;   // weight rows
  if (W >= kMaxDim || K > kMaxElems / W || (M > 0 && (W > kMaxElems / M || K > kMaxElems / M)))
    return FOS_E_SHAPE;
  if ((st = check_stride(x, x_stride, M, K)) != FOS_OK) return st;
  if (M == 0) return FOS_OK;
  fos::WLinearArgs a = {};
  a.x = static_cast<const uint16_t*>(x);
  a.x_stride = x_stride;
  a.wd = wd;
  a.ws = ws;
  a.wt = wt;
  a.bias = static_cast<const uint16_t*>(e->bias_bf16);
  a.y = y;
  a.M = M;
  a.N = W;
  a.K = K;
  a.mx = mx;
  a.f32_out = e->out_dtype == FOS_OUT_F32;
  a.fused = true;
  a.gated = e->gated != 0;
  a.e = epilogue_args(e, M, N, y);
  if (fos::wlinear_threads(a) > kMaxThreads) return FOS_E_SHAPE;
  if (!x || !wd || !ws || !y || (!mx && !wt)) return FOS_E_NULL;
  if (!aligned(x, 16) || (M > 1 && x_stride % 8) || !aligned(wd, 16) || !aligned(ws, 4) ||
      !aligned(wt, 4))
    return FOS_E_ALIGN;
  return status_of(fos::launch_wlinear(a, static_cast<hipStream_t>(stream)));
}

// Columns of a pre-activation [M][N] (with a gate [M][2N]) whose sizes are accepted, or 0.
int64_t preact_cols(int64_t M, int64_t N, int gated) {
  if (M < 0 || N < 1 || M >= kMaxDim || N >= kMaxDim / 2 || (gated != 0 && gated != 1)) return 0;
  const int64_t width = gated ? 2 * N : N;
  if (M > kMaxElems / width || fos::epilogue_bwd_grid(M, N) > fos::kMaxGrid) return 0;
  return width;
}

}  // namespace

extern "C" {

fos_status fos_rmsnorm_fwd(const void* x_bf16, int64_t x_stride, const void* residual_bf16,
                           int64_t residual_stride, const void* weight_bf16, int64_t rows,
                           int64_t cols, double eps, void* h_bf16, float* rstd, void* y_bf16,
                           int record, int rule, uint8_t* data, uint8_t* scales,
                           float* tensor_scale, int tensor_scale_given, void* workspace,
                           size_t workspace_bytes, void* stream) {
  fos_status st = check_norm_shape(rows, cols);
  if (st != FOS_OK) return st;
  if (record < FOS_RECORD_NONE || record > FOS_RECORD_MXFP4 ||
      (rule != FOS_RULE_4OVER6 && rule != FOS_RULE_6ONLY) || !std::isfinite(eps) || eps < kMinEps)
    return FOS_E_FLAGS;
  const bool nv = record == FOS_RECORD_NVFP4, computed = nv && !tensor_scale_given;
  if (record == FOS_RECORD_MXFP4 && cols % 32) return FOS_E_SHAPE;
  if ((st = check_stride(x_bf16, x_stride, rows, cols)) != FOS_OK ||
      (st = check_stride(residual_bf16, residual_stride, rows, cols)) != FOS_OK)
    return st;
  if (nv && !tensor_scale) return FOS_E_NULL;
  if (nv && !aligned(tensor_scale, 4)) return FOS_E_ALIGN;
  if (rows > 0) {
    if (!x_bf16 || !weight_bf16 || (record == FOS_RECORD_NONE ? !y_bf16 : !data || !scales))
      return FOS_E_NULL;
    // the second launch reads what the first has stored
    if (computed && (!rstd || (residual_bf16 && !h_bf16))) return FOS_E_NULL;
    if (!aligned(x_bf16, 16) || !aligned(residual_bf16, 16) || !aligned(weight_bf16, 16) ||
        !aligned(h_bf16, 16) || !aligned(y_bf16, 16) || !aligned(rstd, 4) ||
        (rows > 1 && (x_stride % 8 || (residual_bf16 && residual_stride % 8))) ||
        (record != FOS_RECORD_NONE && !aligned(data, 8)))
      return FOS_E_ALIGN;
    if (computed && (!workspace || !aligned(workspace, 16) ||
                     workspace_bytes < fos_quantize_workspace_bytes()))
      return FOS_E_WORKSPACE;
  }
  fos::NormArgs a = {};
  a.x = static_cast<const uint16_t*>(x_bf16);
  a.r = static_cast<const uint16_t*>(residual_bf16);
  a.x_stride = x_stride;
  a.r_stride = residual_stride;
  a.w = static_cast<const uint16_t*>(weight_bf16);
  a.M = rows;
  a.K = (int)cols;
  a.eps = eps;
  a.h = static_cast<uint16_t*>(h_bf16);
  a.rstd = rstd;
  a.y = static_cast<uint16_t*>(y_bf16);
  a.record = record;
  a.four_over_six = rule == FOS_RULE_4OVER6;
  a.data = data;
  a.scales = scales;
  a.t = tensor_scale;
  a.t_given = !computed;
  a.partials = static_cast<float*>(workspace);
  return status_of(fos::launch_rmsnorm(a, static_cast<hipStream_t>(stream)));
}

size_t fos_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
  if (check_norm_shape(rows, cols) != FOS_OK) return 0;
  return sizeof(float) * (size_t)cols * (rows ? fos::norm_bwd_partials(rows, (int)cols) : 1);
}

fos_status fos_rmsnorm_bwd(const void* dy_bf16, const void* h_bf16, const void* weight_bf16,
                           const float* rstd, const void* dh_bf16, int64_t rows, int64_t cols,
                           void* dx_bf16, float* dweight, void* workspace, size_t workspace_bytes,
                           void* stream) {
  const fos_status st = check_norm_shape(rows, cols);
  if (st != FOS_OK) return st;
  if (rows > 0 && (!dy_bf16 || !h_bf16 || !weight_bf16 || !rstd || !dx_bf16)) return FOS_E_NULL;
  if (!aligned(dy_bf16, 16) || !aligned(h_bf16, 16) || !aligned(weight_bf16, 16) ||
      !aligned(rstd, 4) || !aligned(dh_bf16, 16) || !aligned(dx_bf16, 16) || !aligned(dweight, 16))
    return FOS_E_ALIGN;
  if (rows > 0 && dweight && (!workspace || !aligned(workspace, 16) ||
                              workspace_bytes < fos_rmsnorm_bwd_workspace_bytes(rows, cols)))
    return FOS_E_WORKSPACE;
  fos::NormBwdArgs a = {};
  a.dy = static_cast<const uint16_t*>(dy_bf16);
  a.h = static_cast<const uint16_t*>(h_bf16);
  a.w = static_cast<const uint16_t*>(weight_bf16);
  a.dh = static_cast<const uint16_t*>(dh_bf16);
  a.rstd = rstd;
  a.M = rows;
  a.K = (int)cols;
  a.dx = static_cast<uint16_t*>(dx_bf16);
  a.dw = dweight;
  a.partials = static_cast<float*>(workspace);
  return status_of(fos::launch_rmsnorm_bwd(a, static_cast<hipStream_t>(stream)));
}

fos_status fos_qlinear_epilogue_fwd(const uint8_t* x_data, const uint8_t* x_scales,
                                    const float* x_tensor_scale, const uint8_t* w_data,
                                    const uint8_t* w_scales, const float* w_tensor_scale,
                                    int64_t M, int64_t N, int64_t K, const fos_epilogue* epilogue,
                                    void* y, void* stream) {
  return run_qlinear(x_data, x_scales, x_tensor_scale, w_data, w_scales, w_tensor_scale, false, M,
                     N, K, epilogue, y, stream);
}

fos_status fos_mx_qlinear_epilogue_fwd(const uint8_t* a_data, const uint8_t* a_scales,
                                       const uint8_t* b_data, const uint8_t* b_scales, int64_t M,
                                       int64_t N, int64_t K, const fos_epilogue* epilogue, void* y,
                                       void* stream) {
  return run_qlinear(a_data, a_scales, nullptr, b_data, b_scales, nullptr, true, M, N, K, epilogue,
                     y, stream);
}

fos_status fos_wlinear_epilogue_fwd(const void* x_bf16, int64_t x_stride, const uint8_t* w_data,
                                    const uint8_t* w_scales, const float* w_tensor_scale,
                                    int64_t M, int64_t N, int64_t K, const fos_epilogue* epilogue,
                                    void* y, void* stream) {
  return run_wlinear(x_bf16, x_stride, w_data, w_scales, w_tensor_scale, false, M, N, K, epilogue,
                     y, stream);
}

fos_status fos_mx_wlinear_epilogue_fwd(const void* x_bf16, int64_t x_stride,
                                       const uint8_t* w_data, const uint8_t* w_scales, int64_t M,
                                       int64_t N, int64_t K, const fos_epilogue* epilogue, void* y,
                                       void* stream) {
  return run_wlinear(x_bf16, x_stride, w_data, w_scales, nullptr, true, M, N, K, epilogue, y,
                     stream);
}

size_t fos_epilogue_bwd_workspace_bytes(int64_t M, int64_t N, int gated) {
  const int64_t width = preact_cols(M, N, gated);
  if (width == 0) return 0;
  return sizeof(float) *
         ((size_t)width * fos::epilogue_bwd_groups(M, N) + (size_t)fos::epilogue_bwd_grid(M, N) + 4);
}

fos_status fos_epilogue_bwd(const void* dy_bf16, const void* preact_bf16, int64_t M, int64_t N,
                            int activation, int gated, void* dz_bf16, float* dbias,
                            float* tensor_scale, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (activation < FOS_ACT_NONE || activation > FOS_ACT_SILU || (gated != 0 && gated != 1))
    return FOS_E_FLAGS;
  if (preact_cols(M, N, gated) == 0) return FOS_E_SHAPE;
  if (M > 0 && (!dy_bf16 || !preact_bf16 || !dz_bf16)) return FOS_E_NULL;
  if (!aligned(dy_bf16, 2) || !aligned(preact_bf16, 2) || !aligned(dz_bf16, 2) ||
      !aligned(dbias, 4) || !aligned(tensor_scale, 4))
    return FOS_E_ALIGN;
  if ((dbias || tensor_scale) && (!workspace || !aligned(workspace, 16) ||
                                  workspace_bytes < fos_epilogue_bwd_workspace_bytes(M, N, gated)))
    return FOS_E_WORKSPACE;
  fos::EpilogueBwdArgs a = {};
  a.dy = static_cast<const uint16_t*>(dy_bf16);
  a.z = static_cast<const uint16_t*>(preact_bf16);
  a.M = M;
  a.N = N;
  a.act = activation;
  a.gated = gated != 0;
  a.dz = static_cast<uint16_t*>(dz_bf16);
  a.dbias = dbias;
  a.t = tensor_scale;
  a.partials = static_cast<float*>(workspace);
  return status_of(fos::launch_epilogue_bwd(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
