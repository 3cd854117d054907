// layer.cu -- host side of include/ag_layer.h's norm and gated activation: argument checks
// and launches.  (The 4-bit products share a plan with the others: moe.cu.)
#include "ag_layer.h"

#include <cmath>

#include "checks.h"
#include "host.h"
#include "layer_rows.cuh"

using agg::aligned16;
using agg::fail;
using agg::float_type;
using agg::kMaxRowLen;
using agg::launched;

namespace {

int check_rows(int64_t rows, int64_t cols, int dtype) {
  if (!float_type(dtype)) return fail(AG_GEMM_ERR_INVALID, "rows must be fp16, bf16 or fp32 (got type %d)", dtype);
  if (rows < 0 || cols < 1)
    return fail(AG_GEMM_ERR_INVALID, "need rows >= 0 and a length >= 1 (got %lld, %lld)", (long long)rows, (long long)cols);
  if (rows >= (1LL << 31) || cols > kMaxRowLen)
    return fail(AG_GEMM_ERR_UNSUPPORTED, "at most 2^31 - 1 rows of %lld columns", (long long)kMaxRowLen);
  return AG_GEMM_OK;
}

int check_weight(int weight_dtype, int dtype) {
  if (weight_dtype != dtype && weight_dtype != AG_MOE_F32)
    return fail(AG_GEMM_ERR_INVALID, "weights must have the rows' type or be fp32 (got type %d)", weight_dtype);
  return AG_GEMM_OK;
}

int check_pitch(const char* name, int64_t ld, int64_t cols) {
  if (ld < cols)
    return fail(AG_GEMM_ERR_INVALID, "%s: row pitch %lld is less than %lld columns", name, (long long)ld, (long long)cols);
  if (ld >= (1LL << 36)) return fail(AG_GEMM_ERR_UNSUPPORTED, "%s: row pitch too large", name);
  return AG_GEMM_OK;
}

// Codes with scales as an output: whole 16 bytes of codes a row.
int check_codes(int code_type, int64_t cols, const void* q, const void* scales) {
  if (code_type != AG_MOE_E4M3 && code_type != AG_MOE_E2M1)
    return fail(AG_GEMM_ERR_INVALID, "code_type must be AG_MOE_E4M3 or AG_MOE_E2M1 (got %d)", code_type);
  const int unit = code_type == AG_MOE_E4M3 ? 16 : 32;
  if (cols % unit != 0)
    return fail(AG_GEMM_ERR_INVALID, "rows of these codes must be a multiple of %d long (got %lld)", unit, (long long)cols);
  if (!q || !scales || !aligned16(q) || !aligned16(scales))
    return fail(AG_GEMM_ERR_INVALID, "q and scales must be 16-byte aligned and not NULL");
  return AG_GEMM_OK;
}

int norm_args(agg::NormArgs& a, int64_t rows, int64_t H, int dtype, const void* x, int64_t ldx, const void* residual,
              int64_t ldr, const void* weight, int weight_dtype, float eps, void* h) {
  if (int rc = check_rows(rows, H, dtype)) return rc;
  if (int rc = check_weight(weight_dtype, dtype)) return rc;
  if (!(eps >= 0.0f) || std::isinf(eps)) return fail(AG_GEMM_ERR_INVALID, "eps must be a number from 0 on");
  if (rows > 0) {
    if (!x || !weight || (residual && !h)) return fail(AG_GEMM_ERR_INVALID, "a pointer is NULL");
    if (int rc = check_pitch("x", ldx, H)) return rc;
    if (residual)
      if (int rc = check_pitch("residual", ldr, H)) return rc;
  }
  a = agg::NormArgs{};
  a.rows = rows;
  a.H = H;
  a.x = x;
  a.ldx = ldx;
  a.residual = residual;
  a.ldr = ldr;
  a.weight = weight;
  a.weight_f32 = weight_dtype == AG_MOE_F32;
  a.eps = eps;
  a.h = h;
  return AG_GEMM_OK;
}

}  // namespace

extern "C" {

int ag_norm_rms(int64_t rows, int64_t H, int dtype, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                const void* weight, int weight_dtype, float eps, void* y, void* h, float* rstd, void* stream) {
  agg::NormArgs a;
  if (int rc = norm_args(a, rows, H, dtype, x, ldx, residual, ldr, weight, weight_dtype, eps, h)) return rc;
  if (rows == 0) return AG_GEMM_OK;
  if (!y) return fail(AG_GEMM_ERR_INVALID, "y is NULL");
  a.out = y;
  a.rstd = rstd;
  return launched(agg::launch_norm(a, dtype, dtype, static_cast<cudaStream_t>(stream)), "norm launch");
}

int ag_norm_rms_quantized(int64_t rows, int64_t H, int dtype, const void* x, int64_t ldx, const void* residual,
                          int64_t ldr, const void* weight, int weight_dtype, float eps, int code_type, void* q,
                          void* scales, void* h, void* stream) {
  agg::NormArgs a;
  if (int rc = norm_args(a, rows, H, dtype, x, ldx, residual, ldr, weight, weight_dtype, eps, h)) return rc;
  if (rows == 0) return AG_GEMM_OK;
  if (int rc = check_codes(code_type, H, q, scales)) return rc;
  if (int rc = agg::check_matrix("x", x, ldx, H, dtype)) return rc;
  if (residual)
    if (int rc = agg::check_matrix("residual", residual, ldr, H, dtype)) return rc;
  if (!aligned16(weight) || (residual && !aligned16(h)))
    return fail(AG_GEMM_ERR_INVALID, "weight and h must be 16-byte aligned");
  a.out = q;
  a.scales = scales;
  return launched(agg::launch_norm(a, dtype, code_type, static_cast<cudaStream_t>(stream)), "norm launch");
}

int64_t ag_norm_rms_backward_workspace(int64_t rows, int64_t H) {
  if (int rc = check_rows(rows, H, AG_MOE_F32)) return rc;
  return agg::norm_parts(rows) * H * 4;
}

int ag_norm_rms_backward(int64_t rows, int64_t H, int dtype, const void* dy, int64_t lddy, const void* h, int64_t ldh,
                         const void* weight, int weight_dtype, const float* rstd, const void* dh, int64_t lddh, void* dx,
                         float* dweight, void* workspace, void* stream) {
  if (int rc = check_rows(rows, H, dtype)) return rc;
  if (int rc = check_weight(weight_dtype, dtype)) return rc;
  if (!dweight) return fail(AG_GEMM_ERR_INVALID, "dweight is NULL");
  if (rows > 0) {
    if (!dy || !h || !weight || !rstd || !dx || !workspace) return fail(AG_GEMM_ERR_INVALID, "a pointer is NULL");
    if (!aligned16(workspace)) return fail(AG_GEMM_ERR_INVALID, "workspace must be 16-byte aligned");
    if (int rc = check_pitch("dy", lddy, H)) return rc;
    if (int rc = check_pitch("h", ldh, H)) return rc;
    if (dh)
      if (int rc = check_pitch("dh", lddh, H)) return rc;
  }
  agg::NormBackwardArgs a{};
  a.rows = rows;
  a.H = H;
  a.dy = dy;
  a.lddy = lddy;
  a.h = h;
  a.ldh = ldh;
  a.weight = weight;
  a.weight_f32 = weight_dtype == AG_MOE_F32;
  a.rstd = rstd;
  a.dh = dh;
  a.lddh = lddh;
  a.dx = dx;
  a.dweight = dweight;
  a.parts = static_cast<float*>(workspace);
  return launched(agg::launch_norm_backward(a, dtype, static_cast<cudaStream_t>(stream)), "norm gradient launch");
}

int ag_act_swiglu(int64_t rows, int64_t N, int dtype, const void* x, int64_t ldx, void* y, void* stream) {
  if (int rc = check_rows(rows, N, dtype)) return rc;
  if (rows == 0) return AG_GEMM_OK;
  if (!x || !y) return fail(AG_GEMM_ERR_INVALID, "a pointer is NULL");
  if (int rc = check_pitch("x", ldx, 2 * N)) return rc;
  agg::GateArgs a{};
  a.rows = rows;
  a.N = N;
  a.x = x;
  a.ldx = ldx;
  a.out = y;
  return launched(agg::launch_swiglu(a, dtype, dtype, static_cast<cudaStream_t>(stream)), "activation launch");
}

int ag_act_swiglu_quantized(int64_t rows, int64_t N, int dtype, const void* x, int64_t ldx, int code_type, void* q,
                            void* scales, void* stream) {
  if (int rc = check_rows(rows, N, dtype)) return rc;
  if (rows == 0) return AG_GEMM_OK;
  if (int rc = check_codes(code_type, N, q, scales)) return rc;
  if (int rc = agg::check_matrix("x", x, ldx, 2 * N, dtype)) return rc;
  agg::GateArgs a{};
  a.rows = rows;
  a.N = N;
  a.x = x;
  a.ldx = ldx;
  a.out = q;
  a.scales = scales;
  return launched(agg::launch_swiglu(a, dtype, code_type, static_cast<cudaStream_t>(stream)), "activation launch");
}

int ag_act_swiglu_backward(int64_t rows, int64_t N, int dtype, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                           void* dx, void* stream) {
  if (int rc = check_rows(rows, N, dtype)) return rc;
  if (rows == 0) return AG_GEMM_OK;
  if (!dy || !x || !dx) return fail(AG_GEMM_ERR_INVALID, "a pointer is NULL");
  if (int rc = check_pitch("dy", lddy, N)) return rc;
  if (int rc = check_pitch("x", ldx, 2 * N)) return rc;
  agg::GateArgs a{};
  a.rows = rows;
  a.N = N;
  a.x = x;
  a.ldx = ldx;
  a.dy = dy;
  a.lddy = lddy;
  a.out = dx;
  return launched(agg::launch_swiglu_backward(a, dtype, static_cast<cudaStream_t>(stream)), "activation gradient launch");
}

}  // extern "C"
