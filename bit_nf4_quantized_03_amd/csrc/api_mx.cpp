// C ABI of the microscaled formats, RMSNorm and the microscaled products:
// argument checks and dispatch. Every check runs on the host before anything
// is launched; a failed check launches nothing.
#include <cmath>
#include <cstdint>

#include "../../include/qlora_mx.h"
#include "error.h"
#include "mx.h"

namespace {

using qnf4::api_fail;

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxCols = qnf4::kMxMaxK;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool valid_shape(int64_t rows, int64_t cols) {
  return rows > 0 && cols > 0 && cols <= kMaxCols && cols % QLORA_MX_BLOCK == 0 && rows <= kMaxElems / cols;
}

bool valid_type(int type) { return type == QLORA_MX_FP4 || type == QLORA_MX_FP8; }

int check_shape(const char *fn, int64_t rows, int64_t cols) {
  if (!valid_shape(rows, cols))
    return api_fail(QLORA_ERR_SHAPE, "%s: %lld x %lld: needs rows >= 1 and cols a multiple of %d up to %lld", fn,
                    static_cast<long long>(rows), static_cast<long long>(cols), QLORA_MX_BLOCK,
                    static_cast<long long>(kMaxCols));
  return QLORA_OK;
}

int check_matrix(const char *fn, const char *name, const qlora_mx_matrix *q) {
  if (!q) return api_fail(QLORA_ERR_NULL, "%s: %s is NULL", fn, name);
  const int st = check_shape(fn, q->rows, q->cols);
  if (st != QLORA_OK) return st;
  if (!valid_type(q->type))
    return api_fail(QLORA_ERR_FORMAT, "%s: type %d of %s is not a qlora_mx_type", fn, static_cast<int>(q->type), name);
  if (!q->codes || !q->scales) return api_fail(QLORA_ERR_NULL, "%s: a buffer of %s is NULL", fn, name);
  if (!aligned16(q->codes) || !aligned16(q->scales))
    return api_fail(QLORA_ERR_ALIGN, "%s: the buffers of %s must be 16-byte aligned", fn, name);
  return QLORA_OK;
}

int check_dtype(const char *fn, const char *name, int dtype) {
  if (dtype != QLORA_F32 && dtype != QLORA_BF16)
    return api_fail(QLORA_ERR_DTYPE, "%s: %s %d is not QLORA_F32 or QLORA_BF16", fn, name, dtype);
  return QLORA_OK;
}

int check_norm_shape(const char *fn, int64_t rows, int64_t cols) {
  const int st = check_shape(fn, rows, cols);
  if (st != QLORA_OK) return st;
  if (cols > qnf4::kRmsMaxCols)
    return api_fail(QLORA_ERR_SHAPE, "%s: cols = %lld past %lld", fn, static_cast<long long>(cols),
                    static_cast<long long>(qnf4::kRmsMaxCols));
  return QLORA_OK;
}

// The checks that both forward norms share, and their arguments.
int norm_args(const char *fn, const void *X, const void *residual, const void *weight, int w_dtype, int64_t rows,
              int64_t cols, double eps, void *H, qnf4::RmsFwd *a) {
  int st = check_norm_shape(fn, rows, cols);
  if (st != QLORA_OK) return st;
  st = check_dtype(fn, "w_dtype", w_dtype);
  if (st != QLORA_OK) return st;
  if (!X || !weight) return api_fail(QLORA_ERR_NULL, "%s: X and weight must not be NULL", fn);
  if (residual && !H) return api_fail(QLORA_ERR_NULL, "%s: a residual needs H", fn);
  if (!residual && H) return api_fail(QLORA_ERR_SHAPE, "%s: without a residual H must be NULL", fn);
  if (!aligned16(X) || !aligned16(residual) || !aligned16(weight) || !aligned16(H))
    return api_fail(QLORA_ERR_ALIGN, "%s: tensors must be 16-byte aligned", fn);
  if (!(eps >= 0.0) || !std::isfinite(eps)) return api_fail(QLORA_ERR_SHAPE, "%s: eps must be finite and >= 0", fn);
  *a = qnf4::RmsFwd{};
  a->X = X;
  a->residual = residual;
  a->weight = weight;
  a->w_bf16 = w_dtype == QLORA_BF16;
  a->rows = rows;
  a->cols = cols;
  a->eps = eps;
  a->H = H;
  return QLORA_OK;
}

// The checks that both products share; n: the rows of one weight.
int check_product(const char *fn, const qlora_mx_matrix *X, const qlora_mx_matrix *W, int64_t n, const void *Y) {
  if (!Y) return api_fail(QLORA_ERR_NULL, "%s: Y must not be NULL", fn);
  if (!aligned16(Y)) return api_fail(QLORA_ERR_ALIGN, "%s: Y must be 16-byte aligned", fn);
  if (W->type != QLORA_MX_FP4) return api_fail(QLORA_ERR_FORMAT, "%s: W must hold 4-bit elements", fn);
  if (X->cols != W->cols)
    return api_fail(QLORA_ERR_SHAPE, "%s: X has %lld columns but W has %lld", fn, static_cast<long long>(X->cols),
                    static_cast<long long>(W->cols));
  if (X->rows > qnf4::kMxMaxRows || n > qnf4::kMxMaxRows || X->rows > qnf4::kMxMaxOut / n)
    return api_fail(QLORA_ERR_SHAPE, "%s: Y of %lld x %lld is too large", fn, static_cast<long long>(X->rows),
                    static_cast<long long>(n));
  return QLORA_OK;
}

qnf4::MxLinear product_args(const qlora_mx_matrix *X, const qlora_mx_matrix *W, int64_t n, void *Y) {
  qnf4::MxLinear a{};
  a.M = X->rows;
  a.N = n;
  a.K = X->cols;
  a.x_type = X->type;
  a.x = X->codes;
  a.xs = X->scales;
  a.w = W->codes;
  a.ws = W->scales;
  a.Y = Y;
  return a;
}

}  // namespace

namespace qnf4 {

int api_check_matrix(const char *fn, const char *name, const qlora_mx_matrix *q) { return check_matrix(fn, name, q); }

}  // namespace qnf4

extern "C" {

int64_t qlora_mx_scale_pitch(int64_t cols) { return valid_shape(1, cols) ? qnf4::mx_pitch(cols) : 0; }

size_t qlora_mx_storage_bytes(int64_t rows, int64_t cols, int type) {
  if (!valid_shape(rows, cols) || !valid_type(type)) return 0;
  return static_cast<size_t>(rows * (qnf4::mx_row_bytes(cols, type) + qnf4::mx_pitch(cols)));
}

int qlora_mx_quantize(const void *X, int x_dtype, int64_t rows, int64_t cols, const qlora_mx_matrix *out,
                      void *stream) {
  const char *fn = "qlora_mx_quantize";
  if (!X) return api_fail(QLORA_ERR_NULL, "%s: X is NULL", fn);
  int st = check_dtype(fn, "x_dtype", x_dtype);
  if (st != QLORA_OK) return st;
  st = check_matrix(fn, "out", out);
  if (st != QLORA_OK) return st;
  if (out->rows != rows || out->cols != cols)
    return api_fail(QLORA_ERR_SHAPE, "%s: out is %lld x %lld but X is %lld x %lld", fn,
                    static_cast<long long>(out->rows), static_cast<long long>(out->cols),
                    static_cast<long long>(rows), static_cast<long long>(cols));
  if (!aligned16(X)) return api_fail(QLORA_ERR_ALIGN, "%s: X must be 16-byte aligned", fn);
  return qnf4::api_hip_status(qnf4::launch_mx_quantize(X, x_dtype == QLORA_BF16, rows, cols, out->type, out->codes,
                                                       out->scales, static_cast<hipStream_t>(stream)), fn);
}

int qlora_mx_dequantize(const qlora_mx_matrix *q, void *out, int out_dtype, void *stream) {
  const char *fn = "qlora_mx_dequantize";
  int st = check_matrix(fn, "q", q);
  if (st != QLORA_OK) return st;
  st = check_dtype(fn, "out_dtype", out_dtype);
  if (st != QLORA_OK) return st;
  if (!out) return api_fail(QLORA_ERR_NULL, "%s: out is NULL", fn);
  if (!aligned16(out)) return api_fail(QLORA_ERR_ALIGN, "%s: out must be 16-byte aligned", fn);
  return qnf4::api_hip_status(qnf4::launch_mx_dequantize(q->codes, q->scales, q->rows, q->cols, q->type, out,
                                                         out_dtype == QLORA_BF16, static_cast<hipStream_t>(stream)),
                              fn);
}

int qlora_rmsnorm_fwd(const void *X, const void *residual, const void *weight, int w_dtype, int64_t rows,
                      int64_t cols, double eps, void *Y, void *H, float *rstd, void *stream) {
  const char *fn = "qlora_rmsnorm_fwd";
  qnf4::RmsFwd a;
  const int st = norm_args(fn, X, residual, weight, w_dtype, rows, cols, eps, H, &a);
  if (st != QLORA_OK) return st;
  if (!Y) return api_fail(QLORA_ERR_NULL, "%s: Y must not be NULL", fn);
  if (Y == H) return api_fail(QLORA_ERR_SHAPE, "%s: Y and H must differ", fn);
  if (!aligned16(Y) || !aligned16(rstd)) return api_fail(QLORA_ERR_ALIGN, "%s: tensors must be 16-byte aligned", fn);
  a.Y = Y;
  a.rstd = rstd;
  return qnf4::api_hip_status(qnf4::launch_rms_fwd(a, static_cast<hipStream_t>(stream)), fn);
}

int qlora_rmsnorm_mx(const void *X, const void *residual, const void *weight, int w_dtype, int64_t rows, int64_t cols,
                     double eps, const qlora_mx_matrix *Y, void *H, void *stream) {
  const char *fn = "qlora_rmsnorm_mx";
  int st = check_matrix(fn, "Y", Y);
  if (st != QLORA_OK) return st;
  qnf4::RmsFwd a;
  st = norm_args(fn, X, residual, weight, w_dtype, rows, cols, eps, H, &a);
  if (st != QLORA_OK) return st;
  if (Y->rows != rows || Y->cols != cols)
    return api_fail(QLORA_ERR_SHAPE, "%s: Y is %lld x %lld but X is %lld x %lld", fn,
                    static_cast<long long>(Y->rows), static_cast<long long>(Y->cols), static_cast<long long>(rows),
                    static_cast<long long>(cols));
  a.codes = Y->codes;
  a.scales = Y->scales;
  a.type = Y->type;
  return qnf4::api_hip_status(qnf4::launch_rms_fwd(a, static_cast<hipStream_t>(stream)), fn);
}

size_t qlora_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
  if (!valid_shape(rows, cols) || cols > qnf4::kRmsMaxCols) return 0;
  return qnf4::rms_bwd_ws_bytes(rows, cols);
}

int qlora_rmsnorm_bwd(const void *dY, const void *H, const void *weight, int w_dtype, const float *rstd,
                      const void *dH, int64_t rows, int64_t cols, void *dX, float *dW, void *ws, size_t ws_bytes,
                      void *stream) {
  const char *fn = "qlora_rmsnorm_bwd";
  if (!dY || !H || !weight || !rstd || !dX || !dW)
    return api_fail(QLORA_ERR_NULL, "%s: dY, H, weight, rstd, dX and dW must not be NULL", fn);
  int st = check_norm_shape(fn, rows, cols);
  if (st != QLORA_OK) return st;
  st = check_dtype(fn, "w_dtype", w_dtype);
  if (st != QLORA_OK) return st;
  if (dX == H) return api_fail(QLORA_ERR_SHAPE, "%s: dX and H must differ", fn);
  if (!aligned16(dY) || !aligned16(H) || !aligned16(weight) || !aligned16(rstd) || !aligned16(dH) || !aligned16(dX) ||
      !aligned16(dW))
    return api_fail(QLORA_ERR_ALIGN, "%s: tensors must be 16-byte aligned", fn);
  const size_t need = qnf4::rms_bwd_ws_bytes(rows, cols);
  if (need > 0 && (!ws || ws_bytes < need))
    return api_fail(QLORA_ERR_WORKSPACE, "%s: workspace needs %zu bytes, got %zu", fn, need, ws ? ws_bytes : size_t(0));
  if (!aligned16(ws)) return api_fail(QLORA_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
  return qnf4::api_hip_status(qnf4::launch_rms_bwd(dY, H, weight, w_dtype == QLORA_BF16, rstd, dH, rows, cols, dX, dW,
                                                   ws, static_cast<hipStream_t>(stream)), fn);
}

int qlora_mx_linear(const qlora_mx_matrix *X, const qlora_mx_matrix *W, void *Y, void *stream) {
  const char *fn = "qlora_mx_linear";
  int st = check_matrix(fn, "X", X);
  if (st != QLORA_OK) return st;
  st = check_matrix(fn, "W", W);
  if (st != QLORA_OK) return st;
  st = check_product(fn, X, W, W->rows, Y);
  if (st != QLORA_OK) return st;
  return qnf4::api_hip_status(qnf4::launch_mx_linear(product_args(X, W, W->rows, Y), static_cast<hipStream_t>(stream)),
                              fn);
}

int qlora_mx_linear_grouped(const qlora_mx_matrix *X, const qlora_mx_matrix *W, const int32_t *offsets,
                            int32_t experts, void *Y, void *stream) {
  const char *fn = "qlora_mx_linear_grouped";
  int st = check_matrix(fn, "X", X);
  if (st != QLORA_OK) return st;
  st = check_matrix(fn, "W", W);
  if (st != QLORA_OK) return st;
  if (experts < 1 || experts > QLORA_MX_EXPERTS || W->rows % experts != 0)
    return api_fail(QLORA_ERR_SHAPE, "%s: experts = %d must be in [1, %d] and divide W's %lld rows", fn,
                    static_cast<int>(experts), QLORA_MX_EXPERTS, static_cast<long long>(W->rows));
  if (!offsets) return api_fail(QLORA_ERR_NULL, "%s: offsets must not be NULL", fn);
  if ((reinterpret_cast<uintptr_t>(offsets) & 3u) != 0)
    return api_fail(QLORA_ERR_ALIGN, "%s: offsets must be 4-byte aligned", fn);
  if (W->rows > qnf4::kMxMaxExpertRows)
    return api_fail(QLORA_ERR_SHAPE, "%s: W has %lld rows, more than %lld", fn, static_cast<long long>(W->rows),
                    static_cast<long long>(qnf4::kMxMaxExpertRows));
  st = check_product(fn, X, W, W->rows / experts, Y);
  if (st != QLORA_OK) return st;
  qnf4::MxLinear a = product_args(X, W, W->rows / experts, Y);
  a.offsets = offsets;
  a.experts = experts;
  return qnf4::api_hip_status(qnf4::launch_mx_linear(a, static_cast<hipStream_t>(stream)), fn);
}

}  // extern "C"
