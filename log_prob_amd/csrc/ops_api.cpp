// C ABI of the operators around the head: layer norm, microscaled formats and the logits
// of a head with 4-bit weights.  Every check runs on the host before the first HIP call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_util.h"
#include "flce.h"
#include "ops_internal.h"

static_assert(FLCE_BF16 == flce::kBf16 && FLCE_FP32 == flce::kF32, "element types");
static_assert(FLCE_MX_NONE == flce::kMxNone && FLCE_MXFP4 == flce::kMxFp4 &&
                  FLCE_MXFP8 == flce::kMxFp8 && FLCE_MXINT8 == flce::kMxInt8,
              "microscaled formats");

namespace {

using flce::fail;
using flce::is_aligned;
using flce::ok;

constexpr size_t kAlign = 256;

bool is_dtype(int d) { return d == FLCE_BF16 || d == FLCE_FP32; }
size_t bytes_of(int d) { return d == FLCE_BF16 ? 2 : 4; }

flce_status_t hip_fail(hipError_t e, const char* what) {
  return fail(FLCE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

flce_status_t check_rows(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0)
    return fail(FLCE_ERR_INVALID_VALUE, "rows must be >= 0 and columns positive (got %lld x %lld)",
                (long long)rows, (long long)cols);
  if (rows > flce::kMaxRows || cols > flce::kMaxHidden)
    return fail(FLCE_ERR_UNSUPPORTED, "matrix too large (limits: 2^30 rows, 2^20 columns)");
  return FLCE_OK;
}

// A matrix of rows x cols elements: row stride and natural alignment.
flce_status_t check_matrix(const char* name, const void* p, int dtype, int64_t ld, int64_t cols) {
  if (ld < cols)
    return fail(FLCE_ERR_INVALID_VALUE, "%s: row stride %lld is below its %lld columns", name,
                (long long)ld, (long long)cols);
  if (ld > (int64_t(1) << 40))
    return fail(FLCE_ERR_UNSUPPORTED, "%s: row stride too large (limit 2^40)", name);
  if (!is_aligned(p, bytes_of(dtype)))
    return fail(FLCE_ERR_UNSUPPORTED, "%s must be naturally aligned", name);
  return FLCE_OK;
}

// Whether 8 elements can be moved by whole 16-byte accesses.
bool vectors(const void* p, int dtype, int64_t ld) {
  return !p || (is_aligned(p, 16) && ld * int64_t(bytes_of(dtype)) % 16 == 0);
}

bool is_checkpoint_format(int f) { return f == FLCE_MXFP8 || f == FLCE_MXINT8; }

flce_status_t check_mx_buffers(const void* codes, const void* scales) {
  if (!codes || !scales) return fail(FLCE_ERR_INVALID_VALUE, "NULL pointer among codes, scales");
  if (!is_aligned(codes, 16) || !is_aligned(scales, 16))
    return fail(FLCE_ERR_UNSUPPORTED, "codes and scales must be 16-byte aligned");
  return FLCE_OK;
}

}  // namespace

extern "C" {

flce_status_t flce_mx_sizes(int64_t cols, int format, int64_t* code_bytes, int64_t* scale_bytes) {
  flce_status_t st = check_rows(0, cols);
  if (st != FLCE_OK) return st;
  if (format != FLCE_MXFP4 && !is_checkpoint_format(format))
    return fail(FLCE_ERR_INVALID_VALUE, "unknown microscaled format %d", format);
  if (code_bytes) *code_bytes = flce::mx_code_bytes(cols, format);
  if (scale_bytes) *scale_bytes = flce::mx_scale_bytes(cols);
  return ok();
}

flce_status_t flce_layer_norm_forward(const void* x, int x_dtype, int64_t ldx, const void* weight,
                                      const void* bias, int param_dtype, int64_t M, int64_t H,
                                      float eps, void* y, int y_dtype, int64_t ldy, float* mean,
                                      float* rstd, int format, void* codes, void* scales,
                                      hipStream_t stream) {
  flce_status_t st = check_rows(M, H);
  if (st != FLCE_OK) return st;
  if (!is_dtype(x_dtype) || !is_dtype(y_dtype) || !is_dtype(param_dtype))
    return fail(FLCE_ERR_INVALID_VALUE, "unknown element type");
  if (x_dtype == FLCE_BF16 && y_dtype == FLCE_FP32)
    return fail(FLCE_ERR_UNSUPPORTED, "fp32 output needs fp32 input");
  if (!std::isfinite(eps) || eps < 0.f)
    return fail(FLCE_ERR_INVALID_VALUE, "eps must be finite and >= 0");
  if (format != FLCE_MX_NONE && !is_checkpoint_format(format))
    return fail(FLCE_ERR_INVALID_VALUE, "checkpoint format must be none, MXFP8 or MXINT8");
  if (M == 0) return ok();
  if (!x || !y || !mean || !rstd)
    return fail(FLCE_ERR_INVALID_VALUE, "NULL pointer among x, y, mean, rstd");
  if ((st = check_matrix("x", x, x_dtype, ldx, H)) != FLCE_OK) return st;
  if ((st = check_matrix("y", y, y_dtype, ldy, H)) != FLCE_OK) return st;
  if (!is_aligned(weight, bytes_of(param_dtype)) || !is_aligned(bias, bytes_of(param_dtype)) ||
      !is_aligned(mean, 4) || !is_aligned(rstd, 4))
    return fail(FLCE_ERR_UNSUPPORTED, "weight, bias, mean and rstd must be naturally aligned");
  if (format != FLCE_MX_NONE && (st = check_mx_buffers(codes, scales)) != FLCE_OK) return st;
  flce::NormFwdArgs a{};
  a.x = x;
  a.ldx = long(ldx);
  a.weight = weight;
  a.bias = bias;
  a.param_dtype = param_dtype;
  a.M = long(M);
  a.H = int(H);
  a.eps = eps;
  a.y = y;
  a.ldy = long(ldy);
  a.mean = mean;
  a.rstd = rstd;
  a.fmt = format;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = static_cast<uint8_t*>(scales);
  const bool vec = H % 8 == 0 && vectors(x, x_dtype, ldx) && vectors(y, y_dtype, ldy) &&
                   vectors(weight, param_dtype, H) && vectors(bias, param_dtype, H);
  const hipError_t e = flce::launch_norm_fwd(a, x_dtype, y_dtype, vec, stream);
  if (e != hipSuccess) return hip_fail(e, "layer norm kernel launch");
  return ok();
}

flce_status_t flce_layer_norm_backward_workspace(int64_t M, int64_t H, size_t* bytes) {
  flce_status_t st = check_rows(M, H);
  if (st != FLCE_OK) return st;
  if (!bytes) return fail(FLCE_ERR_INVALID_VALUE, "bytes is NULL");
  *bytes = 2 * sizeof(float) * size_t(flce::norm_bwd_groups(long(M), int(H))) * size_t(H);
  return ok();
}

flce_status_t flce_layer_norm_backward(const void* dy, int dy_dtype, int64_t lddy, const void* x,
                                       int x_dtype, int64_t ldx, int format, const void* codes,
                                       const void* scales, const void* weight, int param_dtype,
                                       const float* mean, const float* rstd, int64_t M, int64_t H,
                                       void* dx, int dx_dtype, int64_t lddx, void* dweight,
                                       void* dbias, void* workspace, size_t workspace_bytes,
                                       hipStream_t stream) {
  flce_status_t st = check_rows(M, H);
  if (st != FLCE_OK) return st;
  if (!is_dtype(dy_dtype) || !is_dtype(dx_dtype) || !is_dtype(param_dtype) ||
      (x && !is_dtype(x_dtype)))
    return fail(FLCE_ERR_INVALID_VALUE, "unknown element type");
  if (x ? format != FLCE_MX_NONE : (M > 0 || format != FLCE_MX_NONE) && !is_checkpoint_format(format))
    return fail(FLCE_ERR_INVALID_VALUE,
                "give either x, with no format, or an MXFP8 or MXINT8 checkpoint");
  if (x && dx_dtype != x_dtype)
    return fail(FLCE_ERR_UNSUPPORTED, "dx must have x's element type");
  if (dx_dtype == FLCE_BF16 && dy_dtype == FLCE_FP32)
    return fail(FLCE_ERR_UNSUPPORTED, "fp32 dy needs fp32 dx");
  if (!is_aligned(dweight, bytes_of(param_dtype)) || !is_aligned(dbias, bytes_of(param_dtype)))
    return fail(FLCE_ERR_UNSUPPORTED, "dweight and dbias must be naturally aligned");
  flce::NormBwdArgs a{};
  a.groups = flce::norm_bwd_groups(long(M), int(H));
  if (M > 0) {
    if (!dy || !mean || !rstd || !dx || !workspace)
      return fail(FLCE_ERR_INVALID_VALUE, "NULL pointer among dy, mean, rstd, dx, workspace");
    if ((st = check_matrix("dy", dy, dy_dtype, lddy, H)) != FLCE_OK) return st;
    if ((st = check_matrix("dx", dx, dx_dtype, lddx, H)) != FLCE_OK) return st;
    if (x && (st = check_matrix("x", x, x_dtype, ldx, H)) != FLCE_OK) return st;
    if (!x && (st = check_mx_buffers(codes, scales)) != FLCE_OK) return st;
    if (!is_aligned(weight, bytes_of(param_dtype)) || !is_aligned(mean, 4) || !is_aligned(rstd, 4))
      return fail(FLCE_ERR_UNSUPPORTED, "weight, mean and rstd must be naturally aligned");
    if (!is_aligned(workspace, kAlign))
      return fail(FLCE_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
    const size_t need = 2 * sizeof(float) * size_t(a.groups) * size_t(H);
    if (workspace_bytes < need)
      return fail(FLCE_ERR_WORKSPACE_TOO_SMALL, "layer norm backward needs %zu workspace bytes, got %zu",
                  need, workspace_bytes);
  }
  a.dy = dy;
  a.lddy = long(lddy);
  a.x = x;
  a.ldx = long(ldx);
  a.fmt = format;
  a.codes = static_cast<const uint8_t*>(codes);
  a.scales = static_cast<const uint8_t*>(scales);
  a.weight = weight;
  a.param_dtype = param_dtype;
  a.mean = mean;
  a.rstd = rstd;
  a.M = long(M);
  a.H = int(H);
  a.dx = dx;
  a.lddx = long(lddx);
  a.params = dweight || dbias;
  a.part = static_cast<float*>(workspace);
  if (M > 0) {
    const bool vec = H % 8 == 0 && vectors(dy, dy_dtype, lddy) && vectors(dx, dx_dtype, lddx) &&
                     (!x || vectors(x, x_dtype, ldx)) && vectors(weight, param_dtype, H);
    const hipError_t e = flce::launch_norm_bwd(a, x_dtype, dy_dtype, dx_dtype, vec, stream);
    if (e != hipSuccess) return hip_fail(e, "layer norm backward kernel launch");
  }
  if (dweight || dbias) {
    const flce::NormReduceArgs r{a.part, M > 0 ? a.groups : 0, int(H), dweight, dbias, param_dtype};
    const hipError_t e = flce::launch_norm_reduce(r, stream);
    if (e != hipSuccess) return hip_fail(e, "layer norm weight gradient kernel launch");
  }
  return ok();
}

flce_status_t flce_mx_quantize(const void* x, int x_dtype, int64_t ldx, int64_t rows, int64_t cols,
                               int format, void* codes, void* scales, hipStream_t stream) {
  flce_status_t st = check_rows(rows, cols);
  if (st != FLCE_OK) return st;
  if (!is_dtype(x_dtype)) return fail(FLCE_ERR_INVALID_VALUE, "unknown element type");
  if (format != FLCE_MXFP4 && !is_checkpoint_format(format))
    return fail(FLCE_ERR_INVALID_VALUE, "unknown microscaled format %d", format);
  if (rows == 0) return ok();
  if (!x) return fail(FLCE_ERR_INVALID_VALUE, "x is NULL");
  if ((st = check_matrix("x", x, x_dtype, ldx, cols)) != FLCE_OK) return st;
  if ((st = check_mx_buffers(codes, scales)) != FLCE_OK) return st;
  const flce::MxQuantArgs a{x, long(ldx), nullptr, 0, static_cast<uint8_t*>(codes),
                            static_cast<uint8_t*>(scales), long(rows), long(cols),
                            flce::mx_row_major(cols), nullptr, {}};
  const bool vec = cols % 8 == 0 && vectors(x, x_dtype, ldx);
  const hipError_t e = flce::launch_mx_quantize(a, x_dtype, format, vec, stream);
  if (e != hipSuccess) return hip_fail(e, "quantisation kernel launch");
  return ok();
}

flce_status_t flce_mx_dequantize(const void* codes, const void* scales, int format, int64_t rows,
                                 int64_t cols, void* out, int out_dtype, int64_t ldo,
                                 hipStream_t stream) {
  flce_status_t st = check_rows(rows, cols);
  if (st != FLCE_OK) return st;
  if (!is_dtype(out_dtype)) return fail(FLCE_ERR_INVALID_VALUE, "unknown element type");
  if (format != FLCE_MXFP4 && !is_checkpoint_format(format))
    return fail(FLCE_ERR_INVALID_VALUE, "unknown microscaled format %d", format);
  if (rows == 0) return ok();
  if (!out) return fail(FLCE_ERR_INVALID_VALUE, "out is NULL");
  if ((st = check_matrix("out", out, out_dtype, ldo, cols)) != FLCE_OK) return st;
  if ((st = check_mx_buffers(codes, scales)) != FLCE_OK) return st;
  flce::MxQuantArgs a{nullptr, 0, out, long(ldo),
                      const_cast<uint8_t*>(static_cast<const uint8_t*>(codes)),
                      const_cast<uint8_t*>(static_cast<const uint8_t*>(scales)), long(rows),
                      long(cols), flce::mx_row_major(cols), nullptr, {}};
  const bool vec = cols % 8 == 0 && vectors(out, out_dtype, ldo);
  const hipError_t e = flce::launch_mx_dequantize(a, out_dtype, format, vec, stream);
  if (e != hipSuccess) return hip_fail(e, "dequantisation kernel launch");
  return ok();
}

}  // extern "C"
