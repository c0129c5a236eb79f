// C ABI of the 8-bit path (spear_ec_q8.h): argument validation.  Every check
// runs before any HIP call; no C++ exception leaves this file.
#include "internal.hpp"
#include "q8.hpp"
#include "spear_ec_q8.h"

namespace spear {
namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int check_rows_width(int32_t rows, int32_t width) {
  if (rows < 0 || width <= 0)
    return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "rows is negative or width not positive");
  if (width % 16 != 0 || width > kQ8MaxWidth || rows > 1 << 30)
    return fail(SPEAR_EC_ERR_UNSUPPORTED, "width must be a multiple of 16 up to 65536, rows at most 2^30");
  return SPEAR_EC_OK;
}

// A matrix whose rows begin `stride` elements apart.
int check_strided(const void* p, int64_t stride, int32_t width) {
  if (!p) return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "a matrix is NULL");
  if (stride < width || stride > ((int64_t)1 << 32))
    return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "a row stride is shorter than its row or over 2^32");
  if (!aligned(p, 16) || stride % 8 != 0)
    return fail(SPEAR_EC_ERR_MISALIGNED,
                "a matrix is not 16-byte aligned or its row stride no multiple of 8 elements");
  return SPEAR_EC_OK;
}

int check_codes(const void* codes, const void* scales) {
  if (!codes || !scales)
    return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "codes and scales are required");
  if (!aligned(codes, 16)) return fail(SPEAR_EC_ERR_MISALIGNED, "codes are not 16-byte aligned");
  if (!aligned(scales, 4)) return fail(SPEAR_EC_ERR_MISALIGNED, "scales are not 4-byte aligned");
  return SPEAR_EC_OK;
}

int check_q8_desc(const spear_ec_q8_desc* d) {
  if (!d) return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->d_in <= 0 || d->d_out <= 0)
    return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "desc has a non-positive size");
  if (d->flags & ~(SPEAR_EC_OUT_F32 | SPEAR_EC_Q8_GATED | SPEAR_EC_Q8_GELU))
    return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "unknown desc.flags bits");
  if ((d->flags & SPEAR_EC_Q8_GELU) && !(d->flags & SPEAR_EC_Q8_GATED))
    return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "SPEAR_EC_Q8_GELU needs SPEAR_EC_Q8_GATED");
  if (d->d_in % 16 != 0 || d->d_in > kQ8MaxWidth)
    return fail(SPEAR_EC_ERR_UNSUPPORTED, "d_in must be a multiple of 16 up to 65536");
  if (d->d_out % 16 != 0 || d->d_out > kQ8MaxRows)
    return fail(SPEAR_EC_ERR_UNSUPPORTED, "d_out must be a multiple of 16 up to 262144");
  return SPEAR_EC_OK;
}

Q8Shape make_q8_shape(const spear_ec_q8_desc* d, int tokens) {
  return Q8Shape{d->d_in, d->d_out, tokens, (d->flags & SPEAR_EC_Q8_GATED) != 0,
                 (d->flags & SPEAR_EC_Q8_GELU) != 0, (d->flags & SPEAR_EC_OUT_F32) != 0};
}

}  // namespace
}  // namespace spear

using namespace spear;

extern "C" {

int spear_ec_q8_quantize(int32_t rows, int32_t width, const void* x, int32_t x_f32,
                         int64_t x_stride, int8_t* codes, float* scales, hipStream_t stream) {
  clear_error();
  int rc = check_rows_width(rows, width);
  if (rc || rows == 0) return rc;
  rc = check_strided(x, x_stride, width);
  if (!rc) rc = check_codes(codes, scales);
  if (rc) return rc;
  return hip_status(launch_q8_quantize(rows, width, x, x_f32 != 0, x_stride, codes, scales, stream),
                    "8-bit quantize kernel launch");
}

int spear_ec_q8_dequant_f32(int32_t rows, int32_t width, const int8_t* codes, const float* scales,
                            float* out, hipStream_t stream) {
  clear_error();
  int rc = check_rows_width(rows, width);
  if (rc || rows == 0) return rc;
  rc = check_codes(codes, scales);
  if (!rc) rc = check_strided(out, width, width);
  if (rc) return rc;
  return hip_status(launch_q8_dequant(rows, width, codes, scales, out, stream),
                    "8-bit dequant kernel launch");
}

int spear_ec_q8_rmsnorm(int32_t rows, int32_t width, const void* x, int64_t x_stride,
                        const void* residual, void* sum, const void* weight, double eps, void* y,
                        int8_t* codes, float* scales, hipStream_t stream) {
  clear_error();
  int rc = check_rows_width(rows, width);
  if (rc) return rc;
  if (!(eps > 0.0) || !(eps <= 1e300))
    return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "eps must be positive and at most 1e300");
  if (rows == 0) return SPEAR_EC_OK;
  rc = check_strided(x, x_stride, width);
  if (!rc) rc = check_strided(weight, width, width);
  if (!rc && (residual || sum)) {
    if (!residual || !sum)
      rc = fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "residual and sum are given together or not at all");
    if (!rc) rc = check_strided(residual, width, width);
    if (!rc) rc = check_strided(sum, width, width);
    if (!rc && sum == x && x_stride != width)
      rc = fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "sum in place of x needs x_stride == width");
  }
  if (!rc && !y && !codes)
    rc = fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "at least one of y and codes is required");
  if (!rc && y) rc = check_strided(y, width, width);
  if (!rc && y && (y == x || y == residual || y == sum))
    rc = fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "y must not be x, residual or sum");
  if (!rc && (codes || scales)) rc = check_codes(codes, scales);
  if (rc) return rc;
  Q8Norm a;
  a.x = static_cast<const uint16_t*>(x);
  a.x_stride = x_stride;
  a.residual = static_cast<const uint16_t*>(residual);
  a.weight = static_cast<const uint16_t*>(weight);
  a.sum = static_cast<uint16_t*>(sum);
  a.y = static_cast<uint16_t*>(y);
  a.codes = codes;
  a.scales = scales;
  a.eps = eps;
  return hip_status(launch_q8_norm(rows, width, a, stream), "8-bit norm kernel launch");
}

size_t spear_ec_q8_workspace_bytes(const spear_ec_q8_desc* desc, int32_t max_tokens) {
  if (check_q8_desc(desc) != SPEAR_EC_OK || max_tokens < 0 || max_tokens > kQ8MaxTokens) return 0;
  return q8_product_workspace(make_q8_shape(desc, max_tokens));
}

int spear_ec_q8_linear(const spear_ec_q8_desc* desc, int32_t tokens, const int8_t* xq,
                       const float* xs, const int8_t* wq, const float* ws, void* y,
                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  int rc = check_q8_desc(desc);
  if (rc) return rc;
  if (tokens < 0) return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "tokens is negative");
  if (tokens > kQ8MaxTokens || (int64_t)tokens * desc->d_out > (int64_t)1 << 37)
    return fail(SPEAR_EC_ERR_UNSUPPORTED, "at most 2^20 tokens, tokens * d_out at most 2^37");
  if (tokens == 0) return SPEAR_EC_OK;
  rc = check_codes(xq, xs);
  if (!rc) rc = check_codes(wq, ws);
  if (rc) return rc;
  if (!y) return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "y is required");
  if (!aligned(y, 16)) return fail(SPEAR_EC_ERR_MISALIGNED, "y is not 16-byte aligned");
  if (!workspace) return fail(SPEAR_EC_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned(workspace, 16))
    return fail(SPEAR_EC_ERR_MISALIGNED, "workspace is not 16-byte aligned");
  const Q8Shape s = make_q8_shape(desc, tokens);
  if (workspace_bytes < q8_product_workspace(s))
    return fail(SPEAR_EC_ERR_WORKSPACE, "workspace is smaller than spear_ec_q8_workspace_bytes()");
  return hip_status(launch_q8_product(s, Q8Product{xq, xs, wq, ws, y}, workspace, stream),
                    "8-bit product kernel launch");
}

}  // extern "C"
