// C ABI of the MX operators (declared in include/w4.h): argument validation on
// the host, then the kernel launches on the caller's stream, as in w4_api.cpp.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "w4.h"
#include "w4_launch.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool valid_format(int32_t f) { return f == W4_MXFP4 || f == W4_MXFP8; }
bool valid_dtype(int32_t d) { return d == W4_F32 || d == W4_BF16 || d == W4_F16; }

constexpr int64_t kMaxBlocks = 0x7FFFFFFF;

w4_status launched(hipError_t e) { return e == hipSuccess ? W4_OK : W4_EHIP; }

// The launchers may allocate a workspace or grow a table of them; nothing they
// throw passes the C boundary.
template <typename F>
w4_status guarded(F&& f) {
  try {
    return launched(f());
  } catch (...) {
    return W4_EHIP;
  }
}

// an elementwise call over rows * k values, one block per 2048 of them
w4_status check_array(int32_t format, int64_t rows, int64_t k) {
  if (!valid_format(format) || rows < 0 || k < 0) return W4_EINVAL;
  if (k % 32) return W4_ESHAPE;
  if (k > 0 && rows > kMaxBlocks * 2048 / k) return W4_ESHAPE;
  return W4_OK;
}

w4_status check_product(int32_t x_format, int64_t n, int64_t k, int64_t m, int32_t y_dtype) {
  if (!valid_format(x_format) || n < 0 || k < 0 || m < 0) return W4_EINVAL;
  if (k % 32 || k > W4_MAX_MATMUL_K || n > W4_MAX_MX_N || m > kMaxBlocks) return W4_ESHAPE;
  if (y_dtype != W4_F32 && y_dtype != W4_BF16) return W4_EUNSUPPORTED;
  return W4_OK;
}

w4_status check_operands(const void* w, const void* ws, const void* x, const void* xs) {
  if (!w || !ws || !x || !xs) return W4_EINVAL;
  if (!aligned(w, 16) || !aligned(ws, 16) || !aligned(x, 16) || !aligned(xs, 16)) return W4_EALIGN;
  return W4_OK;
}

w4_status check_y(const void* y, int32_t y_dtype) {
  if (!y) return W4_EINVAL;
  return aligned(y, y_dtype == W4_F32 ? 4 : 2) ? W4_OK : W4_EALIGN;
}

}  // namespace

extern "C" {

w4_status w4_mx_quantize(int32_t format, int64_t rows, int64_t k, const void* x, int32_t x_dtype,
                         uint8_t* elements, uint8_t* scales, void* stream) {
  w4_status st = check_array(format, rows, k);
  if (st != W4_OK) return st;
  if (!valid_dtype(x_dtype)) return W4_EUNSUPPORTED;
  if (rows == 0 || k == 0) return W4_OK;
  if (!x || !elements || !scales) return W4_EINVAL;
  if (!aligned(x, 16) || !aligned(elements, 16) || !aligned(scales, 16)) return W4_EALIGN;
  return guarded([&] {
    return w4::launch_mx_quantize(format, rows, k, x, x_dtype, elements, scales,
                                  static_cast<hipStream_t>(stream));
  });
}

w4_status w4_mx_dequant(int32_t format, int64_t rows, int64_t k, const uint8_t* elements,
                        const uint8_t* scales, void* out, int32_t out_dtype, void* stream) {
  w4_status st = check_array(format, rows, k);
  if (st != W4_OK) return st;
  if (out_dtype != W4_F32 && out_dtype != W4_BF16) return W4_EUNSUPPORTED;
  if (rows == 0 || k == 0) return W4_OK;
  if (!elements || !scales || !out) return W4_EINVAL;
  if (!aligned(elements, 16) || !aligned(scales, 16) || !aligned(out, 16)) return W4_EALIGN;
  return guarded([&] {
    return w4::launch_mx_dequant(format, rows, k, elements, scales, out, out_dtype,
                                 static_cast<hipStream_t>(stream));
  });
}

w4_status w4_mx_rmsnorm(int32_t format, int64_t rows, int64_t k, const void* x,
                        const void* residual, const void* gamma, int32_t dtype, float eps,
                        void* residual_out, void* y, uint8_t* elements, uint8_t* scales,
                        void* stream) {
  w4_status st = check_array(format, rows, k);
  if (st != W4_OK) return st;
  if (rows > kMaxBlocks) return W4_ESHAPE;
  if (!valid_dtype(dtype)) return W4_EUNSUPPORTED;
  if (!(eps >= 0.f) || isinf(eps)) return W4_EINVAL;
  if (rows == 0 || k == 0) return W4_OK;
  if (!x || !gamma || (residual && !residual_out)) return W4_EINVAL;
  if ((!y && !elements) || (elements && !scales)) return W4_EINVAL;
  if (!aligned(x, 16) || !aligned(gamma, 16) || !aligned(residual, 16) || !aligned(y, 16) ||
      !aligned(elements, 16))
    return W4_EALIGN;
  if ((residual && !aligned(residual_out, 16)) || (elements && !aligned(scales, 16)))
    return W4_EALIGN;
  return guarded([&] {
    return w4::launch_mx_rmsnorm(format, rows, k, x, residual, gamma, dtype, eps, residual_out, y,
                                 elements, scales, static_cast<hipStream_t>(stream));
  });
}

w4_status w4_mx_linear(int32_t x_format, int64_t n, int64_t k, const uint8_t* w,
                       const uint8_t* w_scales, const uint8_t* x, const uint8_t* x_scales,
                       int64_t m, void* y, int32_t y_dtype, void* stream) {
  w4_status st = check_product(x_format, n, k, m, y_dtype);
  if (st != W4_OK) return st;
  if (m == 0 || n == 0) return W4_OK;
  st = check_y(y, y_dtype);
  if (st != W4_OK) return st;
  if (k > 0) {
    st = check_operands(w, w_scales, x, x_scales);
    if (st != W4_OK) return st;
  }
  const w4::MxProblem p{w, w_scales, x, x_scales, nullptr, nullptr, y, m, n, k, m, 1,
                        y_dtype == W4_BF16};
  if (w4::mx_linear_blocks(x_format, p) > kMaxBlocks) return W4_ESHAPE;
  return guarded([&] {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return k == 0 ? w4::launch_zero(y, m * n, y_dtype == W4_BF16, s)  // the empty sum
                  : w4::launch_mx_linear(x_format, p, s);
  });
}

w4_status w4_mx_grouped_linear(int32_t x_format, int32_t experts, int64_t n, int64_t k,
                               const uint8_t* w, const uint8_t* w_scales, int64_t tokens,
                               const uint8_t* x, const uint8_t* x_scales, int64_t rows,
                               const int32_t* offsets, const int32_t* row_index, void* y,
                               int32_t y_dtype, void* stream) {
  w4_status st = check_product(x_format, n, k, rows, y_dtype);
  if (st != W4_OK) return st;
  if (experts < 0 || tokens < 0) return W4_EINVAL;
  if (experts > W4_MX_MAX_EXPERTS || tokens > kMaxBlocks) return W4_ESHAPE;
  if (!row_index && tokens < rows) return W4_ESHAPE;
  if (rows == 0 || n == 0) return W4_OK;
  st = check_y(y, y_dtype);
  if (st != W4_OK) return st;
  // no product to compute: no terms, no weights, or (by its index, each row lies outside x) no rows of x
  const bool none = k == 0 || experts == 0 || tokens == 0;
  if (!none) {
    st = check_operands(w, w_scales, x, x_scales);
    if (st != W4_OK) return st;
    if (!offsets) return W4_EINVAL;
    if (!aligned(offsets, 4) || !aligned(row_index, 4)) return W4_EALIGN;
  }
  const w4::MxProblem p{w, w_scales, x, x_scales, offsets, row_index, y, rows, n, k, tokens,
                        experts, y_dtype == W4_BF16};
  if (!none && w4::mx_linear_blocks(x_format, p) > kMaxBlocks) return W4_ESHAPE;
  return guarded([&] {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return none ? w4::launch_zero(y, rows * n, y_dtype == W4_BF16, s)
                : w4::launch_mx_linear(x_format, p, s);
  });
}

}  // extern "C"
