// C ABI of the products of bf16 rows with MXFP4 weights (declared in
// include/w4.h): argument validation on the host, then the kernel launches on
// the caller's stream, as in w4_mx_api.cpp.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "w4.h"
#include "w4_launch.h"
#include "w4_mx_checks.h"

namespace {

using w4::aligned;
using w4::check_y;
using w4::guarded;

constexpr int64_t kMaxRows = 0x7FFFFFFF;

// n: rows of the weight
w4_status check_sizes(int64_t n, int64_t k, int64_t m, int32_t dtype) {
  if (n < 0 || k < 0 || m < 0) return W4_EINVAL;
  if (k % 32 || k > W4_MAX_MATMUL_K || n > W4_MAX_MX_N || m > kMaxRows) return W4_ESHAPE;
  if (dtype != W4_F32 && dtype != W4_BF16) return W4_EUNSUPPORTED;
  return W4_OK;
}

// n: rows of one of the gated weight's halves
w4_status check_gated(int32_t act, int64_t n, int64_t k, int64_t m, int32_t dtype) {
  if (n < 0 || (act != W4_SILU && act != W4_GELU && act != W4_GELU_TANH)) return W4_EINVAL;
  if (n > W4_MAX_MX_N / 2) return W4_ESHAPE;
  return check_sizes(2 * n, k, m, dtype);
}

w4_status check_operands(const void* w, const void* ws, const void* x) {
  if (!w || !ws || !x) return W4_EINVAL;
  return aligned(w, 16) && aligned(ws, 16) && aligned(x, 16) ? W4_OK : W4_EALIGN;
}

w4_status launch(const w4::MxBf16Problem& p, void* stream) {
  if (!w4::mx_bf16_fits(p)) return W4_ESHAPE;
  return guarded([&] { return w4::launch_mx_bf16(p, static_cast<hipStream_t>(stream)); });
}

}  // namespace

extern "C" {

w4_status w4_mx_linear_bf16(int64_t n, int64_t k, const uint8_t* w, const uint8_t* w_scales, const uint16_t* x,
                            int64_t m, void* y, int32_t y_dtype, void* stream) {
  w4_status st = check_sizes(n, k, m, y_dtype);
  if (st != W4_OK) return st;
  if (m == 0 || n == 0) return W4_OK;
  st = check_y(y, y_dtype);
  if (st != W4_OK) return st;
  if (k == 0)  // the empty sum
    return guarded([&] { return w4::launch_zero(y, m * n, y_dtype == W4_BF16, static_cast<hipStream_t>(stream)); });
  st = check_operands(w, w_scales, x);
  if (st != W4_OK) return st;
  return launch({w, w_scales, x, y, nullptr, m, n, k, k, y_dtype == W4_BF16, 0, w4::kMxForward}, stream);
}

w4_status w4_mx_gated_linear(int32_t act, int64_t n, int64_t k, const uint8_t* w, const uint8_t* w_scales,
                             const uint16_t* x, int64_t m, uint16_t* gu, void* y, int32_t y_dtype, void* stream) {
  w4_status st = check_gated(act, n, k, m, y_dtype);
  if (st != W4_OK) return st;
  if (m == 0 || n == 0) return W4_OK;
  st = check_y(y, y_dtype);
  if (st != W4_OK) return st;
  if (!aligned(gu, 2)) return W4_EALIGN;
  if (k == 0)  // the empty sums, and act(0) = 0
    return guarded([&] {
      const hipStream_t s = static_cast<hipStream_t>(stream);
      const hipError_t e = gu ? w4::launch_zero(gu, 2 * m * n, 1, s) : hipSuccess;
      return e != hipSuccess ? e : w4::launch_zero(y, m * n, y_dtype == W4_BF16, s);
    });
  st = check_operands(w, w_scales, x);
  if (st != W4_OK) return st;
  return launch({w, w_scales, x, y, gu, m, n, k, k, y_dtype == W4_BF16, act, w4::kMxGated}, stream);
}

w4_status w4_mx_linear_grad(int64_t n, int64_t k, const uint8_t* w, const uint8_t* w_scales, const uint16_t* dy,
                            int64_t m, void* dx, int32_t dx_dtype, void* stream) {
  w4_status st = check_sizes(n, k, m, dx_dtype);
  if (st != W4_OK) return st;
  if (m == 0 || k == 0) return W4_OK;
  st = check_y(dx, dx_dtype);
  if (st != W4_OK) return st;
  if (n == 0)  // the empty sum
    return guarded([&] { return w4::launch_zero(dx, m * k, dx_dtype == W4_BF16, static_cast<hipStream_t>(stream)); });
  st = check_operands(w, w_scales, dy);
  if (st != W4_OK) return st;
  return launch({w, w_scales, dy, dx, nullptr, m, n, k, n, dx_dtype == W4_BF16, 0, w4::kMxBackward}, stream);
}

w4_status w4_mx_gated_linear_grad(int32_t act, int64_t n, int64_t k, const uint8_t* w, const uint8_t* w_scales,
                                  const uint16_t* dh, const uint16_t* gu, int64_t m, uint16_t* dgu, void* dx,
                                  int32_t dx_dtype, void* stream) {
  w4_status st = check_gated(act, n, k, m, dx_dtype);
  if (st != W4_OK) return st;
  if (m == 0) return W4_OK;
  if (k > 0) {
    st = check_y(dx, dx_dtype);
    if (st != W4_OK) return st;
  }
  if (n == 0) {  // the empty sum
    if (k == 0) return W4_OK;
    return guarded([&] { return w4::launch_zero(dx, m * k, dx_dtype == W4_BF16, static_cast<hipStream_t>(stream)); });
  }
  if (!dh || !gu || !dgu) return W4_EINVAL;
  if (!aligned(dh, 16) || !aligned(gu, 16) || !aligned(dgu, 16)) return W4_EALIGN;
  if (k > 0) {
    st = check_operands(w, w_scales, dgu);
    if (st != W4_OK) return st;
  }
  const w4::MxBf16Problem p{w, w_scales, dgu, dx, nullptr, m, 2 * n, k, 2 * n, dx_dtype == W4_BF16, 0,
                            w4::kMxBackward};
  if (k > 0 && !w4::mx_bf16_fits(p)) return W4_ESHAPE;
  return guarded([&] {
    return w4::launch_mx_gated_grad({dh, gu, dgu, m, n, act}, p, static_cast<hipStream_t>(stream));
  });
}

}  // extern "C"
