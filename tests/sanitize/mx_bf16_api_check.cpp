// Host-side check of the validation layer of the calls on bf16 rows and MXFP4
// weights (w4_mx_bf16_api.cpp), built with AddressSanitizer and
// UndefinedBehaviorSanitizer on the CPU with stub launchers: what reaches a
// launcher, what is refused before it, and that an exception thrown below the C
// boundary becomes a status.  Built and run by tests/test_mx_bf16_abi.py.
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "w4.h"
#include "w4_launch.h"

namespace {
int g_launches = 0;
bool g_throw = false, g_fits = true;
int64_t g_zeros = 0;
w4::MxBf16Problem g_last{};
w4::MxGateGrad g_gate{};
}  // namespace

namespace w4 {
bool mx_bf16_fits(const MxBf16Problem&) { return g_fits; }
hipError_t launch_mx_bf16(const MxBf16Problem& p, hipStream_t) {
  if (g_throw) throw std::bad_alloc();
  ++g_launches;
  g_last = p;
  return hipSuccess;
}
hipError_t launch_mx_gated_grad(const MxGateGrad& g, const MxBf16Problem& p, hipStream_t) {
  if (g_throw) throw std::bad_alloc();
  ++g_launches;
  g_gate = g;
  g_last = p;
  return hipErrorInvalidValue;  // a failed launch
}
hipError_t launch_zero(void*, int64_t count, int, hipStream_t) {
  g_zeros += count;
  return hipSuccess;
}
}  // namespace w4

namespace {
int failures = 0;
#define EXPECT(c)                                            \
  do {                                                       \
    if (!(c)) {                                              \
      fprintf(stderr, "FAIL line %d: %s\n", __LINE__, #c);   \
      ++failures;                                            \
    }                                                        \
  } while (0)
uint8_t* P(uintptr_t a) { return reinterpret_cast<uint8_t*>(a); }
uint16_t* H(uintptr_t a) { return reinterpret_cast<uint16_t*>(a); }
}  // namespace

int main() {
  const uintptr_t A = 0x10000;
  EXPECT(w4_mx_linear_bf16(16, 64, P(A), P(A), H(A), 3, P(A), W4_BF16, nullptr) == W4_OK && g_launches == 1);
  EXPECT(g_last.kind == w4::kMxForward && g_last.m == 3 && g_last.n == 16 && g_last.k == 64);
  EXPECT(g_last.x_pitch == 64 && g_last.y_bf16 == 1 && g_last.gu == nullptr);
  EXPECT(w4_mx_gated_linear(W4_GELU, 16, 64, P(A), P(A), H(A), 3, H(A + 2), P(A + 4), W4_F32, nullptr) == W4_OK);
  EXPECT(g_last.kind == w4::kMxGated && g_last.n == 16 && g_last.act == W4_GELU && g_last.gu == H(A + 2));
  EXPECT(w4_mx_linear_grad(17, 64, P(A), P(A), H(A), 3, P(A), W4_F32, nullptr) == W4_OK);
  EXPECT(g_last.kind == w4::kMxBackward && g_last.n == 17 && g_last.x_pitch == 17 && g_last.y_bf16 == 0);
  EXPECT(w4_mx_gated_linear_grad(W4_SILU, 17, 64, P(A), P(A), H(A), H(A + 64), 3, H(A + 128), P(A), W4_BF16,
                                 nullptr) == W4_EHIP);
  EXPECT(g_last.n == 34 && g_last.x_pitch == 34 && g_last.x == H(A + 128) && g_last.kind == w4::kMxBackward);
  EXPECT(g_gate.n == 17 && g_gate.gu == H(A + 64) && g_gate.dgu == H(A + 128) && g_gate.m == 3);
  // sizes that wrap when doubled or multiplied
  EXPECT(w4_mx_gated_linear(0, INT64_MAX, 64, P(A), P(A), H(A), 3, H(A), P(A), W4_F32, nullptr) == W4_ESHAPE);
  EXPECT(w4_mx_gated_linear(0, INT64_MIN, 64, P(A), P(A), H(A), 3, H(A), P(A), W4_F32, nullptr) == W4_EINVAL);
  EXPECT(w4_mx_gated_linear_grad(0, INT64_MIN, 64, P(A), P(A), H(A), H(A), 3, H(A), P(A), W4_F32, nullptr) ==
         W4_EINVAL);
  g_fits = false;
  g_launches = 0;
  EXPECT(w4_mx_linear_bf16(16, 64, P(A), P(A), H(A), 3, P(A), W4_BF16, nullptr) == W4_ESHAPE);
  EXPECT(w4_mx_gated_linear_grad(0, 16, 64, P(A), P(A), H(A), H(A), 3, H(A), P(A), W4_F32, nullptr) == W4_ESHAPE);
  EXPECT(g_launches == 0);
  g_fits = true;
  g_throw = true;
  EXPECT(w4_mx_linear_grad(16, 64, P(A), P(A), H(A), 3, P(A), W4_BF16, nullptr) == W4_EHIP);
  EXPECT(w4_mx_gated_linear_grad(0, 16, 64, P(A), P(A), H(A), H(A), 3, H(A), P(A), W4_F32, nullptr) == W4_EHIP);
  g_throw = false;
  // empty sums: zeros, whatever the other pointers are
  EXPECT(w4_mx_linear_bf16(16, 0, nullptr, nullptr, nullptr, 3, P(A), W4_F32, nullptr) == W4_OK && g_zeros == 48);
  g_zeros = 0;
  EXPECT(w4_mx_gated_linear(0, 16, 0, nullptr, nullptr, nullptr, 3, H(A), P(A), W4_F32, nullptr) == W4_OK);
  EXPECT(g_zeros == 48 + 96);
  g_zeros = 0;
  EXPECT(w4_mx_linear_grad(0, 64, nullptr, nullptr, nullptr, 3, P(A), W4_F32, nullptr) == W4_OK && g_zeros == 192);
  g_zeros = 0;
  EXPECT(w4_mx_gated_linear_grad(0, 0, 64, nullptr, nullptr, nullptr, nullptr, 3, nullptr, P(A), W4_F32, nullptr) ==
         W4_OK && g_zeros == 192);
  // without columns dgu is computed all the same
  g_launches = 0;
  EXPECT(w4_mx_gated_linear_grad(0, 16, 0, nullptr, nullptr, H(A), H(A), 3, H(A), nullptr, W4_F32, nullptr) ==
         W4_EHIP && g_launches == 1 && g_last.k == 0);
  if (failures) {
    fprintf(stderr, "%d failures\n", failures);
    return 1;
  }
  printf("mx_bf16_api_check ok\n");
  return 0;
}
