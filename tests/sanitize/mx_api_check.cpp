// Host-side check of the MX calls' validation layer (w4_mx_api.cpp), built with
// AddressSanitizer and UndefinedBehaviorSanitizer on the CPU with stub
// launchers: what reaches a launcher, what is refused before it, and that an
// exception thrown below the C boundary becomes a status.  Built and run by
// tests/test_mx_abi.py.
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "w4.h"
#include "w4_launch.h"

namespace {
int g_launches = 0;
bool g_throw = false;
int64_t g_zero = -1, g_blocks = 1;
w4::MxProblem g_last{};
}  // namespace

namespace w4 {
hipError_t launch_mx_quantize(int, int64_t, int64_t, const void*, int, uint8_t*, uint8_t*, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_mx_dequant(int, int64_t, int64_t, const uint8_t*, const uint8_t*, void*, int, hipStream_t) {
  ++g_launches;
  return hipErrorInvalidValue;
}
hipError_t launch_mx_rmsnorm(int, int64_t, int64_t, const void*, const void*, const void*, int, float, void*,
                             void*, uint8_t*, uint8_t*, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
int64_t mx_linear_blocks(int, const MxProblem&) { return g_blocks; }
hipError_t launch_mx_linear(int, const MxProblem& p, hipStream_t) {
  if (g_throw) throw std::bad_alloc();
  ++g_launches;
  g_last = p;
  return hipSuccess;
}
hipError_t launch_zero(void*, int64_t count, int, hipStream_t) {
  ++g_launches;
  g_zero = count;
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
int32_t* I(uintptr_t a) { return reinterpret_cast<int32_t*>(a); }
}  // namespace

int main() {
  const uintptr_t A = 0x10000;
  EXPECT(w4_mx_quantize(0, 4, 64, P(A), W4_F16, P(A), P(A), nullptr) == W4_OK && g_launches == 1);
  EXPECT(w4_mx_quantize(0, INT64_MAX, 64, P(A), W4_F16, P(A), P(A), nullptr) == W4_ESHAPE);
  EXPECT(w4_mx_quantize(0, 1, INT64_MAX - 31, P(A), W4_F16, P(A), P(A), nullptr) == W4_ESHAPE);
  EXPECT(w4_mx_dequant(1, 4, 64, P(A), P(A), P(A), W4_F32, nullptr) == W4_EHIP);  // a failed launch
  EXPECT(w4_mx_rmsnorm(1, 4, 64, P(A), nullptr, P(A), W4_BF16, 0.f, nullptr, nullptr, P(A), P(A), nullptr) ==
         W4_OK);
  EXPECT(w4_mx_rmsnorm(1, 4, 64, P(A), nullptr, P(A), W4_BF16, 0.f, P(A + 8), P(A), nullptr, P(A + 1), nullptr) ==
         W4_OK);  // without residual and elements their outputs are not looked at
  EXPECT(w4_mx_rmsnorm(1, 4, 64, P(A), P(A), P(A), W4_BF16, 0.f, nullptr, P(A), P(A), P(A), nullptr) == W4_EINVAL);
  g_launches = 0;
  EXPECT(w4_mx_linear(1, 16, 64, P(A), P(A), P(A), P(A), 3, P(A), W4_BF16, nullptr) == W4_OK && g_launches == 1);
  EXPECT(g_last.m == 3 && g_last.tokens == 3 && g_last.n == 16 && g_last.k == 64 && g_last.y_bf16 == 1);
  EXPECT(g_last.offsets == nullptr && g_last.row_index == nullptr);
  EXPECT(w4_mx_linear(1, 16, 0, nullptr, nullptr, nullptr, nullptr, 3, P(A), W4_F32, nullptr) == W4_OK);
  EXPECT(g_zero == 48);
  g_blocks = INT64_C(1) << 31;
  EXPECT(w4_mx_linear(1, 16, 64, P(A), P(A), P(A), P(A), 3, P(A), W4_BF16, nullptr) == W4_ESHAPE);
  EXPECT(w4_mx_grouped_linear(1, 2, 16, 64, P(A), P(A), 3, P(A), P(A), 5, I(A), I(A), P(A), W4_F32, nullptr) ==
         W4_ESHAPE);
  g_blocks = 1;
  g_throw = true;
  EXPECT(w4_mx_linear(1, 16, 64, P(A), P(A), P(A), P(A), 3, P(A), W4_BF16, nullptr) == W4_EHIP);
  EXPECT(w4_mx_grouped_linear(1, 2, 16, 64, P(A), P(A), 3, P(A), P(A), 5, I(A), I(A), P(A), W4_F32, nullptr) ==
         W4_EHIP);
  g_throw = false;
  EXPECT(w4_mx_grouped_linear(0, 2, 16, 64, P(A), P(A), 3, P(A), P(A), 5, I(A), I(A), P(A), W4_F32, nullptr) ==
         W4_OK);
  EXPECT(g_last.m == 5 && g_last.tokens == 3 && g_last.experts == 2 && g_last.row_index == I(A));
  // nothing to multiply: zeros, whatever the other pointers are
  g_zero = -1;
  EXPECT(w4_mx_grouped_linear(0, 0, 16, 64, nullptr, nullptr, 5, nullptr, nullptr, 5, nullptr, nullptr, P(A), W4_F32,
                              nullptr) == W4_OK && g_zero == 80);
  g_zero = -1;
  EXPECT(w4_mx_grouped_linear(0, 2, 16, 64, P(A), P(A), 0, nullptr, nullptr, 5, I(A), I(A), P(A), W4_F32, nullptr) ==
         W4_OK && g_zero == 80);
  g_launches = 0;
  EXPECT(w4_mx_grouped_linear(0, 2, 16, 64, P(A), P(A), 4, P(A), P(A), 5, I(A), nullptr, P(A), W4_F32, nullptr) ==
         W4_ESHAPE);  // five rows of x are needed
  EXPECT(w4_mx_grouped_linear(0, 2, 0, 64, nullptr, nullptr, 4, nullptr, nullptr, 4, nullptr, nullptr, nullptr,
                              W4_F32, nullptr) == W4_OK && g_launches == 0);
  if (failures) {
    fprintf(stderr, "%d failures\n", failures);
    return 1;
  }
  printf("mx_api_check ok\n");
  return 0;
}
