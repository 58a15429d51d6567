// Checks that the C ABI's calls of the MX operators share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "w4.h"
#include "w4_launch.h"

namespace w4 {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline w4_status launched(hipError_t e) { return e == hipSuccess ? W4_OK : W4_EHIP; }

template <typename F>
w4_status guarded(F&& f) {
  return launched(caught(f));
}

inline w4_status check_y(const void* y, int32_t y_dtype) {
  if (!y) return W4_EINVAL;
  return aligned(y, y_dtype == W4_F32 ? 4 : 2) ? W4_OK : W4_EALIGN;
}

}  // namespace w4
