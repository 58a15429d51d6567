// Activations of the gated feed-forward block and their derivatives, in fp32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace w4 {

// Codes, as w4_activation.
constexpr int kSilu = 0, kGelu = 1, kGeluTanh = 2;

// e^a, a <= 0, to a few 2^-24 of itself: 2^t with t = a log2(e) kept as two floats (the
// rounding of t alone would cost |t| 2^-24 of the result); below 2^-126, 0.
__device__ __forceinline__ float exp_down(float a) {
  constexpr float kL = 1.44269504e+00f, kLlo = 1.92596303e-08f;  // log2(e), and what its rounding leaves
  const float t = a * kL;
  const float lo = __builtin_fmaf(a, kLlo, __builtin_fmaf(a, kL, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, lo * 6.93147182e-01f, e);  // 2^lo = 1 + lo ln 2, lo < 2^-16
}

// 1 / (1 + e^-z), to a few 2^-24 of itself wherever it is a normal number: e^-|z| <= 1
// neither cancels nor overflows.  Beyond |z| = 128 it is taken as at 128, where
// e^-|z| is 0.  A NaN's value is any: every caller multiplies by what made it.
__device__ __forceinline__ float sigmoid(float z) {
  const float e = exp_down(-fminf(fabsf(z), 128.0f));
  return __builtin_amdgcn_rcpf(1.0f + e) * (z >= 0.0f ? 1.0f : e);
}
// It and 1 / (1 + e^z), which is 1 less it, without the cancellation.
__device__ __forceinline__ void sigmoid_pair(float z, float& p, float& q) {
  const float e = exp_down(-fminf(fabsf(z), 128.0f));
  const float r = __builtin_amdgcn_rcpf(1.0f + e), s = e * r;
  p = z >= 0.0f ? r : s;
  q = z >= 0.0f ? s : r;
}

constexpr float kTanhA = 7.97884583e-01f;  // sqrt(2 / pi)
constexpr float kTanhB = 4.47149985e-02f;  // 0.044715

// g within +-16, where e^-2|y| is 0 in fp32 already: g^3 would overflow.
__device__ __forceinline__ float tanh_inside(float g) { return __builtin_amdgcn_fmed3f(g, -16.0f, 16.0f); }
__device__ __forceinline__ float tanh_argument(float g) {  // 2y
  const float c = tanh_inside(g);
  return 2.0f * kTanhA * __builtin_fmaf(kTanhB * c * c, c, c);
}

// act(g), a NaN for a NaN; an infinite g gives what the formula does (infinity,
// or 0 * infinity below):
//   silu       g / (1 + e^-g)
//   gelu       g Phi(g), Phi(g) = erfc(-g / sqrt 2) / 2
//   gelu_tanh  g (1 + tanh y) / 2 = g / (1 + e^-2y), y = sqrt(2/pi) (g + 0.044715 g^3)
template <int ACT>
__device__ __forceinline__ float activate(float g) {
  if constexpr (ACT == kSilu) return g * sigmoid(g);
  if constexpr (ACT == kGelu) return g * (0.5f * erfcf(g * -7.07106769e-01f));
  return g * sigmoid(tanh_argument(g));
}

// act(g) and act'(g) (a NaN where g is no number or infinite).
template <int ACT>
__device__ __forceinline__ void activate_with_slope(float g, float& a, float& d) {
  float p, q;
  if constexpr (ACT == kSilu) {
    sigmoid_pair(g, p, q);
    a = g * p;
    d = p * __builtin_fmaf(g, q, 1.0f);
  } else if constexpr (ACT == kGelu) {
    const float phi = 0.5f * erfcf(g * -7.07106769e-01f);
    a = g * phi;
    d = __builtin_fmaf(g, 3.98942280e-01f * expf(-0.5f * g * g), phi);  // (1 / sqrt(2 pi)) e^(-g^2/2)
  } else {
    sigmoid_pair(tanh_argument(g), p, q);
    a = g * p;
    const float c = tanh_inside(g);
    const float slope = 2.0f * kTanhA * __builtin_fmaf(3.0f * kTanhB * c, c, 1.0f);  // of 2y
    d = __builtin_fmaf(g * p, q * slope, p);
  }
}

// f(integral_constant<ACT>)
template <typename F>
__host__ __device__ __forceinline__ auto with_activation(int act, F&& f) {
  if (act == kSilu) return f(std::integral_constant<int, kSilu>{});
  if (act == kGelu) return f(std::integral_constant<int, kGelu>{});
  return f(std::integral_constant<int, kGeluTanh>{});
}

}  // namespace w4
