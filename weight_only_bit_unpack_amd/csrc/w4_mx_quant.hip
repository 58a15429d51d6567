// MX quantize, rebuild, and the RMS norm whose output is quantized (gfx950).
//
// All three stream: they are bound by HBM, and by the launch for a few rows.
// A lane holds eight consecutive values (16 bytes of bf16 / fp16), an aligned
// quad of lanes one block of 32, so the block's maximum is two DPP steps and
// every load and store instruction covers contiguous memory.
//
// Measured (kernel trace over three inputs in turn; a 1 GiB copy on such a card
// moves 5.2 TB/s): quantize of 11008 x 4096 bf16 to MXFP4 20.6 us (114 MB, 5.5
// TB/s), the rebuild to bf16 17.7 us; MXFP8 8192 x 4096 rebuilt 16.0 us (102 MB,
// 6.3 TB/s, part of it from the 256 MB cache); the norm with its residual, 8192 x
// 4096 bf16 to MXFP8, 49.9 us (236 MB, 4.7 TB/s), one row of 2048 2.8 us.
#include <type_traits>

#include "w4_launch.h"
#include "w4_mx_device.h"

namespace w4 {
namespace {

// ---------------------------------------------------------------- quantize
// b = clamp(floor(log2 max) - emax + 127, 0, 254); code = RNE of x * 2^(127 - b)
// onto the element's grid, saturating: all in exact fp32 (a power of two times a
// value of at most 24 bits), so the element's rounding is the only one.
// k is a multiple of 32, so rows add nothing: the array is rows * k / 32
// blocks in a line.  `total` counts groups of eight values.
template <int FMT, int DT>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void* __restrict__ x,
                                                          uint8_t* __restrict__ q,
                                                          uint8_t* __restrict__ scales,
                                                          int64_t total) {
  const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (g >= total) return;  // total is a multiple of 4: whole quads leave
  float v[8];
  to_f32<DT>(load8<DT>(x, g), v);
  uint32_t b, e[2];
  mx_quantize8<FMT>(v, b, e);
  mx_store8<FMT>(q, g, e);
  if ((threadIdx.x & 3) == 0) scales[g >> 2] = (uint8_t)b;
}

// ---------------------------------------------------------------- rebuild
// element * 2^(b - 127): at most 4 significant bits, exact in fp32 unless it
// overflows (to infinity), then the one rounding to the output type.
template <int FMT, int DT>
__global__ __launch_bounds__(256) void mx_dequant_kernel(const uint8_t* __restrict__ q,
                                                         const uint8_t* __restrict__ scales,
                                                         void* __restrict__ out, int64_t total) {
  const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (g >= total) return;
  const float s = mx_scale_value(scales[g >> 2]);
  float v[8];
  if constexpr (FMT == kMxFp4) {
    const uint32_t p = reinterpret_cast<const uint32_t*>(q)[g];
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, 1.0f, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, 1.0f, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, 1.0f, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, 1.0f, 3);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = c.x, v[5] = c.y, v[6] = d.x, v[7] = d.y;
  } else {
    const u32x2 p = reinterpret_cast<const u32x2*>(q)[g];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)p[i], false);
      const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)p[i], true);
      v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = b.x, v[4 * i + 3] = b.y;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= s;
  store8<DT>(out, g, from_f32<DT>(v));
}

// ---------------------------------------------------------------- RMS norm
// One row per block.  The squares add up in fp64, which holds those of every
// fp32 number without overflow or underflow, at no cost beside the row's
// memory.  The row's factor 1 / sqrt(mean + eps), which can lie outside
// fp32's range as well, is applied as a power of two, exactly, and a number in
// [1/2, 1) rounded to fp32; gamma comes after it, when the row is of size one.
// So a value takes two roundings more before the element's own.  The second pass reads
// the row back through L2 (8 KB at k = 4096, just written or read by this block),
// not from HBM: the kernel runs at the card's copy rate without holding the row
// in registers, and k has no bound.
template <int FMT, int DT>
__global__ __launch_bounds__(256) void mx_rmsnorm_kernel(const void* x, const void* residual,
                                                         const void* __restrict__ gamma,
                                                         void* residual_out, void* y, uint8_t* q,
                                                         uint8_t* scales, int64_t k, float eps) {
  const int64_t C = k >> 3;  // groups of eight in a row
  const int64_t r0 = (int64_t)blockIdx.x * C;
  const int tid = threadIdx.x;
  double t = 0.0;
  for (int64_t c = tid; c < C; c += 256) {
    float v[8];
    to_f32<DT>(load8<DT>(x, r0 + c), v);
    if (residual) {
      float w[8];
      to_f32<DT>(load8<DT>(residual, r0 + c), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += w[i];
      const Raw8<DT> h = from_f32<DT>(v);
      store8<DT>(residual_out, r0 + c, h);
      to_f32<DT>(h, v);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) t = __builtin_fma((double)v[i], (double)v[i], t);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) t += __shfl_xor(t, o);
  __shared__ double part[4];
  if ((tid & 63) == 0) part[tid >> 6] = t;
  __syncthreads();
  t = (part[0] + part[1]) + (part[2] + part[3]);
  // (0, infinity and NaN have exponent 0 here and stay what they are)
  const double factor = 1.0 / __builtin_sqrt(t / (double)k + (double)eps);
  const int e = __builtin_amdgcn_frexp_exp(factor);
  const float f = (float)__builtin_amdgcn_frexp_mant(factor);
  const void* h = residual ? residual_out : x;  // a thread reads back what it wrote itself
  for (int64_t c = tid; c < C; c += 256) {
    float v[8], w[8];
    to_f32<DT>(load8<DT>(h, r0 + c), v);
    to_f32<DT>(load8<DT>(gamma, c), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_ldexpf(v[i], e) * f * w[i];
    if (y) store8<DT>(y, r0 + c, from_f32<DT>(v));
    if (q) {
      uint32_t b, e[2];
      mx_quantize8<FMT>(v, b, e);
      mx_store8<FMT>(q, r0 + c, e);
      if ((tid & 3) == 0) scales[(r0 + c) >> 2] = (uint8_t)b;
    }
  }
}

template <typename F>
hipError_t by_format(int fmt, F&& f) {
  return fmt == kMxFp4 ? f(std::integral_constant<int, kMxFp4>{})
                       : f(std::integral_constant<int, kMxFp8>{});
}
template <typename F>
hipError_t by_dtype(int dt, F&& f) {
  if (dt == kF32) return f(std::integral_constant<int, kF32>{});
  return dt == kBf16 ? f(std::integral_constant<int, kBf16>{})
                     : f(std::integral_constant<int, kF16>{});
}

// A launch holds fewer than 2^32 threads: arrays of more than 2^31 groups of
// eight values, and norms of more than 2^23 rows, take several, each on its part.
constexpr int64_t kMaxGroups = INT64_C(1) << 31;
constexpr int64_t kMaxRows = INT64_C(1) << 23;
static_assert(kMaxGroups <= kMaxLaunchThreads && kMaxRows * 256 <= kMaxLaunchThreads);

constexpr int64_t mx_bytes(int fmt, int64_t values) { return fmt == kMxFp4 ? values / 2 : values; }
constexpr int64_t dtype_bytes(int dtype, int64_t values) { return values * (dtype == kF32 ? 4 : 2); }

template <typename P>
P* ahead(P* p, int64_t bytes) {
  using Byte = std::conditional_t<std::is_const_v<P>, const uint8_t, uint8_t>;
  return p ? reinterpret_cast<P*>(reinterpret_cast<Byte*>(p) + bytes) : p;
}

}  // namespace

hipError_t launch_mx_quantize(int fmt, int64_t rows, int64_t k, const void* x, int dtype, uint8_t* q,
                              uint8_t* scales, hipStream_t stream) {
  return in_parts(rows * (k / 8), kMaxGroups, [&](int64_t at, int64_t n) {
    const dim3 grid((uint32_t)((n + 255) / 256));
    const void* const xp = ahead(x, dtype_bytes(dtype, 8 * at));
    uint8_t* const qp = ahead(q, mx_bytes(fmt, 8 * at));
    uint8_t* const sp = scales + at / 4;
    return by_format(fmt, [&](auto F) {
      return by_dtype(dtype, [&](auto D) {
        mx_quantize_kernel<decltype(F)::value, decltype(D)::value><<<grid, dim3(256), 0, stream>>>(xp, qp, sp, n);
        return hipGetLastError();
      });
    });
  });
}

hipError_t launch_mx_dequant(int fmt, int64_t rows, int64_t k, const uint8_t* q, const uint8_t* scales,
                             void* out, int dtype, hipStream_t stream) {
  return in_parts(rows * (k / 8), kMaxGroups, [&](int64_t at, int64_t n) {
    const dim3 grid((uint32_t)((n + 255) / 256));
    const uint8_t* const qp = ahead(q, mx_bytes(fmt, 8 * at));
    const uint8_t* const sp = scales + at / 4;
    void* const op = ahead(out, dtype_bytes(dtype, 8 * at));
    return by_format(fmt, [&](auto F) {
      auto go = [&](auto D) {
        mx_dequant_kernel<decltype(F)::value, decltype(D)::value><<<grid, dim3(256), 0, stream>>>(qp, sp, op, n);
        return hipGetLastError();
      };
      return dtype == kF32 ? go(std::integral_constant<int, kF32>{}) : go(std::integral_constant<int, kBf16>{});
    });
  });
}

hipError_t launch_mx_rmsnorm(int fmt, int64_t rows, int64_t k, const void* x, const void* residual,
                             const void* gamma, int dtype, float eps, void* residual_out, void* y,
                             uint8_t* q, uint8_t* scales, hipStream_t stream) {
  return in_parts(rows, kMaxRows, [&](int64_t at, int64_t n) {
    const int64_t b = dtype_bytes(dtype, at * k);
    return by_format(fmt, [&](auto F) {
      return by_dtype(dtype, [&](auto D) {
        mx_rmsnorm_kernel<decltype(F)::value, decltype(D)::value><<<dim3((uint32_t)n), dim3(256), 0, stream>>>(
            ahead(x, b), ahead(residual, b), gamma, ahead(residual_out, b), ahead(y, b),
            ahead(q, mx_bytes(fmt, at * k)), ahead(scales, at * (k / 32)), k, eps);
        return hipGetLastError();
      });
    });
  });
}

}  // namespace w4
