// MX products (gfx950): y = x w^T with both operands in microscaled form, for
// one weight and for many weights whose rows of x are grouped by expert.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes the stored elements and scale bytes
// as they are: nothing is rebuilt, and the sums are the matrix core's fp32.
#include "w4_launch.h"
#include "w4_mx_device.h"

namespace w4 {
namespace {

// One 32 x 32 tile of y per wave, operands read from global memory in matrix
// core order.  Block 256: 2 x 2 tiles.
//
// Grouped: block row t is the t-th 64-row tile when each expert's rows (and at
// last the rows of no expert) are cut into tiles of 64; every block finds its
// expert by walking the offsets.  An offset is taken no lower than the one
// before it and no higher than the number of rows, so that no offsets make
// the kernel leave its buffers.
template <int AF, bool GROUPED>
__global__ __launch_bounds__(256) void mx_linear_kernel(MxProblem P) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 31, g = lane >> 5;
  const int64_t tiles_n = (P.n + 63) / 64;
  const int64_t nt = blockIdx.x % tiles_n;
  int64_t mt = blockIdx.x / tiles_n;
  int64_t lo = 0, hi = P.m;
  int e = 0;
  if constexpr (GROUPED) {
    int64_t at = 0;
    for (; e <= P.experts; ++e) {
      int64_t end = e < P.experts ? (int64_t)P.offsets[e + 1] : P.m;
      end = end < at ? at : end > P.m ? P.m : end;
      const int64_t tiles = (end - at + 63) / 64;
      lo = at, hi = end, at = end;
      if (mt < tiles) break;
      mt -= tiles;
    }
    if (e > P.experts) return;
  }
  const int64_t m0 = lo + mt * 64 + 32 * (wave >> 1), n0 = nt * 64 + 32 * (wave & 1);
  const int64_t K = P.k, kb = K >> 5;
  const bool none = GROUPED && e == P.experts;  // rows of no expert: zeros
  f32x16 acc;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  const int64_t row = m0 + r < hi ? m0 + r : hi - 1, col = n0 + r < P.n ? n0 + r : P.n - 1;
  int64_t src = row;
  if (!none) {
    if (GROUPED && P.row_index) {
      src = P.row_index[row];
      if (src < 0 || src >= P.tokens) src = 0;  // stored as zeros below
    }
    constexpr int kStep = AF == kMxFp8 ? 64 : 32;  // bytes of a 64-k step of x
    const uint8_t* xr = P.x + src * (AF == kMxFp8 ? K : K / 2);
    const uint8_t* wr = P.w + ((int64_t)e * P.n + col) * (K / 2);
    const uint8_t* xs = P.x_scales + src * kb;
    const uint8_t* ws = P.w_scales + ((int64_t)e * P.n + col) * kb;
    for (int64_t t = 0; t < (K + 63) / 64; ++t) {
      const bool two = t * 64 + 32 < K;   // the step has its second block of 32
      const bool mine = g == 0 || two;    // block g of the step exists
      i32x8 a, b;
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = 0, b[i] = 0;
      if (mine) {
        const i32x4 v = *reinterpret_cast<const i32x4*>(wr + t * 32 + 16 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = v[i];
      }
      if constexpr (AF == kMxFp8) {
        const i32x4 v = *reinterpret_cast<const i32x4*>(xr + t * kStep + 16 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = v[i];
        if (two) {
          const i32x4 u = *reinterpret_cast<const i32x4*>(xr + t * kStep + 32 + 16 * g);
#pragma unroll
          for (int i = 0; i < 4; ++i) a[4 + i] = u[i];
        }
      } else if (mine) {
        const i32x4 v = *reinterpret_cast<const i32x4*>(xr + t * kStep + 16 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = v[i];
      }
      const uint32_t sa = mine ? xs[2 * t + g] : 0u, sb = mine ? ws[2 * t + g] : 0u;
      acc = mx_mfma32<AF, 0, 0>(a, b, acc, sa, sb);
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t yr = m0 + 8 * (i >> 2) + 4 * g + (i & 3);
    if (yr < hi && n0 + r < P.n) {
      float v = acc[i];
      if (GROUPED && !none && P.row_index) {
        const int64_t s = P.row_index[yr];
        if (s < 0 || s >= P.tokens) v = 0.f;
      }
      if (P.y_bf16)
        reinterpret_cast<uint16_t*>(P.y)[yr * P.n + n0 + r] = (uint16_t)f32_to_bf16_bits(v);
      else
        reinterpret_cast<float*>(P.y)[yr * P.n + n0 + r] = v;
    }
  }
}

}  // namespace

// Products with few rows a weight: at most one tile of 16, or on average.
static bool skinny(const MxProblem& p) {
  return p.m <= 16 || (p.offsets && p.m <= 16 * (int64_t)p.experts);
}

int64_t mx_linear_blocks(int x_fmt, const MxProblem& p) {
  if (skinny(p)) return mx_skinny_blocks(x_fmt, p);
  const int64_t tiles_m = (p.m + 63) / 64 + (p.offsets ? p.experts + 1 : 0);
  return tiles_m * ((p.n + 63) / 64);
}

hipError_t launch_mx_linear(int x_fmt, const MxProblem& p, hipStream_t stream) {
  if (skinny(p)) return launch_mx_skinny(x_fmt, p, stream);
  const dim3 grid((uint32_t)mx_linear_blocks(x_fmt, p));
  if (p.offsets) {
    if (x_fmt == kMxFp8)
      mx_linear_kernel<kMxFp8, true><<<grid, dim3(256), 0, stream>>>(p);
    else
      mx_linear_kernel<kMxFp4, true><<<grid, dim3(256), 0, stream>>>(p);
  } else {
    if (x_fmt == kMxFp8)
      mx_linear_kernel<kMxFp8, false><<<grid, dim3(256), 0, stream>>>(p);
    else
      mx_linear_kernel<kMxFp4, false><<<grid, dim3(256), 0, stream>>>(p);
  }
  return hipGetLastError();
}

}  // namespace w4
