// Around the products of bf16 rows with MXFP4 weights (gfx950): the gated block's
// backward pass up to its product, rows padded to whole 16-byte units, and the
// workspace that holds them and the product's partial sums.
//
// Bound by HBM: each value is read or written once, eight a thread (16 bytes) where
// the rows are whole units.
#include <type_traits>

#include "w4_launch.h"
#include "w4_mx_act.h"
#include "w4_mx_device.h"

namespace w4 {
namespace {

// dgu = [dh u act'(g), dh act(g)] as bf16.  The products are fp32, rounded once.
template <int ACT>
__device__ __forceinline__ void gate_grad(float dh, float g, float u, float& dg, float& du) {
  float a, d;
  activate_with_slope<ACT>(g, a, d);
  dg = dh * u * d;
  du = dh * a;
}

// n and n / 8 units of a row; the threads take units in order.
template <int ACT>
__global__ __launch_bounds__(256) void gate_grad_kernel(MxGateGrad G, int64_t first, int64_t count) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= count) return;
  const int64_t units = G.n >> 3, row = (first + at) / units, c = (first + at) - row * units;
  const int64_t g0 = 2 * row * units + c;
  float dh[8], g[8], u[8];
  to_f32<kBf16>(load8<kBf16>(G.dh, row * units + c), dh);
  to_f32<kBf16>(load8<kBf16>(G.gu, g0), g);
  to_f32<kBf16>(load8<kBf16>(G.gu, g0 + units), u);
#pragma unroll
  for (int i = 0; i < 8; ++i) gate_grad<ACT>(dh[i], g[i], u[i], g[i], u[i]);
  store8<kBf16>(G.dgu, g0, from_f32<kBf16>(g));
  store8<kBf16>(G.dgu, g0 + units, from_f32<kBf16>(u));
}

// The same for any n, a value of each half a thread; `padded` (or nullptr) gets
// dgu with rows of `pitch` values, the ones behind the row's end zeros.
template <int ACT>
__global__ __launch_bounds__(256) void gate_grad_any_kernel(MxGateGrad G, int64_t first, int64_t count,
                                                            uint16_t* padded, int64_t pitch) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= count) return;
  const int64_t n = G.n, row = (first + at) / n, c = (first + at) - row * n;
  const int64_t g0 = 2 * row * n + c;
  float dg, du;
  gate_grad<ACT>(bf16_bits_to_f32(G.dh[row * n + c]), bf16_bits_to_f32(G.gu[g0]), bf16_bits_to_f32(G.gu[g0 + n]), dg,
                 du);
  const uint16_t a = (uint16_t)f32_to_bf16_bits(dg), b = (uint16_t)f32_to_bf16_bits(du);
  G.dgu[g0] = a;
  G.dgu[g0 + n] = b;
  if (padded) {
    uint16_t* const p = padded + row * pitch;
    p[c] = a;
    p[n + c] = b;
    if (c < pitch - 2 * n) p[2 * n + c] = 0;  // (at most 7)
  }
}

// rows of n values to rows of `pitch`, zeros behind; a value a thread
__global__ __launch_bounds__(256) void pad_kernel(const uint16_t* x, int64_t n, uint16_t* y, int64_t pitch,
                                                  int64_t first, int64_t count) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= count) return;
  const int64_t row = (first + at) / pitch, c = (first + at) - row * pitch;
  y[first + at] = c < n ? x[row * n + c] : (uint16_t)0;
}

// f(first, count, grid) over launches of at most 2^31 threads
template <typename F>
hipError_t in_launches(int64_t total, F&& f) {
  return in_parts(total, INT64_C(1) << 31, [&](int64_t first, int64_t count) {
    f(first, count, dim3((uint32_t)((count + 255) / 256)));
    return hipGetLastError();
  });
}

int64_t padded_pitch(int64_t n) { return (n + 7) / 8 * 8; }
// bytes of the padded rows in the workspace, whole 256
size_t padded_bytes(int64_t m, int64_t n) {
  return n % 8 ? ((size_t)m * padded_pitch(n) * 2 + 255) / 256 * 256 : 0;
}

// The product over rows padded to whole units, which lie in the workspace;
// write(rows, pitch) enqueues what fills them.
template <typename F>
hipError_t launch_padded(const MxBf16Problem& p, hipStream_t stream, F&& write) {
  struct Fill final : MxBf16Fill {
    F& write;
    explicit Fill(F& w) : write(w) {}
    hipError_t operator()(MxBf16Problem& on, char* ws) override {
      on.x = reinterpret_cast<const uint16_t*>(ws);
      return write(reinterpret_cast<uint16_t*>(ws), on.x_pitch);
    }
  } fill(write);
  MxBf16Problem on = p;
  on.x_pitch = padded_pitch(p.n);
  return launch_mx_bf16_with(on, padded_bytes(p.m, p.n), &fill, stream);
}

}  // namespace

hipError_t launch_mx_bf16(const MxBf16Problem& p, hipStream_t stream) {
  if (p.kind != kMxBackward || p.n % 8 == 0) return launch_mx_bf16_with(p, 0, nullptr, stream);
  return launch_padded(p, stream, [&](uint16_t* rows, int64_t pitch) {
    return in_launches(p.m * pitch, [&](int64_t first, int64_t count, dim3 grid) {
      pad_kernel<<<grid, dim3(256), 0, stream>>>(p.x, p.n, rows, pitch, first, count);
    });
  });
}

hipError_t launch_mx_gated_grad(const MxGateGrad& g, const MxBf16Problem& p, hipStream_t stream) {
  auto any = [&](uint16_t* rows, int64_t pitch) {
    return with_activation(g.act, [&](auto ACT) {
      return in_launches(g.m * g.n, [&](int64_t first, int64_t count, dim3 grid) {
        gate_grad_any_kernel<decltype(ACT)::value><<<grid, dim3(256), 0, stream>>>(g, first, count, rows, pitch);
      });
    });
  };
  if (p.n % 8 && p.k > 0) return launch_padded(p, stream, any);
  hipError_t e;
  if (g.n % 8 == 0)
    e = with_activation(g.act, [&](auto ACT) {
      return in_launches(g.m * (g.n / 8), [&](int64_t first, int64_t count, dim3 grid) {
        gate_grad_kernel<decltype(ACT)::value><<<grid, dim3(256), 0, stream>>>(g, first, count);
      });
    });
  else
    e = any(nullptr, 0);
  if (e != hipSuccess || p.k == 0) return e;
  return launch_mx_bf16_with(p, 0, nullptr, stream);
}

}  // namespace w4
