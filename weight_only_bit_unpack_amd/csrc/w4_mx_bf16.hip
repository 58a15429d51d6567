// Around the products of bf16 rows with MXFP4 weights (gfx950): the gated block's
// backward pass up to its product, rows padded to whole 16-byte units, and the
// workspace that holds them and the product's partial sums.
//
// Bound by HBM: each value is read or written once, eight a thread (4096 x 11008 69 us, 6.5
// TB/s; rows that are no whole units, 333 x 2730 with the padded copy, 5 to 6 us).
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

// Blocks of 256 threads take a row's values 2048 at a time (`chunks` blocks a row, from
// row `first` on), eight a thread: as one unit of 16 bytes where the rows are whole units, ...
template <int ACT>
__global__ __launch_bounds__(256) void gate_grad_kernel(MxGateGrad G, uint32_t chunks, int64_t first) {
  const int64_t row = first + blockIdx.x / chunks, units = G.n >> 3;
  const int64_t c = (int64_t)(blockIdx.x % chunks) * 256 + threadIdx.x;
  if (c >= units) return;
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

// ... and otherwise one (n odd) or two at a time, 256 threads' apart.  `padded` (or
// nullptr) gets dgu with rows of `pitch` values, the ones behind the row's end zeros.
template <int ACT, typename V>  // V: uint16_t, or uint32_t for two values
__global__ __launch_bounds__(256) void gate_grad_any_kernel(MxGateGrad G, uint32_t chunks, int64_t first,
                                                            uint16_t* padded, int64_t pitch) {
  constexpr int W = sizeof(V) / 2, E = 8 / W;
  const int64_t row = first + blockIdx.x / chunks, n = G.n / W;
  const int64_t c0 = (int64_t)(blockIdx.x % chunks) * (2048 / W) + threadIdx.x;
  const V* const dh = reinterpret_cast<const V*>(G.dh + row * G.n);
  const V* const gu = reinterpret_cast<const V*>(G.gu + 2 * row * G.n);
  V* const dgu = reinterpret_cast<V*>(G.dgu + 2 * row * G.n);
  V* const pad = reinterpret_cast<V*>(padded + row * pitch);
  V x[E], g[E], u[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int64_t c = c0 + 256 * i < n ? c0 + 256 * i : n - 1;
    x[i] = dh[c];
    g[i] = gu[c];
    u[i] = gu[n + c];
  }
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int64_t c = c0 + 256 * i;
    if (padded && c < pitch / W - 2 * n) pad[2 * n + c] = 0;  // (at most 7 values, maybe more than n)
    if (c >= n) continue;
    V a = 0, b = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      auto value = [&](uint32_t v) { return bf16_bits_to_f32(v >> (16 * w) & 0xFFFFu); };
      float dg, du;
      gate_grad<ACT>(value(x[i]), value(g[i]), value(u[i]), dg, du);
      a |= (V)(f32_to_bf16_bits(dg) << (16 * w));
      b |= (V)(f32_to_bf16_bits(du) << (16 * w));
    }
    dgu[c] = a;
    dgu[n + c] = b;
    if (padded) {
      pad[c] = a;
      pad[n + c] = b;
    }
  }
}

// rows of n values to rows of `pitch`, zeros behind
__global__ __launch_bounds__(256) void pad_kernel(const uint16_t* x, int64_t n, uint16_t* y, int64_t pitch,
                                                  uint32_t chunks, int64_t first) {
  const int64_t row = first + blockIdx.x / chunks, c0 = (int64_t)(blockIdx.x % chunks) * 2048 + threadIdx.x;
  uint16_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t c = c0 + 256 * i;
    v[i] = c < n ? x[row * n + c] : (uint16_t)0;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c0 + 256 * i < pitch) y[row * pitch + c0 + 256 * i] = v[i];
}

// f(chunks, first row, grid) over launches of at most 2^23 blocks (or one row): rows of
// n values in chunks of 2048
template <typename F>
hipError_t over_rows(int64_t rows, int64_t n, F&& f) {
  const int64_t chunks = (n + 2047) / 2048, most = (INT64_C(1) << 23) / chunks;
  return in_parts(rows, most > 0 ? most : 1, [&](int64_t first, int64_t count) {
    f((uint32_t)chunks, first, dim3((uint32_t)(count * chunks)));
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
    return over_rows(p.m, pitch, [&](uint32_t chunks, int64_t first, dim3 grid) {
      pad_kernel<<<grid, dim3(256), 0, stream>>>(p.x, p.n, rows, pitch, chunks, first);
    });
  });
}

hipError_t launch_mx_gated_grad(const MxGateGrad& g, const MxBf16Problem& p, hipStream_t stream) {
  auto any = [&](uint16_t* rows, int64_t pitch) {
    return with_activation(g.act, [&](auto ACT) {
      return over_rows(g.m, g.n, [&](uint32_t chunks, int64_t first, dim3 grid) {
        if (g.n % 2 == 0)
          gate_grad_any_kernel<decltype(ACT)::value, uint32_t><<<grid, dim3(256), 0, stream>>>(g, chunks, first, rows, pitch);
        else
          gate_grad_any_kernel<decltype(ACT)::value, uint16_t><<<grid, dim3(256), 0, stream>>>(g, chunks, first, rows, pitch);
      });
    });
  };
  if (p.n % 8 && p.k > 0) return launch_padded(p, stream, any);
  hipError_t e;
  if (g.n % 8 == 0)
    e = with_activation(g.act, [&](auto ACT) {
      return over_rows(g.m, g.n, [&](uint32_t chunks, int64_t first, dim3 grid) {
        gate_grad_kernel<decltype(ACT)::value><<<grid, dim3(256), 0, stream>>>(g, chunks, first);
      });
    });
  else
    e = any(nullptr, 0);
  if (e != hipSuccess || p.k == 0) return e;
  return launch_mx_bf16_with(p, 0, nullptr, stream);
}

}  // namespace w4
