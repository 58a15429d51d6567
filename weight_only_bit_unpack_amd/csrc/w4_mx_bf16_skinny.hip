// Products of at most 16 bf16 rows with MXFP4 weights (gfx950): decode.  y = x W^T
// and the gated block act(x Wg^T) * (x Wu^T).
//
// Bound by the weights' bytes (17/32 byte each) and, on small weights, by the
// latencies of one pass over them.  A wave loads a 256-k step of 16 weight rows as
// whole 128-byte lines and moves it through LDS into the operand order of
// v_mfma_f32_16x16x32_bf16, where a lane's 16 bytes are one MX block, rebuilt to
// bf16 in the registers (v_cvt_scalef32_pk_bf16_fp4, exact but for values below
// 2^-126).  The rows of x are the other operand, loaded and moved in the same way
// by every wave for its own steps, two steps ahead: no barrier until the end.  KS
// waves share their weight rows, wave i takes the steps i, i + KS, ..., and their
// sums are added in wave order through LDS, in fp32.  Gated, a wave has as many
// gate as up rows, and a lane ends with both factors of an output.
//
// One row through 2048 x 2048 takes 3.2 us (1.4 of them a launch that does nothing),
// through 11008 x 4096 6.7 us (3.6 TB/s); at 16 rows the rows of x, twice the weights'
// bytes through LDS, count as well: gated 11008 x 4096 15.0 us (3.2 TB/s).
#include <type_traits>

#include "w4_launch.h"
#include "w4_mx_act.h"
#include "w4_mx_device.h"

namespace w4 {
namespace {

constexpr int kRows = 16;  // rows of x at most

// A step's loads: 16 bytes l % 8 of weight rows l / 8 and 8 + l / 8 of each row
// tile; the scale bytes of the two blocks, 2 (l / 16) and the next, of row l % 16
// that the lane multiplies with; of x 16 bytes l % 32 of rows 2 i + l / 32.
template <int R, int XI, bool EVEN>
struct Step {
  u32x4 w[R][2];
  uint32_t s[R][EVEN ? 1 : 2];
  u32x4 x[XI];
};

// R: row tiles of 16 a wave (gated: half of them gate rows, the others up rows);
// KS waves along k, WN beside; XI: load instructions for x, two rows each; EVEN: a
// row has an even number of blocks, so that two scale bytes are one aligned load.
template <bool GATE, int XI, int R, int KS, int WN, bool EVEN>
__global__ __launch_bounds__(KS * WN * 64) void mx_bf16_skinny_kernel(MxBf16Problem P) {
  using Loads = Step<R, XI, EVEN>;
  constexpr int ST = 2;                       // steps in flight
  constexpr int RO = GATE ? R / 2 : R;        // tiles of outputs
  constexpr int UNITS = R * 128 + XI * 64;    // of a wave's LDS
  constexpr int NW = KS * WN;
  __shared__ u32x4 lds[NW * (UNITS > R * 64 ? UNITS : R * 64)];
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = wid % KS, wn = wid / KS;  // part of k, row tile
  const int r = lane & 15, g = lane >> 4;
  const int64_t N = P.n, K = P.k, n0 = ((int64_t)blockIdx.x * WN + wn) * 16 * RO;
  const int rows_n = (int)(N - n0 < 0 ? 0 : N - n0 < 16 * RO ? N - n0 : 16 * RO);
  const int rows_m = (int)P.m;
  const uint32_t half = (uint32_t)(K >> 1), blocks = (uint32_t)(K >> 5);

  // this wave's shuffle area: R tiles of 16 rows x 128 bytes of the weight and
  // 2 XI rows x 512 bytes of x (16-byte units XOR-swizzled by the row, so that
  // both sides are free of bank conflicts)
  u32x4* const lw = lds + wid * UNITS;
  u32x4* const lx = lw + R * 128;

  // a tile's weights and scales, by halves where gated; rows past the last read zeros
  auto weights = [&](int hf) { return mx_rsrc(P.w + (hf * N + n0) * half, (uint32_t)rows_n * half); };
  auto scales = [&](int hf) { return mx_rsrc(P.w_scales + (hf * N + n0) * blocks, (uint32_t)rows_n * blocks); };
  const __amdgpu_buffer_rsrc_t wr[2] = {weights(0), weights(GATE ? 1 : 0)};
  const __amdgpu_buffer_rsrc_t sr[2] = {scales(0), scales(GATE ? 1 : 0)};
  const __amdgpu_buffer_rsrc_t xr = mx_rsrc(P.x, (uint32_t)rows_m * (uint32_t)(2 * K));
  const uint32_t lr = lane >> 3, lc = lane & 7;
  uint32_t xo[XI];  // rows of x past the last one repeat it and are never stored
#pragma unroll
  for (int i = 0; i < XI; ++i) {
    const int row = 2 * i + (lane >> 5);
    xo[i] = (uint32_t)(row < rows_m ? row : rows_m - 1) * (uint32_t)(2 * K);
  }

  f32x4 acc[R];
#pragma unroll
  for (int j = 0; j < R; ++j) acc[j] = (f32x4){0.f, 0.f, 0.f, 0.f};

  // Past the end of k all read zeros (an offset past the resource).
  auto load = [&](Loads& t, uint32_t s) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int hf = j / RO, row0 = 16 * (j % RO);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        t.w[j][u] = mx_load16(wr[hf], 8 * s + lc < blocks ? (row0 + 8 * u + lr) * half + 16 * (8 * s + lc) : kMxOOB);
      const uint32_t c = 8 * s + 2 * g, at = (row0 + r) * blocks + c;
      if constexpr (EVEN) {
        t.s[j][0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(sr[hf], c < blocks ? at : kMxOOB, 0, 0);
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) t.s[j][u] = mx_load1(sr[hf], c + u < blocks ? at + u : kMxOOB);
      }
    }
    const uint32_t at = 512 * s + 16 * (lane & 31);
#pragma unroll
    for (int i = 0; i < XI; ++i) t.x[i] = mx_load16(xr, at < 2 * (uint32_t)K ? xo[i] + at : kMxOOB);
  };
  auto mma = [&](const Loads& t) {
    wave_lds_sync();
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) lw[j * 128 + (8 * u + lr) * 8 + (lc ^ ((4 * u + (lr >> 1)) & 7))] = t.w[j][u];
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int row = 2 * i + (lane >> 5);
      lx[row * 32 + ((lane & 31) ^ row)] = t.x[i];
    }
    wave_lds_sync();
    const int xrow = r < 2 * XI ? r : 0;  // rows that were loaded
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      u32x4 b[4];  // rows of x, block 2 g + u
#pragma unroll
      for (int d = 0; d < 4; ++d) b[d] = lx[xrow * 32 + ((4 * (2 * g + u) + d) ^ xrow)];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const u32x4 a = lw[j * 128 + r * 8 + ((2 * g + u) ^ (r >> 1))];
        const uint32_t s = EVEN ? t.s[j][0] >> (8 * u) : t.s[j][EVEN ? 0 : u];
#pragma unroll
        for (int d = 0; d < 4; ++d) acc[j] = mfma16x16x32(mx_rebuild8(a[d], s), b[d], acc[j]);
      }
    }
  };

  const uint32_t steps = (blocks + 7) / 8;
  Loads t[ST];
#pragma unroll
  for (int i = 0; i < ST; ++i) load(t[i], wave + i * KS);
  for (uint32_t s = 0; s < steps; s += KS * ST) {
#pragma unroll
    for (int v = 0; v < ST; ++v) {
      mma(t[v]);  // a step past the end adds zeros
      load(t[v], s + wave + (v + ST) * KS);
    }
  }

  // the waves' sums in wave order
  if constexpr (KS > 1) {
    __syncthreads();
    f32x4* const part = reinterpret_cast<f32x4*>(lds);  // (the shuffle areas are done with)
#pragma unroll
    for (int j = 0; j < R; ++j) part[(wid * R + j) * 64 + lane] = acc[j];
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int i = 1; i < KS; ++i) acc[j] += part[((wid + i) * R + j) * 64 + lane];
  }
  // D[weight row 4 g + i][row of x r]: four consecutive outputs of row r
  if (r >= rows_m) return;
#pragma unroll
  for (int j = 0; j < RO; ++j) {
    const int64_t c = n0 + 16 * j + 4 * g;
    f32x4 v = acc[j];
    if constexpr (GATE) {
      const f32x4 u = acc[RO + j];
      if (P.gu) {
        mx_store4(P.gu, 1, r * 2 * N, c, N, v);
        mx_store4(P.gu, 1, r * 2 * N + N, c, N, u);
      }
      with_activation(P.act, [&](auto ACT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = activate<decltype(ACT)::value>(v[i]) * u[i];
      });
    }
    mx_store4(P.y, P.y_bf16, r * N, c, N, v);
  }
}

// Shapes of a block: R row tiles of 16 a wave (twice as many gated), KS waves along
// k, WN beside.
template <int R_, int KS_, int WN_>
struct Shape {
  static constexpr int R = R_, KS = KS_, WN = WN_;
};
template <bool GATE>
using Long = Shape<GATE ? 2 : 1, 8, 1>;
template <bool GATE>
using Split = Shape<GATE ? 2 : 1, 4, 1>;
using Wide = Shape<2, 2, 2>;
constexpr int kLong = 0, kSplit = 1, kWide = 2;

}  // namespace

// By the 16-row weight tiles of an output half and the steps of 256 along k.  Four
// waves share a tile; eight, while tiles are too few to fill the GPU and k is long
// (not for many rows of an ungated weight, whose LDS then keeps blocks off a CU); two,
// each with two tiles, where tiles are many or k is short and a step's rows of x cost
// as much as its weights, so that they, and the joining of sums, are paid less often.
// Measured (us, graph replays, Long / Split / Wide): m = 1, 1024 x 11008 5.2 / 7.0 / 15,
// 2816 x 2048 3.6 / 3.4 / 5.3, 11008 x 4096 7.0 / 6.7 / 9.1, 32768 x 4096 14.3 / 13.6 / 14.6;
// 5632 x 1024 4.3 / 3.6 / 4.1, 32768 x 1024 10.9 / 7.0 / 5.6; m = 8, 11008 x 1024 7.2 / 4.7 /
// 4.5, 32768 x 4096 18.9 / 16.7 / 15.6; m = 13, 4095 x 5632 7.3 / 6.5 / 14; m = 16, 11008 x
// 4096 13.6 / 11.1 / 11.5, 22016 x 2048 21 / 12.9 / 10.4, 32768 x 1024 23 / 12 / 7.2; gated m =
// 8, 1024 x 11008 10.9 / 12.5 / 21, 5632 x 1024 7.5 / 5.4 / 4.4, 11008 x 4096 13.6 / 13.3 / 14.7,
// 22016 x 2048 18.8 / 12.9 / 12.7.  Twice the tiles for a wave of Split or Long (gated two
// of each kind) are no faster than the best of these on any of them.
int mx_bf16_skinny_shape(const MxBf16Problem& p) {
  const int64_t tiles = (p.n + 15) / 16, steps = (p.k + 255) / 256;
  const bool gated = p.kind == kMxGated, shorter = steps <= 4;
  const bool wide = gated || p.m > 8 ? tiles >= (shorter ? 320 : 1024)
                                     : tiles >= (shorter ? 600 : 1536) && (shorter || p.m > 4);
  if (wide) return kWide;
  return tiles <= 256 && steps > 12 && (p.m <= 8 || gated) ? kLong : kSplit;
}

hipError_t launch_mx_bf16_skinny(const MxBf16Problem& p, int shape, hipStream_t stream) {
  auto go = [&](auto GATE, auto S, auto XI, auto EVEN) {
    using T = decltype(S);
    constexpr bool gate = decltype(GATE)::value;
    constexpr int cols = 16 * (gate ? T::R / 2 : T::R) * T::WN;
    const dim3 grid((uint32_t)((p.n + cols - 1) / cols)), block(T::KS * T::WN * 64);
    mx_bf16_skinny_kernel<gate, decltype(XI)::value, T::R, T::KS, T::WN, decltype(EVEN)::value>
        <<<grid, block, 0, stream>>>(p);
    return hipGetLastError();
  };
  auto scales = [&](auto GATE, auto S, auto XI) {
    return p.k % 64 == 0 ? go(GATE, S, XI, std::true_type{}) : go(GATE, S, XI, std::false_type{});
  };
  auto rows = [&](auto GATE, auto S) {
    if (p.m <= 2) return scales(GATE, S, std::integral_constant<int, 1>{});
    if (p.m <= 4) return scales(GATE, S, std::integral_constant<int, 2>{});
    if (p.m <= 8) return scales(GATE, S, std::integral_constant<int, 4>{});
    return scales(GATE, S, std::integral_constant<int, 8>{});
  };
  auto shapes = [&](auto GATE) {
    constexpr bool gate = decltype(GATE)::value;
    if (shape == kLong) return rows(GATE, Long<gate>{});
    return shape == kSplit ? rows(GATE, Split<gate>{}) : rows(GATE, Wide{});
  };
  return p.kind == kMxGated ? shapes(std::true_type{}) : shapes(std::false_type{});
}

}  // namespace w4
