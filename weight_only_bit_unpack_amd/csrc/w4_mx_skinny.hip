// MX products for few rows of x (gfx950): decode, and experts with few rows.
//
// Bound by the weights' bytes (17/32 byte each).  A wave loads a 256-k step of
// its weight rows as whole 128-byte lines and moves it through LDS into the
// operand order of v_mfma_scale_f32_16x16x128_f8f6f4: loaded straight in that
// order, each 16 lanes touch 16 lines and the address path holds the kernel at
// 2.6 TB/s (measured, 29 experts of 4096 x 2048).  The weight is operand A, up
// to 16 rows of x operand B, loaded and moved in the same way by every wave for
// its own steps, two steps ahead: no barrier until the end.  (x staged once per
// block instead: 8.0 against 5.2 us at 13 rows of 4095 x 5632 fp4.)  KS waves
// share the 16 R rows, wave i takes the steps i, i + KS, ..., and their sums
// are added in wave order through LDS.
//
// Measured (HIP graph replays, three weights in turn; calls in a row overlap
// their starts and ends and take 6.2, 4.9 and 31): one token, 4096 -> 11008, 6.8
// us (3.5 TB/s with the start and end, 1.4 us in a kernel that does nothing); 13
// rows of 4095 x 5632, fp4, 5.2 us; 96 rows over 29 experts of 4096 x 2048 32 us
// (4.0 TB/s).
#include "w4_launch.h"
#include "w4_mx_device.h"
#include "w4_mx_group.h"

namespace w4 {
namespace {

constexpr int kRows = 16;  // rows of x of a block

// Scale bytes of one 256-k step of 16 rows, eight a row.  DWORD (rows of whole
// dwords): lanes 0-31 take half a row each; otherwise a lane takes two bytes of
// row l / 4.
template <bool DWORD>
struct Scales {
  uint32_t v[DWORD ? 1 : 2];
  // offset(row, c): where the scale of block c of the row is
  template <typename L, typename F>
  __device__ __forceinline__ void load(int lane, uint32_t s, L&& ld, F&& offset) {
    if constexpr (DWORD) {
      v[0] = ld(offset((lane & 31) >> 1, 8 * s + 4 * (lane & 1)));
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u) v[u] = ld(offset(lane >> 2, 8 * s + 2 * (lane & 3) + u));
    }
  }
  // as [16][8] bytes
  __device__ __forceinline__ void put(uint8_t* p, int lane) const {
    if constexpr (DWORD) {
      reinterpret_cast<uint32_t*>(p)[lane & 31] = v[0];  // lanes 32-63 hold the same
    } else {
      reinterpret_cast<uint16_t*>(p)[lane] = (uint16_t)(v[0] | v[1] << 8);
    }
  }
};

// Raw loads of one 256-k step, as whole 128-byte lines: lane l takes 16 bytes
// l % 8 of weight rows l / 8 and 8 + l / 8 of each row tile, and of x 16 bytes
// of XI rows in the same way (fp8: 256 bytes a row, l % 16 of row l / 16).
template <int R, int XI, bool DWORD>
struct Step {
  u32x4 w[R][2];
  u32x4 x[XI];
  Scales<DWORD> ws[R], xs;
};

// XI: load instructions for x (fp8: 4 rows each, fp4: 8).
template <int AF, int XI, int R, int KS, int WN, bool DWORD, bool GROUPED>
__global__ __launch_bounds__(KS * WN * 64) void mx_skinny_kernel(MxProblem P, uint32_t tiles_n) {
  constexpr int NW = KS * WN;
  constexpr int ST = 2;  // steps in flight (3 and 4: slower or the same)
  constexpr int XU = AF == kMxFp8 ? 16 : 8;       // 16-byte units of a row of x in a step
  constexpr int UNITS = R * 136 + 16 * XU + 8;    // of a wave's LDS
  __shared__ u32x4 lds[NW * (UNITS > R * 64 ? UNITS : R * 64)];
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = wid % KS, wn = wid / KS;  // part of k, row tile
  const int r = lane & 15, g = lane >> 4;
  const uint32_t nt = blockIdx.x % tiles_n;
  GroupTile T{0, 0, (int32_t)P.m};
  if constexpr (GROUPED) {
    GroupScan<kRows> scan(P.offsets, P.experts, (int32_t)P.m);
    scan.read();
    T = scan.find(blockIdx.x / tiles_n);
    if (T.e < 0) return;
  }
  const bool none = GROUPED && T.e == P.experts;  // rows of no expert
  const int64_t N = P.n, K = P.k, n0 = ((int64_t)nt * WN + wn) * 16 * R;
  const int rows_n = (int)(N - n0 < 0 ? 0 : N - n0 < 16 * R ? N - n0 : 16 * R);
  const int rows_m = T.hi - T.lo < kRows ? T.hi - T.lo : kRows;
  const uint32_t half = (uint32_t)(K >> 1), blocks = (uint32_t)(K >> 5);

  f32x4 acc[R];
#pragma unroll
  for (int j = 0; j < R; ++j) acc[j] = (f32x4){0.f, 0.f, 0.f, 0.f};

  if (!none) {
    // this wave's shuffle area: R tiles of 16 rows x 128 bytes of the weight
    // and 16 rows of x (16-byte units XOR-swizzled by the row, so that both
    // sides are free of bank conflicts), then their scales
    u32x4* const lw = lds + wid * UNITS;
    u32x4* const lx = lw + R * 128;
    uint8_t* const lws = reinterpret_cast<uint8_t*>(lx + 16 * XU);
    uint8_t* const lxs = lws + R * 128;

    const int64_t wrow = (int64_t)T.e * N + n0;
    const __amdgpu_buffer_rsrc_t wr = mx_rsrc(P.w + wrow * half, (uint32_t)rows_n * half);
    const __amdgpu_buffer_rsrc_t sr = mx_rsrc(P.w_scales + wrow * blocks, (uint32_t)rows_n * blocks);
    const uint32_t lr = lane >> 3, lc = lane & 7;

    // rows of x past the last one repeat it and are never stored
    auto row_of_x = [&](int i) {
      const int64_t row = T.lo + (i < rows_m ? i : rows_m - 1);
      if (!(GROUPED && P.row_index)) return row;
      const int64_t src = P.row_index[row];
      return src < 0 || src >= P.tokens ? 0 : src;  // stored as zeros
    };
    const uint32_t x_bytes = AF == kMxFp8 ? (uint32_t)K : half;
    const uint8_t* xp[XI];
#pragma unroll
    for (int i = 0; i < XI; ++i) xp[i] = P.x + row_of_x(64 / XU * i + lane / XU) * x_bytes;
    const uint8_t* const xsp = P.x_scales + row_of_x(DWORD ? (lane & 31) >> 1 : lane >> 2) * blocks;

    // Past the end of k the weights read zeros (an offset past the resource)
    // with scale 0, and x its row's last bytes and scales: what those make of
    // the row (a NaN) it is already.
    auto load = [&](Step<R, XI, DWORD>& t, uint32_t s) {
      const bool in = 8 * s + lc < blocks;
#pragma unroll
      for (int j = 0; j < R; ++j) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
          t.w[j][u] = mx_load16(wr, in ? (16 * j + 8 * u + lr) * half + 16 * (8 * s + lc) : kMxOOB);
        t.ws[j].load(
            lane, s,
            [&](uint32_t o) {
              if constexpr (DWORD) return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(sr, o, 0, 0);
              return mx_load1(sr, o);
            },
            [&](int row, uint32_t c) { return c < blocks ? (16 * j + row) * blocks + c : kMxOOB; });
      }
      const uint32_t o = 16 * (XU * s + lane % XU), at = o < x_bytes ? o : x_bytes - 16;
#pragma unroll
      for (int i = 0; i < XI; ++i) t.x[i] = *reinterpret_cast<const u32x4*>(xp[i] + at);
      t.xs.load(
          lane, s,
          [&](uint32_t o) {
            if constexpr (DWORD) return *reinterpret_cast<const uint32_t*>(xsp + o);
            return (uint32_t)xsp[o];
          },
          [&](int, uint32_t c) { return c < blocks ? c : blocks - (DWORD ? 4 : 1); });
    };
    auto mma = [&](const Step<R, XI, DWORD>& t) {
      wave_lds_sync();
#pragma unroll
      for (int j = 0; j < R; ++j) {
#pragma unroll
        for (int u = 0; u < 2; ++u) lw[j * 128 + (8 * u + lr) * 8 + (lc ^ ((4 * u + (lr >> 1)) & 7))] = t.w[j][u];
        t.ws[j].put(lws + j * 128, lane);
      }
#pragma unroll
      for (int i = 0; i < XI; ++i) {
        const int row = 64 / XU * i + lane / XU;
        lx[row * XU + ((lane ^ (XU == 16 ? row : row >> 1)) & (XU - 1))] = t.x[i];
      }
      t.xs.put(lxs, lane);
      wave_lds_sync();
      const int xr = r < 64 / XU * XI ? r : 0;  // rows that were loaded
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        u32x4 x0, x1;
        if constexpr (AF == kMxFp8) {
          x0 = lx[xr * 16 + ((8 * u + g) ^ xr)];
          x1 = lx[xr * 16 + ((8 * u + 4 + g) ^ xr)];
        } else {
          x0 = x1 = lx[xr * 8 + ((4 * u + g) ^ (xr >> 1))];
        }
        const i32x8 b = mx_operand<AF>(x0, x1);
        const uint32_t sb = lxs[xr * 8 + 4 * u + g];
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const u32x4 a = lw[j * 128 + r * 8 + ((4 * u + g) ^ (r >> 1))];
          const uint32_t sa = lws[j * 128 + r * 8 + 4 * u + g];
          acc[j] = mx_mfma16<kMxFp4, AF>(mx_operand<kMxFp4>(a, a), b, acc[j], sa, sb);
        }
      }
    };

    const uint32_t steps = (blocks + 7) / 8;
    Step<R, XI, DWORD> t[ST];
#pragma unroll
    for (int i = 0; i < ST; ++i) load(t[i], wave + i * KS);
    for (uint32_t s = 0; s < steps; s += KS * ST) {
#pragma unroll
      for (int v = 0; v < ST; ++v) {
        mma(t[v]);  // a step past the end adds zeros
        load(t[v], s + wave + (v + ST) * KS);
      }
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
  bool dead = none;
  if (GROUPED && P.row_index && !none) {
    const int64_t src = P.row_index[T.lo + r];
    dead = src < 0 || src >= P.tokens;
  }
#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (dead) acc[j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    mx_store4(P.y, P.y_bf16, (T.lo + r) * N, n0 + 16 * j + 4 * g, N, acc[j]);
  }
}

// Shapes of a block: R row tiles of 16 a wave, KS waves along k, WN beside.
template <int R_, int KS_, int WN_>
struct Shape {
  static constexpr int R = R_, KS = KS_, WN = WN_, BN = 16 * R * WN;
};
using Split = Shape<1, 4, 1>;
using Wide = Shape<2, 2, 2>;
using Long = Shape<2, 1, 4>;

// The shape by the number of 16-row weight tiles of the launch.  While those
// are few, four waves share one, or the GPU would not fill; as they get many,
// a wave takes more rows and more of k, so that x, the offsets' walk and the
// joining of sums are paid less often.  Measured (us, MXFP8 x to bf16, Split /
// Wide / Long): 2048 x 2048 at m = 1 3.0 / 4.5 / 6.2; 8192 x 8192 at m = 16
// 11.2 / 14.1 / 24; 32768 x 4096 (2048 tiles) at m = 1 12.8 / 13.9 / 14.1 and
// at m = 16 19.2 / 15.1 / 15.5; 64 rows over 40 experts of 1024 x 4096 (2560
// tiles) 25.2 / 21.2 / 27.1; 96 rows over 29 experts of 4096 x 2048 (7424
// tiles) 47.5 / 33.7 / 32.2; 256 rows over 63 experts of 4096 x 1024 85 / 40 / 34.
// One row of x to four is loaded by one instruction a step instead of four, so
// the split shape pays up to twice the tiles there.
constexpr int kSplit = 0, kWide = 1, kLong = 2;
int shape_by(int64_t tiles, bool few) {
  if (tiles <= (few ? 2048 : 1024)) return kSplit;
  return tiles <= 8192 ? kWide : kLong;
}

template <typename F>
auto with_shape(int shape, F&& f) {
  if (shape == kSplit) return f(Split{});
  return shape == kWide ? f(Wide{}) : f(Long{});
}

// Tiles of up to 16 rows of y that the groups can make at most: with G groups
// that have rows (the rows of no expert among them) one each, and one more for
// every 16 rows beyond G.
int64_t row_tiles(const MxProblem& p) {
  if (!p.offsets) return 1;
  const int64_t G = p.m < p.experts + 1 ? p.m : p.experts + 1;
  return G + (p.m - G) / kRows;
}

// x's rows of a step in one load instruction
bool few_rows(int x_fmt, const MxProblem& p) { return p.m <= (x_fmt == kMxFp8 ? 4 : 8); }

}  // namespace

int mx_skinny_shape(int x_fmt, const MxProblem& p) {
  return shape_by(row_tiles(p) * ((p.n + 15) / 16), few_rows(x_fmt, p));
}

int64_t mx_skinny_blocks(int x_fmt, const MxProblem& p) {
  return with_shape(mx_skinny_shape(x_fmt, p), [&](auto S) {
    using T = decltype(S);
    const int64_t blocks = row_tiles(p) * ((p.n + T::BN - 1) / T::BN);
    return blocks * (T::KS * T::WN * 64) > kMaxLaunchThreads ? INT64_C(1) << 31 : blocks;
  });
}

hipError_t launch_mx_skinny(int x_fmt, const MxProblem& p, int shape, hipStream_t stream) {
  const bool few = few_rows(x_fmt, p), dword = p.k % 128 == 0;
  return with_shape(shape, [&](auto S) {
    using T = decltype(S);
    const uint32_t tiles_n = (uint32_t)((p.n + T::BN - 1) / T::BN);
    const dim3 grid(tiles_n * (uint32_t)row_tiles(p)), block(T::KS * T::WN * 64);
    auto go = [&](auto AF, auto XI, auto DW) {
      constexpr int af = decltype(AF)::value, xi = decltype(XI)::value;
      constexpr bool dw = decltype(DW)::value;
      if (p.offsets)
        mx_skinny_kernel<af, xi, T::R, T::KS, T::WN, dw, true><<<grid, block, 0, stream>>>(p, tiles_n);
      else
        mx_skinny_kernel<af, xi, T::R, T::KS, T::WN, dw, false><<<grid, block, 0, stream>>>(p, tiles_n);
      return hipGetLastError();
    };
    auto rows = [&](auto AF, auto DW) {
      if (few) return go(AF, std::integral_constant<int, 1>{}, DW);
      return go(AF, std::integral_constant<int, decltype(AF)::value == kMxFp8 ? 4 : 2>{}, DW);
    };
    auto format = [&](auto DW) {
      return x_fmt == kMxFp8 ? rows(std::integral_constant<int, kMxFp8>{}, DW)
                             : rows(std::integral_constant<int, kMxFp4>{}, DW);
    };
    return dword ? format(std::true_type{}) : format(std::false_type{});
  });
}

}  // namespace w4
