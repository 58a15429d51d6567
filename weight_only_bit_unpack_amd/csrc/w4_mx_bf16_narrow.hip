// Gradients of few bf16 rows through MXFP4 weights (gfx950): dx = dy W.
//
// Bound by latencies: such a product has few tiles, and a wave's own chain of loads,
// rebuilding and matrix instructions (165 instructions a step, which one wave issues
// every eight cycles or so) is what takes the time.  So a wave works alone on 32 rows by
// 64 columns and every fourth step of 64 terms, with the loads of two steps in its
// registers (three and four: the same or slower) and no barrier until the sums are
// joined; four waves make a block (eight: the same), and where the tiles are still few,
// blocks share a tile's terms.  24 rows of a weight of 11264 x 2048 take 12.0 us in eight
// parts (37.6 in one, 20.2 on 64 x 128 tiles), 64 of 4096 x 4096 12.1 in two (15.6).
//
// The weight's 4 bits lie along the columns, the sum goes over its rows: the 64 rows of
// a step are rebuilt to bf16 by the lanes that loaded them into 8 KB of the wave's own
// LDS, and ds_read_b64_tr_b16 gives a lane four rows of one column.  A wave's LDS
// accesses are carried out in order, so nothing waits in between; a step's rows are
// rebuilt behind the last step's reads, since they share the area.
#include "w4_launch.h"
#include "w4_mx_device.h"
#include "w4_mx_parts.h"

namespace w4 {
namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr int kRows = 32, kCols = 64;  // a tile
constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kAhead = 2;  // steps in flight

struct NarrowArgs {
  uint32_t tiles_m, tiles_n, splits;  // splits: blocks that share a tile
  uint64_t* partial;                  // [tile][split][kRows kCols / 2], pairs of fp32
  uint32_t* counted;                  // [tile], zeros between launches
};

// 16-byte unit c of a row of 128 bytes of x lies at unit c ^ swizzle_x(row) in LDS,
// of rebuilt weights at c ^ swizzle_r(row): neither the writes nor the reads (16
// rows; four rows of four units) meet on a bank.
__device__ __forceinline__ int swizzle_x(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int swizzle_r(int row) {
  const int n0 = row & 1, n1 = (row >> 1) & 1;
  return n1 << 2 | n1 << 1 | n0;
}

__global__ __launch_bounds__(kThreads) void mx_bf16_narrow_kernel(MxBf16Problem P, NarrowArgs G) {
  constexpr int UNITS = 768;  // of a wave's LDS: 32 rows of x, 64 of rebuilt weights
  __shared__ u32x4 lds[kWaves * UNITS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;

  // Blocks are dealt to the 8 XCDs round robin; each XCD takes a contiguous range of
  // the parts, whose rows of x and w meet in its L2.  (The grid is a multiple of 8.)
  const uint32_t total = G.tiles_m * G.tiles_n * G.splits, range = (total + 7) / 8;
  const uint32_t L = blockIdx.x % 8 * range + blockIdx.x / 8;
  if (blockIdx.x / 8 >= range || L >= total) return;
  const uint32_t split = L % G.splits, tile = L / G.splits, mt = tile % G.tiles_m, nt = tile / G.tiles_m;

  const int64_t m0 = (int64_t)mt * kRows, k0 = (int64_t)nt * kCols;
  const int rows_m = (int)(P.m - m0 < kRows ? P.m - m0 : kRows);
  const int cols_k = (int)(P.k - k0 < kCols ? P.k - k0 : kCols);
  const uint32_t half = (uint32_t)(P.k >> 1), blocks = (uint32_t)(P.k >> 5);
  const uint32_t terms = (uint32_t)P.n, steps = (terms + 63) / 64;
  const uint32_t t0 = (uint32_t)((uint64_t)split * steps / G.splits);
  const uint32_t t1 = (uint32_t)((uint64_t)(split + 1) * steps / G.splits);
  const uint32_t end = split + 1 == G.splits ? terms : 64 * t1;  // of the part's terms

  u32x4* const lx = lds + wave * UNITS;
  u32x4* const lr = lx + 256;

  // ---- a step's loads.  x (dy): unit lane % 8 of rows 8 i + lane / 8.  Weights: unit
  // lane % 2 of rows 32 i + lane / 2 in the tile's columns, and its scale.  Past the
  // rows, the columns and the part's terms all read zeros.
  struct Loads {
    u32x4 x[4], w[2];
    uint32_t s[2];
  };
  const uint32_t pitch = (uint32_t)(2 * P.x_pitch), unit = (uint32_t)(k0 >> 5) + (lane & 1);
  const __amdgpu_buffer_rsrc_t xr =
      mx_rsrc(uniform(reinterpret_cast<const uint8_t*>(P.x + m0 * P.x_pitch)), (uint32_t)rows_m * pitch);
  auto load = [&](Loads& v, uint32_t t) {
    const uint32_t c = 64 * t + 8 * (lane & 7);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v.x[i] = mx_load16(xr, t < t1 && c < end ? (uint32_t)(8 * i + (lane >> 3)) * pitch + 2 * c : kMxOOB);
    const int64_t row0 = 64 * (int64_t)t;
    const uint32_t rows = t >= t1 ? 0 : end - 64 * t < 64 ? end - 64 * t : 64;
    const __amdgpu_buffer_rsrc_t wr = mx_rsrc(uniform(P.w + row0 * half), rows * half);
    const __amdgpu_buffer_rsrc_t sr = mx_rsrc(uniform(P.w_scales + row0 * blocks), rows * blocks);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t row = 32 * i + (lane >> 1);
      v.w[i] = mx_load16(wr, unit < blocks ? row * half + 16 * unit : kMxOOB);
      v.s[i] = mx_load1(sr, unit < blocks ? row * blocks + unit : kMxOOB);
    }
  };

  f32x16 acc[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[j][q] = 0.f;
  auto multiply = [&](const Loads& v) {
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 8 * i + (lane >> 3);
      lx[8 * row + ((lane & 7) ^ swizzle_x(row))] = v.x[i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 32 * i + (lane >> 1);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        lr[8 * row + ((4 * (lane & 1) + e) ^ swizzle_r(row))] = mx_rebuild8(v.w[i][e], v.s[i]);
    }
    wave_lds_sync();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const u32x4 a = lx[8 * r + ((4 * h + q) ^ swizzle_x(r))];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        u32x4 b;
        // sixteen lanes' addresses are four rows of four eight-byte pieces
        const int p = lane & 15, from = 4 * j + 2 * ((lane >> 4) & 1) + ((p & 3) >> 1);
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const int row = 32 * h + 8 * q + 4 * d + (p >> 2);
          const u32x2* const at = reinterpret_cast<const u32x2*>(lr + 8 * row + (from ^ swizzle_r(row))) + (p & 1);
          const u32x2 y = __builtin_bit_cast(
              u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)at));
          b[2 * d] = y.x;
          b[2 * d + 1] = y.y;
        }
        acc[j] = mfma32x32x16(a, b, acc[j]);
      }
    }
  };
  Loads v[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(v[i], t0 + wave + i * kWaves);
  for (uint32_t t = t0 + wave; t < t1; t += kAhead * kWaves) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      multiply(v[i]);  // a step past the end adds zeros
      load(v[i], t + (i + kAhead) * kWaves);
    }
  }

  // ---- the waves' sums, in the order of the waves: wave w takes rows 8 w + 4 h + e,
  // e = 0 .. 3, of both tiles (D[row of x][column]: register 4 w + e)
  f32x4 sum[2];
  {
    f32x4* const part = reinterpret_cast<f32x4*>(lds);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int w = 0; w < 4; ++w)
        part[(wave * 8 + 2 * w + j) * 64 + lane] =
            (f32x4){acc[j][4 * w], acc[j][4 * w + 1], acc[j][4 * w + 2], acc[j][4 * w + 3]};
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const f32x4* const from = part + (2 * wave + j) * 64 + lane;
      sum[j] = from[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) sum[j] += from[w * 512];
    }
  }
  if (G.splits > 1) {
    uint64_t* const parts = G.partial + (uint64_t)tile * G.splits * (4 * kThreads) + threadIdx.x;
    put_part<4>(parts + (uint64_t)split * (4 * kThreads), kThreads, [&](int i) {
      const f32x4& s = sum[i / 2];
      return (f32x2){s[i % 2 * 2], s[i % 2 * 2 + 1]};
    });
    if (!last_part(G.counted + tile, G.splits, reinterpret_cast<uint32_t*>(lds))) return;
    add_parts<4, 16>(parts, 4 * kThreads, kThreads, G.splits, [&](int i, const f32x2& x) {
      sum[i / 2][i % 2 * 2] = x.x;
      sum[i / 2][i % 2 * 2 + 1] = x.y;
    });
  }
  // ---- outputs: columns 32 j + r
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = 32 * j + r;
    if (c >= cols_k) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = 8 * wave + 4 * h + e;
      if (row >= rows_m) continue;
      const int64_t at = (m0 + row) * P.k + k0 + c;
      if (P.y_bf16)
        reinterpret_cast<uint16_t*>(P.y)[at] = (uint16_t)f32_to_bf16_bits(sum[j][e]);
      else
        reinterpret_cast<float*>(P.y)[at] = sum[j][e];
    }
  }
}

}  // namespace

hipError_t launch_mx_bf16_narrow(const MxBf16Problem& p, uint32_t splits, char* partial, uint32_t* counted,
                                 hipStream_t stream) {
  const int64_t tiles_m = (p.m + kRows - 1) / kRows, tiles_n = (p.k + kCols - 1) / kCols, tiles = tiles_m * tiles_n;
  const NarrowArgs g{(uint32_t)tiles_m, (uint32_t)tiles_n, splits, reinterpret_cast<uint64_t*>(partial), counted};
  const dim3 grid((uint32_t)((tiles * splits + 7) / 8 * 8));
  mx_bf16_narrow_kernel<<<grid, dim3(kThreads), 0, stream>>>(p, g);
  return hipGetLastError();
}

}  // namespace w4
