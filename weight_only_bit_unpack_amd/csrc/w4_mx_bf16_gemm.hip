// Products of bf16 rows with MXFP4 weights (gfx950): y = x W^T, the gated block
// h = act(x Wg^T) * (x Wu^T), and dx = dy W.
//
// The weight's values are rebuilt to bf16 between LDS and the matrix core
// (v_cvt_scalef32_pk_bf16_fp4: two values an instruction, exact but for values
// below 2^-126, which bf16 rounds) and multiplied by v_mfma_f32_32x32x16_bf16
// with fp32 sums.  LDS holds the stored 4 bits, so that a step's weights cost an
// eighth of the rows' LDS traffic, and a wave rebuilds only its own columns.
//
// Both directions take steps of 64 of the summed index.  Lane half h works on
// 32 h .. 32 h + 31 of a step, eight at a time (a quarter), the same eight for
// both operands, so the sums are over the same pairs whatever the order.
//
// Forward, the sum is along the rows of W: a lane's 32 values of a step are one
// MX block, 16 bytes with one scale.  Of a wave's 64 weight rows, tile j = 0, 1
// takes rows 2 r + j (r the lane's column), so that a lane ends with neighbouring
// outputs; gated, tile 0 takes gate rows and tile 1 the up rows beside them, so
// that a lane ends with both factors, and of two rows one half of 32 lanes stores the
// first and the other the second, neighbouring outputs a lane.
//
// Backward, the sum is over the rows of W, and its 4 bits lie along the other
// index: a step's weights are rebuilt a step ahead, once for the block, to bf16
// rows in LDS, and ds_read_b64_tr_b16 gives a lane four rows of one column.
//
// Bound, many rows: by the card's power and the matrix cores, 61% busy with the clock down
// to 1.6 to 1.9 GHz (gated 4096 x 11008 x 4096 600 us, 1.23 PFLOP/s; 2048 x 4096 x 11008 150
// us, 1.23; backward 4096 x 22016 x 4096 560 us, 1.32; the vendor library's dense product
// of bf16 at 4096 x 22016 x 4096 624 us); few rows: by the chain of a step (0.4 to 0.8 us a
// step of 64 whatever the tile below 128 x 256), the start and end of a launch and the
// joining of parts (96 x 2048 x 5632 backward 14.3 us, 3 of them the join).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "w4_launch.h"
#include "w4_lds_copy.h"
#include "w4_mx_act.h"
#include "w4_mx_device.h"
#include "w4_mx_parts.h"

namespace w4 {
namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));

// A block of BM rows of x by BN columns (forward: weight rows): WM x WN waves,
// each with MT x 2 accumulators of 32 x 32, and WK groups of such waves that take
// the steps of 64 in turn, each with LDS of its own: where there are too few
// tiles to give a SIMD two waves otherwise, its instructions' latencies are the
// bound.  NS (backward: NB) steps of a group in LDS: one read, the others arriving.
//
// LC > 0: forward, the scales of LC steps of every group come at once, copied by the
// whole block: then a copy reads eight neighbouring bytes of eight rows, not two of
// 32 rows with a line each, which keep the cache busy longer than the waves where two
// of them share a SIMD (1024 x 4096 x 4096 on T1 44.1 instead of 49.7 us, 333 x 5504 x
// 4096 on T3 29.9, 36.5).  Where a wave is alone there, or power is the bound, the extra
// instructions cost more (333 x 5504 x 4096 on T2 34.4, 31.0; 2048 x 4096 x 11008 on T0
// 205, 192; T4 within 2%).
template <int BM_, int BN_, int WM_, int WN_, int WK_, int NS_, int NB_, int LC_ = 0>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, WK = WK_, NS = NS_, NB = NB_, LC = LC_;
  static constexpr int NW = WM * WN, THREADS = 64 * NW * WK, MT = BM / WM / 32;
  static_assert(BN == 64 * WN && BM == 32 * WM * MT, "waves of 32 MT x 64");
  // 16-byte units of a step: rows of x, weights, scale bytes (a dword each)
  static constexpr int A = BM * 8, W = BN * 2, S = BN / 2;
  static constexpr int R = BN * 8;  // backward: 64 rows of BN rebuilt weights
  static constexpr int IA = A / (64 * NW), IW = W / (64 * NW), IS = 4 * S / (64 * NW);  // copies of a wave
  static_assert(IA * 64 * NW == A && IW * 64 * NW == W && IS == IW, "the waves share the copies");
  // a chunk of scales: blocks, units, copies of a wave
  static constexpr int SC = LC > 0 ? 2 * WK * LC : 8, C = LC > 0 ? BN * SC / 4 : 0, IC = C / (16 * NW * WK);
  static_assert(LC == 0 || (NS <= LC + 1 && IC * 16 * NW * WK == C), "what a chunk overwrites is read; waves share");
  // units of a group's LDS, and of a block's
  static constexpr int FORWARD = NS * (A + W + (LC > 0 ? 0 : S)), BACKWARD = NB * (A + W + S) + 2 * R;
  static constexpr int ALL_FORWARD = WK * FORWARD + 2 * C, ALL_BACKWARD = WK * BACKWARD;
  static_assert(ALL_FORWARD < 10240 && ALL_BACKWARD < 10240, "the LDS of a CU");
  static_assert((WK - 1) * BM * BN / 4 <= WK * FORWARD, "the groups' sums fit in it");
};
using T0 = Tile<256, 256, 2, 4, 1, 3, 2>;
using T1 = Tile<128, 256, 2, 4, 1, 3, 3, 4>;
using T2 = Tile<128, 128, 2, 2, 1, 3, 2>;
using T3 = Tile<64, 128, 2, 2, 2, 3, 2, 2>;
using T4 = Tile<32, 64, 1, 1, 4, 3, 0>;  // (backward: the narrow kernel, whose tiles are the same)
constexpr int kTiles = 5;

constexpr uint32_t kMaxSplits = kMxMaxSplits;
// An offset past the resource of a tile's outputs (below 2^31 bytes), also with
// the offset of a row added.
constexpr uint32_t kStoreOOB = 0x80000000u;

// The first `whole` of the tiles are one block's each.  The sums of the others
// (all, or what is left of the last round of blocks) are cut into `splits`
// parts, a block each: a part writes its sums to partial, and the block that
// counts last adds the parts of its tile in order.  Nobody waits.
struct GemmArgs {
  uint32_t tiles_m, tiles_n, whole, splits;
  uint64_t* partial;  // [tile behind the whole ones][part][BM BN / 2], pairs of fp32
  uint32_t* counted;  // [tile behind the whole ones], zeros between launches
};

// What a copy past the end of the summed index reads.
__device__ const u32x4 kZeros[1] = {};

// 16-byte unit c of row `row` of x lies at unit c ^ swizzle_x(row) of its 128
// bytes in LDS: the reads of 16 rows take 16 different units of the banks' 256
// bytes.
__device__ __forceinline__ int swizzle_x(int row) { return (row >> 1) & 7; }
// The same for the weights forward (rows of two units).
__device__ __forceinline__ int swizzle_w(int row) { return (row >> 3) & 1; }
// Where unit c of row `row` of the rebuilt weights lies in its row: the writes
// (16 lanes: rows beside each other, every fourth unit) and the transposing reads
// (32 lanes: four rows, four units each) both take all of the banks' units.
template <int BN>
__device__ __forceinline__ int swizzle_r(int row, int c) {
  const int n0 = row & 1, n1 = (row >> 1) & 1, c3 = (c >> 3) & 1, c4 = (c >> 4) & 1;
  static_assert(BN == 256 || BN == 128, "the tiles of the backward products");
  return c ^ (n1 << 3 | n0 << 2 | (n0 ^ c3) << 1 | (BN == 256 ? c4 : n1));
}

// Gated, lane r works on column gate_column(r) of a wave's 32: neighbours lie 16 lanes
// apart.
__device__ __forceinline__ int gate_column(int r) { return 2 * (r & 15) + (r >> 4); }

template <int KIND, typename T>
__global__ __launch_bounds__(T::THREADS) void mx_bf16_gemm_kernel(MxBf16Problem P, GemmArgs G) {
  constexpr bool kBack = KIND == kMxBackward, kGate = KIND == kMxGated;
  constexpr bool kChunks = !kBack && T::LC > 0;
  constexpr int MT = T::MT, NS = kBack ? T::NB : T::NS, SC = T::SC, LC = kChunks ? T::LC : 1;
  // of a wave and step (a chunk's come before those of its first step, so that a wait
  // that counts without them waits for them too)
  constexpr int kCopies = T::IA + T::IW + (kChunks ? 0 : T::IS);
  constexpr int U = T::BN / 32;                        // backward: units of a weight row in the tile
  constexpr int OUT = kGate ? T::BN / 2 : T::BN;       // outputs of a row in the tile
  extern __shared__ u32x4 lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int waves = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave = waves % T::NW, group = waves / T::NW;  // of the group
  const int wm = wave % T::WM, wn = wave / T::WM;
  const int r = lane & 31, h = lane >> 5;

  // Blocks are dealt to the 8 XCDs round robin; each XCD takes a contiguous
  // range of the whole tiles, and then of the parts, whose rows of x and w meet in
  // its L2: eight tiles of rows beside each other, then the next tile of columns.
  // (Each of the two kinds has a multiple of 8 blocks.)
  const uint32_t first = (G.whole + 7) / 8 * 8;
  const bool cut = blockIdx.x >= first;
  const uint32_t items = cut ? (G.tiles_m * G.tiles_n - G.whole) * G.splits : G.whole;
  const uint32_t at = cut ? blockIdx.x - first : blockIdx.x, L = at % 8 * ((items + 7) / 8) + at / 8;
  if (at / 8 >= (items + 7) / 8 || L >= items) return;
  const uint32_t splits = cut ? G.splits : 1, split = L % splits, tile = (cut ? G.whole : 0) + L / splits;
  const uint32_t band = tile / (8 * G.tiles_n), in = tile % (8 * G.tiles_n);
  const uint32_t height = G.tiles_m - 8 * band < 8 ? G.tiles_m - 8 * band : 8;
  const uint32_t mt = 8 * band + in % height, nt = in / height;

  const int64_t N = kBack ? P.k : P.n;                 // outputs of a row
  const int64_t m0 = (int64_t)mt * T::BM, n0 = (int64_t)nt * OUT;
  const int rows_m = (int)(P.m - m0 < T::BM ? P.m - m0 : T::BM);
  const int cols_n = (int)(N - n0 < OUT ? N - n0 : OUT);
  const uint32_t half = (uint32_t)(P.k >> 1), blocks = (uint32_t)(P.k >> 5);
  // this part's steps of 64 terms, t0 .. t1 - 1, of which the group takes every
  // WK-th; `count` each (a group's last may lie behind t1: zeros)
  const uint32_t terms = (uint32_t)(kBack ? P.n : P.k), steps = (terms + 63) / 64;
  const uint32_t t0 = (uint32_t)((uint64_t)split * steps / splits);
  const uint32_t t1 = (uint32_t)((uint64_t)(split + 1) * steps / splits);
  const uint32_t end = split + 1 == splits ? terms : 64 * t1;  // of the part's terms
  const uint32_t count = (t1 - t0 + T::WK - 1) / T::WK;
  auto step_at = [&](uint32_t i) { return t0 + group + T::WK * i; };

  // where a step's slots start, in units: ring slot s, the rebuilt weights of step i
  const uint32_t base = group * (kBack ? T::BACKWARD : T::FORWARD);
  auto slot_a = [&](uint32_t s) { return base + s * T::A; };
  auto slot_w = [&](uint32_t s) { return base + NS * T::A + s * T::W; };
  auto slot_s = [&](uint32_t s) { return base + NS * (T::A + T::W) + s * T::S; };
  auto slot_c = [&](uint32_t c) { return T::WK * T::FORWARD + (c & 1) * T::C; };  // chunk c of scales
  auto slot_r = [&](uint32_t i) { return base + NS * (T::A + T::W + T::S) + (i & 1) * T::R; };
  const uint32_t lds0 = lds_address(lds);

  // ---- copies: unit `wave * I + i` of 64 of the step's, one 16-byte unit (scales: one byte) a lane.
  // Rows and columns past the last repeat it and are never stored; past the end
  // of the sum both operands read zeros (and scales byte 0, no NaN).
  const uint8_t* const zeros = reinterpret_cast<const uint8_t*>(kZeros);
  const uint8_t* const xb = uniform(reinterpret_cast<const uint8_t*>(P.x + m0 * P.x_pitch));
  auto unit_x = [&](int l, int i) {  // its unit in the row of x
    const int u = (wave * T::IA + i) * 64 + l;
    return (u & 7) ^ swizzle_x(u >> 3);
  };
  uint32_t xv[T::IA];  // (a block's rows: at most 256 of 2^23 bytes)
#pragma unroll
  for (int i = 0; i < T::IA; ++i) {
    const int row = ((wave * T::IA + i) * 64 + lane) >> 3;
    xv[i] = (uint32_t)(row < rows_m ? row : rows_m - 1) * (uint32_t)(2 * P.x_pitch) + 16u * unit_x(lane, i);
  }
  // forward: the weight row of LDS row i
  auto weight_row = [&](int i) -> int64_t {
    if constexpr (kGate) {
      const int c = (i >> 6) * 32 + gate_column(i & 31);
      return n0 + (c < cols_n ? c : cols_n - 1) + ((i >> 5) & 1) * P.n;
    } else {
      const int c = (i & ~63) + 2 * (i & 31) + ((i >> 5) & 1);
      return n0 + (c < cols_n ? c : cols_n - 1);
    }
  };
  // the row (backward) or block (forward) of the step that a lane copies
  auto at_w = [&](int l, int i) {
    const int u = (wave * T::IW + i) * 64 + l;
    return kBack ? u / U : (u & 1) ^ swizzle_w(u >> 1);
  };
  auto at_s = [&](int l, int i) {
    const int u = (wave * T::IS + i) * 64 + l;
    return kBack ? u / U : u & 1;
  };
  const uint8_t* wp[T::IW];
#pragma unroll
  for (int i = 0; i < T::IW; ++i) {
    const int u = (wave * T::IW + i) * 64 + lane;
    if constexpr (kBack) {
      const uint32_t c = (uint32_t)(n0 >> 5) + u % U;
      wp[i] = P.w + (int64_t)(u / U) * half + 16 * (int64_t)(c < blocks ? c : blocks - 1);
    } else {
      wp[i] = P.w + weight_row(u >> 1) * half + 16 * at_w(lane, i);
    }
  }
  const uint8_t* sp[T::IS];
#pragma unroll
  for (int i = 0; i < T::IS; ++i) {
    const int u = (wave * T::IS + i) * 64 + lane;
    if constexpr (kChunks) {
      sp[i] = nullptr;
    } else if constexpr (kBack) {
      const uint32_t c = (uint32_t)(n0 >> 5) + u % U;
      sp[i] = P.w_scales + (int64_t)(u / U) * blocks + (c < blocks ? c : blocks - 1);
    } else {
      sp[i] = P.w_scales + weight_row(u >> 1) * blocks + (u & 1);
    }
  }
  // Chunk c: dword p of a row's SC holds block p ^ swizzle_c(row) of it, so that the
  // reads of 32 rows and two blocks take all banks.
  auto swizzle_c = [](int row) { return row / (64 / SC) % (SC / 2) * 2; };
  const uint8_t* const cb = uniform(P.w_scales + n0 * (int64_t)blocks + 2 * t0);
  uint32_t cv[kChunks ? T::IC : 1];  // (a tile's rows: at most 256 of 2^17 bytes; not the way to the up rows)
  if constexpr (kChunks) {
#pragma unroll
    for (int i = 0; i < T::IC; ++i) {
      const int row = ((waves * T::IC + i) * 64 + lane) / SC;
      const int c = kGate ? (row >> 6) * 32 + gate_column(row & 31) : (row & ~63) + 2 * (row & 31) + ((row >> 5) & 1);
      cv[i] = (uint32_t)(c < cols_n ? c : cols_n - 1) * blocks + ((lane % SC) ^ swizzle_c(row));
    }
  }
  auto copy_chunk = [&](uint32_t c) {
    const uint32_t b0 = 2 * t0 + SC * c;
#pragma unroll
    for (int i = 0; i < T::IC; ++i) {
      const int at = (waves * T::IC + i) * 64;  // (rows of one half of 64)
      const uint8_t* const from = uniform(cb + SC * c + (kGate ? (at / SC >> 5 & 1) * (P.n * blocks) : 0));
      const uint32_t to = lds0 + 16 * slot_c(c) + 4 * at;
      if (32 * (b0 + SC) <= end)
        copy_byte(from, cv[i], to);
      else
        copy_byte(32 * (b0 + ((lane % SC) ^ swizzle_c((at + lane) / SC))) < end ? from + cv[i] : zeros, to);
    }
  };
  const int64_t step_w = kBack ? 64 * (int64_t)half : 32, step_s = kBack ? 64 * (int64_t)blocks : 2;
  auto inside = [&](uint32_t t, int at) {  // row or block `at` of step t lies before the end of the sum
    return 64 * t + (kBack ? 1 : 32) * at < end;
  };
  // the weights and scales of the group's step i to ring slot s; WHOLE: all of it
  // lies before the end of the sum
  auto copy_weights = [&](uint32_t i, uint32_t s, auto WHOLE) {
    constexpr bool whole = decltype(WHOLE)::value;
    const uint32_t t = step_at(i);
#pragma unroll
    for (int c = 0; c < T::IW; ++c) {
      const uint8_t* from = wp[c] + t * step_w;
      if (!whole) from = inside(t, at_w(lane, c)) ? from : zeros;
      copy16(from, lds0 + 16 * (slot_w(s) + (wave * T::IW + c) * 64));
    }
    if constexpr (!kChunks) {
#pragma unroll
      for (int c = 0; c < T::IS; ++c) {
        const uint8_t* from = sp[c] + t * step_s;
        if (!whole) from = inside(t, at_s(lane, c)) ? from : zeros;
        copy_byte(from, lds0 + 16 * slot_s(s) + (wave * T::IS + c) * 256);
      }
    }
  };
  // step i to ring slot s (backward: with the weights of step i + 1, to the next slot)
  auto copy = [&](uint32_t i, uint32_t s, auto WHOLE) {
    const uint32_t t = step_at(i);
    if constexpr (kChunks)
      if (i % LC == 0) copy_chunk(i / LC);
    const uint32_t to_a = lds0 + 16 * (slot_a(s) + wave * T::IA * 64);
    const uint8_t* const xs = uniform(xb + (uint64_t)t * 128);
#pragma unroll
    for (int c = 0; c < T::IA; ++c) {
      if constexpr (decltype(WHOLE)::value)
        copy16(xs, xv[c], to_a + c * 1024);
      else
        copy16(64 * t + 8 * unit_x(lane, c) < end ? xs + xv[c] : zeros, to_a + c * 1024);
    }
    if constexpr (kBack)
      copy_weights(i + 1, s + 1 == NS ? 0 : s + 1, WHOLE);
    else
      copy_weights(i, s, WHOLE);
  };
  // steps i that copy() may take as whole
  const uint32_t full = end / 64 > step_at(0) ? (end / 64 - step_at(0) + T::WK - 1) / T::WK : 0;
  const uint32_t whole = kBack && full > 0 ? full - 1 : full;

  f32x16 acc[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;

  // ---- operands.  Forward, of a step: the lane's block and scale of each tile.
  // Of a quarter: x, and the weights rebuilt.
  struct Step {
    u32x4 w[2];
    uint32_t s[2];
  };
  struct Quarter {
    u32x4 a[MT];
  };
  struct Weights {
    u32x4 b[2];
  };
  auto read_step = [&](Step& v, uint32_t s, uint32_t i) {
    if constexpr (!kBack) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = wn * 64 + 32 * j + r;
        v.w[j] = lds[slot_w(s) + 2 * row + (h ^ swizzle_w(row))];
        if constexpr (kChunks)
          v.s[j] = reinterpret_cast<const uint32_t*>(
              lds + slot_c(i / LC))[row * SC + ((2 * T::WK * (i % LC) + 2 * group + h) ^ swizzle_c(r))];
        else
          v.s[j] = reinterpret_cast<const uint32_t*>(lds + slot_s(s))[2 * row + h];
      }
    }
  };
  auto read = [&](Quarter& v, uint32_t s, auto Q) {
    constexpr int q = decltype(Q)::value;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int row = wm * (32 * MT) + 32 * i + r;
      v.a[i] = lds[slot_a(s) + 8 * row + ((4 * h + q) ^ swizzle_x(row))];
    }
  };
  // a quarter's weights of step n: forward rebuilt, backward read as they were rebuilt
  auto weights = [&](Weights& v, const Step& st, uint32_t n, auto Q) {
    constexpr int q = decltype(Q)::value;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (kBack) {
        // sixteen lanes' addresses are four rows of four eight-byte pieces
        const int p = lane & 15, c = wn * 64 + 32 * j + 16 * ((lane >> 4) & 1) + 4 * (p & 3);
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const int row = 32 * h + 8 * q + 4 * d + (p >> 2);
          const u32x4* const at = lds + slot_r(n) + row * (T::BN / 8) + swizzle_r<T::BN>(row, c >> 3);
          const u32x2 x = __builtin_bit_cast(
              u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                         (__attribute__((address_space(3))) i16x4*)(reinterpret_cast<const u32x2*>(at) + (p & 1))));
          v.b[j][2 * d] = x.x;
          v.b[j][2 * d + 1] = x.y;
        }
      } else {
        v.b[j] = mx_rebuild8(st.w[j][q], st.s[j]);
      }
    }
  };
  // ---- backward: the weights of step n, in ring slot s, rebuilt to rows of bf16.
  // A wave takes the unit a lane that it copied itself: 32 values of one row and block.
  struct Unit {
    u32x4 w;
    uint32_t s;
  };
  auto read_unit = [&](Unit& v, uint32_t s) {
    const int u = wave * 64 + lane;
    v.w = lds[slot_w(s) + u];
    v.s = reinterpret_cast<const uint32_t*>(lds + slot_s(s))[u];
  };
  auto rebuild_unit = [&](const Unit& v, uint32_t n) {
    if constexpr (kBack) {
      const int u = wave * 64 + lane, row = u / U, c = u % U;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        lds[slot_r(n) + row * (T::BN / 8) + swizzle_r<T::BN>(row, 4 * c + e)] = mx_rebuild8(v.w[e], v.s);
    }
  };
  auto multiply_row = [&](const Quarter& o, const Weights& v, int i) {
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = mfma32x32x16(o.a[i], v.b[j], acc[i][j]);
  };
  auto multiply = [&](const Quarter& o, const Weights& v) {
#pragma unroll
    for (int i = 0; i < MT; ++i) multiply_row(o, v, i);
  };
  // Forward, a quarter's products with the next one's reads and rebuilding between
  // them: left alone, the compiler puts the reads behind the products and waits for
  // them before the next (4096 x 22016 x 4096 594 against 587 us).  Backward, where the
  // LDS has more to do, its order is the better one (563 against 584).
  auto interleave = [&]() {
    if constexpr (!kBack) {
      constexpr int products = 2 * MT, valu = 8 / products + 1;
#pragma unroll
      for (int n = 0; n < products; ++n) {
        if (n < MT) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, valu, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  using Q0 = std::integral_constant<int, 0>;
  using Q1 = std::integral_constant<int, 1>;
  using Q2 = std::integral_constant<int, 2>;
  using Q3 = std::integral_constant<int, 3>;

  // ---- the loop.  A quarter's operands are read and rebuilt while the one before
  // is multiplied, backward the next step's weights too, in the first quarter.  The
  // barrier of a step comes before its last quarter: by then every wave holds that
  // in registers, so the step's slot can take the copies of step t + NS, and the
  // next step's first operands are read, while it is multiplied.
  static_assert(!kBack || T::IW == 1, "a wave rebuilds one unit a lane");
  Step st;
  Quarter o0, o1;
  Weights b0, b1;
  Unit unit;
  uint32_t cur = 0;
  auto step = [&](uint32_t n, auto FAST) {
    constexpr bool fast = decltype(FAST)::value;  // step n + NS exists and is whole
    const uint32_t next = cur + 1 == NS ? 0 : cur + 1;
    if constexpr (kBack) read_unit(unit, next);
    read(o1, cur, Q1{});
    weights(b1, st, n, Q1{});
    multiply(o0, b0);
    interleave();
    if constexpr (kBack) rebuild_unit(unit, n + 1);
    read(o0, cur, Q2{});
    weights(b0, st, n, Q2{});
    multiply(o1, b1);
    interleave();
    read(o1, cur, Q3{});
    weights(b1, st, n, Q3{});
    multiply(o0, b0);
    interleave();
    // the last operands (on every path here: after the branch the compiler's
    // own wait would be for the next step's reads too)
    __builtin_amdgcn_s_waitcnt(kWaitLds);
    if (fast || n + 1 < count) {
      // the next step's copies: all but those of the NS - 2 steps after it
      if (fast || n + NS <= count)
        __builtin_amdgcn_s_waitcnt(wait_vm((NS - 2) * kCopies));
      else
        __builtin_amdgcn_s_waitcnt(wait_vm(0));
      lds_barrier();
      read_step(st, next, n + 1);
      read(o0, next, Q0{});
      if constexpr (kBack) weights(b0, st, n + 1, Q0{});
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (!fast) {
        if (n + NS < count) copy(n + NS, cur, std::false_type{});
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    multiply_row(o1, b1, 0);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (fast) copy(n + NS, cur, std::true_type{});
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 1; i < MT; ++i) multiply_row(o1, b1, i);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (!kBack) weights(b0, st, n + 1, Q0{});  // (of no step, behind the last)
    cur = next;
  };
  if constexpr (kBack) copy_weights(0, 0, std::false_type{});
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    if (kBack && i == NS - 1) {
      // these copies bring weights to the slot of t0's, which are rebuilt first
      // (behind a barrier: nothing else keeps their reads below the wait)
      if (NS - 1 <= count)
        __builtin_amdgcn_s_waitcnt(wait_vm((NS - 1) * kCopies));
      else
        __builtin_amdgcn_s_waitcnt(wait_vm(0));
      lds_barrier();
      read_unit(unit, 0);
      rebuild_unit(unit, 0);
      __builtin_amdgcn_s_waitcnt(kWaitLds);
      lds_barrier();
    }
    if (i < count) copy(i, i, std::false_type{});
  }
  if (NS <= count)
    __builtin_amdgcn_s_waitcnt(wait_vm((NS - 1) * kCopies));
  else
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
  lds_barrier();
  read_step(st, 0, 0);
  read(o0, 0, Q0{});
  weights(b0, st, 0, Q0{});
  const uint32_t fast = whole < count ? whole : count;  // steps n with n + NS < fast
  uint32_t n = 0;
  for (; n + NS < fast; ++n) step(n, std::true_type{});
  for (; n < count; ++n) step(n, std::false_type{});

  // ---- the groups' sums, in the order of the groups, to the first one, which goes
  // on (the others keep it company at the barriers)
  if constexpr (T::WK > 1) {
    constexpr int kVectors = MT * 2 * 4;  // of a thread
    f32x4* const sums = reinterpret_cast<f32x4*>(lds) + wave * 64 + lane;
    __syncthreads();  // (every copy has arrived and every operand is read)
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            sums[((group - 1) * kVectors + (i * 2 + j) * 4 + v) * (64 * T::NW)] =
                (f32x4){acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2], acc[i][j][4 * v + 3]};
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int g = 1; g < T::WK; ++g)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const f32x4 x = sums[((g - 1) * kVectors + (i * 2 + j) * 4 + v) * (64 * T::NW)];
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][j][4 * v + e] += x[e];
            }
    }
  }
  const bool lead = T::WK == 1 || group == 0;

  if (splits > 1) {
    constexpr int kPairs = MT * 2 * 8, kLead = 64 * T::NW;  // of a thread, threads
    uint64_t* const parts = G.partial + (uint64_t)(tile - G.whole) * splits * (kPairs * kLead) + tid;
    if (lead)
      put_part<kPairs>(parts + (uint64_t)split * (kPairs * kLead), kLead, [&](int v) {
        const f32x16& a = acc[v / 16][v / 8 % 2];
        return (f32x2){a[v % 8 * 2], a[v % 8 * 2 + 1]};
      });
    if (!last_part(G.counted + (tile - G.whole), splits, reinterpret_cast<uint32_t*>(lds)) || !lead) return;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        add_parts<8, 4>(parts + (i * 2 + j) * 8 * kLead, kPairs * kLead, kLead, splits, [&](int v, const f32x2& x) {
          acc[i][j][2 * v] = x.x;
          acc[i][j][2 * v + 1] = x.y;
        });
  }

  if (!lead) return;

  // ---- outputs.  D[row of x][column]: lane half h, register q hold row
  // 8 (q / 4) + 4 h + q % 4 of column r.  Stores go through a resource that ends
  // with the last row; columns past the last take an offset past it.
  const int row0 = wm * (32 * MT) + 4 * h;
  auto row_of = [](int i, int q) { return 32 * i + 8 * (q >> 2) + (q & 3); };
  auto resource = [&](void* base, int64_t pitch, int64_t col, int size) {
    const uint8_t* const b0 = uniform(reinterpret_cast<const uint8_t*>(base) + (m0 * pitch + col) * size);
    return mx_rsrc(b0, (uint32_t)(rows_m - 1) * (uint32_t)(pitch * size) + (uint32_t)cols_n * size);
  };
  // one value a lane at column c of the tile, fp32 or bf16
  auto put_f32 = [&](__amdgpu_buffer_rsrc_t d, uint32_t pitch, int c, auto&& value) {
    const uint32_t at = c < cols_n ? (uint32_t)row0 * pitch + 4u * c : kStoreOOB;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int q = 0; q < 16; ++q)
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, (float)value(i, q)), d,
                                              at + row_of(i, q) * pitch, 0, 0);
  };
  // PAIRS: neighbouring lanes' columns, 4-byte aligned: of rows q and q + 1 a
  // lane and its neighbour keep one each and swap the other
  auto put_bf16 = [&](__amdgpu_buffer_rsrc_t d, uint32_t pitch, int c, bool pairs, auto&& value) {
    if (pairs) {
      const int odd = lane & 1;
      const uint32_t at = c < cols_n ? (uint32_t)(row0 + odd) * pitch + 2u * (c & ~1) : kStoreOOB;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < 16; q += 2) {
          const float e = value(i, q), f = value(i, q + 1);
          // quad_perm [1,0,3,2]
          const float got = __builtin_bit_cast(
              float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, odd ? e : f), 0xB1, 0xF, 0xF, true));
          __builtin_amdgcn_raw_buffer_store_b32(cvt_pk_bf16(odd ? got : e, odd ? f : got), d,
                                                at + row_of(i, q) * pitch, 0, 0);
        }
    } else {
      const uint32_t at = c < cols_n ? (uint32_t)row0 * pitch + 2u * c : kStoreOOB;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q)
          __builtin_amdgcn_raw_buffer_store_b16((uint16_t)f32_to_bf16_bits(value(i, q)), d,
                                                at + row_of(i, q) * pitch, 0, 0);
    }
  };
  // Gated: rows q and q + 1 of a lane's column (v_permlane16_swap_b32) become the
  // columns beside each other of row q in the first 16 lanes of 32, of q + 1 in the others.
  // With lanes of the two rows by turns 4096 x 11008 x 4096 took 616 instead of 608 us
  // (stores past the caches: gu the same, y 592, but the next product reads y).
  auto put_gated = [&](void* base, int64_t out_pitch, int64_t col, bool bf16, auto&& value) {
    const int size = bf16 ? 2 : 4;
    const __amdgpu_buffer_rsrc_t d = resource(base, out_pitch, col, size);
    const uint32_t pitch = (uint32_t)out_pitch * size;
    if ((N & 1) == 0 && (reinterpret_cast<uintptr_t>(base) & 3) == 0) {
      const int c = wn * 32 + 2 * (r & 15);
      const uint32_t at = c < cols_n ? (uint32_t)(row0 + (r >> 4)) * pitch + (uint32_t)(size * c) : kStoreOOB;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < 16; q += 2) {
          const auto v = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, (float)value(i, q)),
                                                          __builtin_bit_cast(uint32_t, (float)value(i, q + 1)), false, false);
          const uint32_t even = v[0], odd = v[1];  // (a cast of the element itself takes the first one)
          if (bf16)
            __builtin_amdgcn_raw_buffer_store_b32(
                cvt_pk_bf16(__builtin_bit_cast(float, even), __builtin_bit_cast(float, odd)), d,
                at + row_of(i, q) * pitch, 0, 0);
          else
            __builtin_amdgcn_raw_buffer_store_b64((u32x2){even, odd}, d, at + row_of(i, q) * pitch, 0, 0);
        }
    } else if (bf16) {
      put_bf16(d, pitch, wn * 32 + gate_column(r), false, value);
    } else {
      put_f32(d, pitch, wn * 32 + gate_column(r), value);
    }
  };
  if constexpr (kGate) {
    auto gate = [&](int i, int q) -> float { return acc[i][0][q]; };
    auto up = [&](int i, int q) -> float { return acc[i][1][q]; };
    if (P.gu) {
      put_gated(P.gu, 2 * N, n0, true, gate);
      put_gated(P.gu, 2 * N, N + n0, true, up);
    }
    with_activation(P.act, [&](auto ACT) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][0][q] = activate<decltype(ACT)::value>(acc[i][0][q]) * acc[i][1][q];
    });
    put_gated(P.y, N, n0, P.y_bf16, gate);
  } else {
    const int size = P.y_bf16 ? 2 : 4;
    const __amdgpu_buffer_rsrc_t d = resource(P.y, N, n0, size);
    const uint32_t pitch = (uint32_t)N * size;
    const bool pairs = (N & 1) == 0 && (reinterpret_cast<uintptr_t>(P.y) & 3) == 0;
    if constexpr (kBack) {  // tile j's columns 32 j + r
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        auto value = [&](int i, int q) -> float { return acc[i][j][q]; };
        if (size == 2)
          put_bf16(d, pitch, wn * 64 + 32 * j + r, pairs, value);
        else
          put_f32(d, pitch, wn * 64 + 32 * j + r, value);
      }
      return;
    }
    const int c = wn * 64 + 2 * r;
    if (size == 2 && pairs) {
      const uint32_t at = c < cols_n ? (uint32_t)row0 * pitch + 2u * c : kStoreOOB;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q)
          __builtin_amdgcn_raw_buffer_store_b32(cvt_pk_bf16(acc[i][0][q], acc[i][1][q]), d,
                                                at + row_of(i, q) * pitch, 0, 0);
    } else if (size == 2) {
#pragma unroll
      for (int j = 0; j < 2; ++j) put_bf16(d, pitch, c + j, false, [&](int i, int q) -> float { return acc[i][j][q]; });
    } else if ((N & 1) == 0) {
      const uint32_t at = c < cols_n ? (uint32_t)row0 * pitch + 4u * c : kStoreOOB;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q)
          __builtin_amdgcn_raw_buffer_store_b64(
              (u32x2){__builtin_bit_cast(uint32_t, (float)acc[i][0][q]), __builtin_bit_cast(uint32_t, (float)acc[i][1][q])},
              d, at + row_of(i, q) * pitch, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) put_f32(d, pitch, c + j, [&](int i, int q) -> float { return acc[i][j][q]; });
    }
  }
}

int device_cus() {
  int dev = 0, cus = 256;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    cus = 256;
  return cus;
}

template <typename F>
auto with_tile(int tile, F&& f) {
  switch (tile) {
    case 0: return f(T0{});
    case 1: return f(T1{});
    case 2: return f(T2{});
    case 3: return f(T3{});
    default: return f(T4{});
  }
}

// tiles_m * tiles_n tiles, the first `whole` unsplit, the others in `splits` parts.
struct Plan {
  int tile;
  uint32_t splits;
  int64_t tiles_m, tiles_n, whole;
  int64_t cut() const { return tiles_m * tiles_n - whole; }
  int64_t blocks() const { return (whole + 7) / 8 * 8 + (cut() * splits + 7) / 8 * 8; }
};

int64_t outputs(const MxBf16Problem& p) { return p.kind == kMxBackward ? p.k : p.n; }
int64_t steps_of(const MxBf16Problem& p) { return ((p.kind == kMxBackward ? p.n : p.k) + 63) / 64; }

constexpr int64_t kMaxParts = kMxMaxParts;

// Tile number t, the tiles from `whole` on in s parts (s == 1: none); tile < 0
// where they do not fit the problem: a tile's rows of x and of outputs stay below
// 2^31 bytes, each part has a step, and a launch holds the blocks.
template <typename T>
Plan plan_on(const MxBf16Problem& p, int t, uint32_t s, int64_t whole) {
  const int64_t N = outputs(p), wide = p.kind == kMxGated ? 2 * N : N;
  const int64_t cols = p.kind == kMxGated ? T::BN / 2 : T::BN;
  Plan q{t, s, (p.m + T::BM - 1) / T::BM, (N + cols - 1) / cols, whole};
  const int64_t tiles = q.tiles_m * q.tiles_n;
  if (s == 1) q.whole = tiles;
  constexpr int64_t kTileBytes = (INT64_C(1) << 31) - 1;
  if (4 * wide > kTileBytes / T::BM || 2 * p.x_pitch > kTileBytes / T::BM) q.tile = -1;
  if (q.whole > tiles || (int64_t)s > steps_of(p) || (s > 1 && q.cut() * s > kMaxParts)) q.tile = -1;
  if (std::is_same_v<T, T4> && p.kind == kMxBackward && s > 1 && q.whole > 0) q.tile = -1;  // (all tiles or none)
  if ((tiles + kMaxParts + 14) * T::THREADS > kMaxLaunchThreads) q.tile = -1;
  return q;
}

// What a product costs on a tile: a block alone on its CU takes first + step us for
// its start and end and per step of a group, two blocks that share one (where they
// fit) first2 + step2; but a step of all blocks together no less than its operations
// at `rate` (PFLOP/s, tile 0 and the others), which is what the card's power allows.
// A launch takes `launch`, and sums in parts take `join` and, for each part, `part` and
// its bytes at 64 KB a `copy`.  perf/mx_bf16_plans.py times every tile and number of parts
// and fits these; the table in profiles/mx_bf16_plans.txt holds 8735 times of 447 products of
// 1 to 8192 rows, 300 to 22016 columns and sums of 300 to 22016, on which their error is 7.7
// to 8.0% (root mean square).  The plans they choose take 0.8% more there than the best ones
// on average, and at most 1.22 times as long (333 x 5500 x 4096, 30.5 us in three parts on
// tile 1, 24.9 on tile 3 with the last round's tiles in four): plans beside each other differ
// by less than the error.  Examples (us, graph replays): 64 x 1000 x 4096 8.5 on tile 4 in
// four parts, 10.7 in one, 11.6 on tile 3 in four; gated 333 x 2730 x 2080 21.1 on tile 2,
// 21.7 on tile 3 and 19.2 there with the last round's tiles in three parts, 23.5 on tile 4;
// 2048 x 4096 x 11008 148 on tile 1, 155 on tile 0 in two parts, 192 in one; backward 163 on
// tile 0 with the last round's tiles in two parts, 184 without, 191 on tile 1.
struct Cost {
  float first, step, first2, step2;  // first2 == 0: one block a CU
};
struct Costs {
  Cost tile[kTiles];
  float launch, join, part, copy, rate[2];
};
constexpr Costs kCosts[3] = {
    {{{7.20f, 1.03f, 0, 0}, {4.46f, 0.59f, 0, 0}, {2.52f, 0.42f, 6.61f, 0.89f}, {1.79f, 0.55f, 3.95f, 1.01f}, {2.17f, 0.42f, 2.58f, 0.78f}},
     1.6f, 2.09f, 0.24f, 0.92f, {1.30f, 1.26f}},
    {{{12.4f, 1.07f, 0, 0}, {7.02f, 0.60f, 0, 0}, {3.92f, 0.42f, 6.90f, 0.93f}, {2.31f, 0.55f, 4.30f, 1.04f}, {2.45f, 0.42f, 3.19f, 0.80f}},
     2.1f, 2.09f, 0.24f, 0.90f, {1.38f, 1.28f}},
    {{{8.26f, 1.30f, 0, 0}, {5.07f, 0.95f, 0, 0}, {3.82f, 0.62f, 8.80f, 0.97f}, {3.42f, 0.80f, 0, 0}, {2.19f, 0.78f, 2.83f, 1.37f}},
     0.5f, 2.26f, 0.11f, 0.99f, {1.29f, 1.32f}}};

Plan make_plan(const MxBf16Problem& p) {
  const int64_t cus = device_cus();
  const Costs& costs = kCosts[p.kind];
  Plan best{4, 1, 0, 0, 0};
  double least = 0;
  for (int t = 0; t < kTiles; ++t)
    with_tile(t, [&](auto X) {
      using T = decltype(X);
      const Cost& c = costs.tile[t];
      // us of a block and step of its groups at the rate
      const double power = T::BM * T::BN * T::WK * 128e-9 / costs.rate[t > 0];
      auto steps_in = [](int64_t steps) { return (double)((steps + T::WK - 1) / T::WK); };
      // blocks of so many steps each, in rounds over the CUs
      auto rounds = [&](int64_t blocks, int64_t steps) {
        const bool pairs = c.first2 > 0;
        const int64_t per = pairs ? 2 * cus : cus, rest = blocks % per;
        auto round = [&](bool pair, int64_t n) {
          return (pair ? c.first2 : c.first) + steps_in(steps) * std::max<double>(pair ? c.step2 : c.step, n * power);
        };
        return (double)(blocks / per) * round(pairs, per) + (rest > 0 ? round(rest > cus, rest) : 0);
      };
      for (uint32_t s : {1u, 2u, 3u, 4u, 6u, 8u, 12u, 16u}) {
        Plan q = plan_on<T>(p, t, s, 0);
        const int64_t tiles = q.tiles_m * q.tiles_n;
        if (s > 1 && tiles > cus) q = plan_on<T>(p, t, s, tiles / cus * cus);
        if (q.tile < 0) continue;
        double us = costs.launch + rounds(q.whole, steps_of(p));
        if (s > 1) {
          // behind an odd number of rounds of whole tiles that leave room beside them, the
          // parts run beside the last round and slow it down
          const int64_t steps = (steps_of(p) + s - 1) / s, parts = q.cut() * s;
          if (c.first2 > 0 && q.whole / cus % 2 == 1)
            us += steps_in(steps) * std::max<double>(c.step2 - c.step, std::min(parts, cus) * power) +
                  rounds(parts > cus ? parts - cus : 0, steps);
          else
            us += rounds(parts, steps);
          us += costs.join + s * (costs.part + costs.copy * T::BM * T::BN / 16384.0);
        }
        if (best.tiles_m == 0 || us < least) {
          least = us;
          best = q;
        }
      }
    });
  if (best.tiles_m == 0) best.tiles_m = best.tiles_n = best.whole = INT64_C(1) << 31;  // too many tiles of every size
  return best;
}

template <int KIND, typename T>
hipError_t launch_tile(const MxBf16Problem& p, const GemmArgs& g, uint32_t blocks, hipStream_t stream) {
  constexpr int lds = 16 * (KIND == kMxBackward ? T::ALL_BACKWARD : T::ALL_FORWARD);
  // the LDS limit is raised once per device (one bit each for the first 64);
  // callers racing here all set the same value
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&mx_bf16_gemm_kernel<KIND, T>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    configured.fetch_or(bit, std::memory_order_release);
  }
  mx_bf16_gemm_kernel<KIND, T><<<dim3(blocks), dim3(T::THREADS), lds, stream>>>(p, g);
  return hipGetLastError();
}

// The workspace: the caller's `reserve` bytes (whole 256), then the parts' sums.
template <typename F>
hipError_t launch_plan(const MxBf16Problem& problem, const Plan& q, size_t reserve, hipStream_t stream, F&& fill) {
  MxBf16Problem p = problem;
  GemmArgs g{(uint32_t)q.tiles_m, (uint32_t)q.tiles_n, (uint32_t)q.whole, q.splits, nullptr, nullptr};
  return with_tile(q.tile, [&](auto X) -> hipError_t {
    using T = decltype(X);
    const size_t bytes = reserve + (q.splits > 1 ? (size_t)q.cut() * q.splits * T::BM * T::BN * sizeof(float) : 0);
    char* ws = nullptr;
    std::unique_lock<std::mutex> turn;  // (parts are put and added in one launch)
    if (reserve > 0) turn = stream_turn(stream);
    hipError_t e = bytes ? stream_workspace(kWorkspaceMx, stream, bytes, &ws) : hipSuccess;
    if (e == hipSuccess && q.splits > 1) e = stream_counters(stream, q.splits, &g.counted);
    if (e == hipSuccess) e = fill(p, ws);
    if (e != hipSuccess) return e;
    g.partial = reinterpret_cast<uint64_t*>(ws + reserve);
    const uint32_t blocks = (uint32_t)q.blocks();
    if (p.kind == kMxGated) return launch_tile<kMxGated, T>(p, g, blocks, stream);
    if (p.kind == kMxForward) return launch_tile<kMxForward, T>(p, g, blocks, stream);
    if constexpr (std::is_same_v<T, T4>)
      return launch_mx_bf16_narrow(p, q.splits, ws + reserve, g.counted, stream);
    else
      return launch_tile<kMxBackward, T>(p, g, blocks, stream);
  });
}

// Forward products with few rows have a kernel of their own.
bool skinny(const MxBf16Problem& p) { return p.m <= 16 && p.kind != kMxBackward; }

}  // namespace

bool mx_bf16_fits(const MxBf16Problem& p) {
  // No tile is smaller than 32 x 32 outputs or has more than 512 threads, and the
  // few-row kernels have fewer blocks: where a launch holds the blocks of that, it
  // holds any plan's, and the costs are computed by the launch only.
  if (((p.m + 31) / 32 * ((outputs(p) + 31) / 32) + kMaxParts + 14) * 512 <= kMaxLaunchThreads) return true;
  return make_plan(p).blocks() <= 0x7FFFFFFF;
}

hipError_t launch_mx_bf16_with(const MxBf16Problem& p, size_t reserve, MxBf16Fill* fill, hipStream_t stream) {
  if (skinny(p)) return launch_mx_bf16_skinny(p, mx_bf16_skinny_shape(p), stream);
  return launch_plan(p, make_plan(p), reserve, stream, [&](MxBf16Problem& on, char* ws) {
    return fill ? (*fill)(on, ws) : hipSuccess;
  });
}

extern "C" int32_t w4_mx_bf16_kernel_of(int32_t kind, int64_t n, int64_t k, int64_t m) {
  const MxBf16Problem p{nullptr, nullptr, nullptr, nullptr, nullptr, m, n, k, kind == kMxBackward ? n : k, 0, 0, kind};
  if (skinny(p)) return 4096 + mx_bf16_skinny_shape(p);
  const Plan q = make_plan(p);
  return (q.whole > 0 && q.splits > 1 ? 1024 : 0) + 16 * (int32_t)q.splits + q.tile;
}

extern "C" int32_t w4_mx_bf16_product_on(int32_t kernel, int32_t kind, int32_t act, int64_t n, int64_t k,
                                         const uint8_t* w, const uint8_t* w_scales, const uint16_t* x, int64_t m,
                                         uint16_t* gu, void* y, int32_t y_bf16, void* stream) {
  const MxBf16Problem p{w, w_scales, x, y, gu, m, n, k, kind == kMxBackward ? n : k, y_bf16, act, kind};
  if (kind < kMxForward || kind > kMxBackward || (kind == kMxBackward && n % 8)) return hipErrorInvalidValue;
  if (kernel >= 4096) {
    if (kernel > 4098 || kind == kMxBackward || m > 16) return hipErrorInvalidValue;
    return launch_mx_bf16_skinny(p, kernel - 4096, static_cast<hipStream_t>(stream));
  }
  const int32_t parts = kernel % 1024 / 16, tile = kernel % 16;
  if (kernel < 0 || kernel >= 2048 || tile >= kTiles || parts < 1 || parts > (int32_t)kMaxSplits)
    return hipErrorInvalidValue;
  const Plan q = with_tile(tile, [&](auto X) {
    const Plan all = plan_on<decltype(X)>(p, tile, (uint32_t)parts, 0);
    if (kernel < 1024) return all;
    const int64_t tiles = all.tiles_m * all.tiles_n, cus = device_cus();
    return plan_on<decltype(X)>(p, tile, (uint32_t)parts, tiles > cus ? tiles / cus * cus : tiles / 2 / 8 * 8);
  });
  if (q.tile < 0) return hipErrorInvalidValue;
  return caught([&] {
    return launch_plan(p, q, 0, static_cast<hipStream_t>(stream), [](MxBf16Problem&, char*) { return hipSuccess; });
  });
}

}  // namespace w4
