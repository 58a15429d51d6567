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
// that a lane ends with both factors.
//
// Backward, the sum is over the rows of W, and its 4 bits lie along the other
// index.  ds_read_b64_tr_b8 gives a lane one byte, two neighbouring columns, of
// eight rows; each byte is rebuilt with its row's scale, and v_perm pairs rows:
// tile j takes columns 2 r + j.  The rows' scales, one byte each for 32 columns,
// are copied a step ahead of the weights and turned by the wave that copied them
// into 64 bytes a block of columns.
#include <atomic>
#include <type_traits>

#include "w4_launch.h"
#include "w4_lds_copy.h"
#include "w4_mx_act.h"
#include "w4_mx_device.h"

namespace w4 {
namespace {

typedef int i32x2 __attribute__((ext_vector_type(2)));

// A block of BM rows of x by BN columns (forward: weight rows): WM x WN waves,
// each with MT x 2 accumulators of 32 x 32.  NS steps of 64 in LDS: one read,
// the others arriving.
template <int BM_, int BN_, int WM_, int WN_, int NS_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int NW = WM * WN, THREADS = 64 * NW, MT = BM / WM / 32;
  static_assert(BN == 64 * WN && BM == 32 * WM * MT, "waves of 32 MT x 64");
  // 16-byte units of a step: rows of x, weights, scale bytes (a dword each)
  static constexpr int A = BM * 8, W = BN * 2, S = BN / 2;
  static constexpr int P = BN / 8;  // backward: the scales turned, 64 bytes for 32 columns
  static constexpr int IA = A / THREADS, IW = W / THREADS, IS = 4 * S / THREADS;  // copies of a wave
  static_assert(IA * THREADS == A && IW * THREADS == W && IS * THREADS == 4 * S, "the waves share the copies");
  static constexpr int COPIES = IA + IW + IS;
  static constexpr int LDS = NS * (A + W + S) + 2 * P;
  static_assert(LDS * 16 <= 160 * 1024, "the LDS of a CU");
};
using T0 = Tile<256, 256, 2, 4, 3>;
using T1 = Tile<128, 256, 2, 4, 3>;
using T2 = Tile<128, 128, 2, 2, 3>;
using T3 = Tile<64, 128, 2, 2, 3>;
using T4 = Tile<32, 128, 1, 2, 3>;
constexpr int kTiles = 5;

constexpr uint32_t kMaxSplits = 8;
// An offset past the resource of a tile's outputs (below 2^31 bytes), also with
// the offset of a row added.
constexpr uint32_t kStoreOOB = 0x80000000u;

struct GemmArgs {
  uint32_t tiles_m, tiles_n;
  uint32_t splits;  // parts of the sum, each to its own fp32 array at partial
  float* partial;
};

// What a copy past the end of the summed index reads.
__device__ const u32x4 kZeros[1] = {};

// 16-byte unit c of row `row` of x lies at unit c ^ swizzle_x(row) of its 128
// bytes in LDS: the reads of 16 rows take 16 different units of the banks' 256
// bytes.
__device__ __forceinline__ int swizzle_x(int row) { return (row >> 1) & 7; }
// The same for the weights, forward (rows of two units) ...
__device__ __forceinline__ int swizzle_w(int row) { return (row >> 3) & 1; }
// ... and backward (rows of U units, read in pairs of units, eight rows at a time).
template <int U>
__device__ __forceinline__ int swizzle_wt(int row) {
  return 2 * (row / (16 / U) % (U / 2));
}

template <int KIND, typename T>
__global__ __launch_bounds__(T::THREADS) void mx_bf16_gemm_kernel(MxBf16Problem P, GemmArgs G) {
  constexpr bool kBack = KIND == kMxBackward, kGate = KIND == kMxGated;
  constexpr int MT = T::MT, NS = T::NS;
  constexpr int U = T::BN / 32;                        // backward: units of a weight row in the tile
  constexpr int OUT = kGate ? T::BN / 2 : T::BN;       // outputs of a row in the tile
  extern __shared__ u32x4 lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % T::WM, wn = wave / T::WM;
  const int r = lane & 31, h = lane >> 5;

  // Blocks are dealt to the 8 XCDs round robin; each XCD takes a contiguous
  // range of the tiles, whose rows of x and w meet in its L2: eight tiles of
  // rows beside each other, then the next tile of columns.  (The grid is a
  // multiple of 8.)
  const uint32_t tiles = G.tiles_m * G.tiles_n, total = tiles * G.splits;
  const uint32_t range = (total + 7) / 8, L = blockIdx.x % 8 * range + blockIdx.x / 8;
  if (blockIdx.x / 8 >= range || L >= total) return;
  const uint32_t split = L / tiles, tile = L % tiles;
  const uint32_t band = tile / (8 * G.tiles_n), in = tile % (8 * G.tiles_n);
  const uint32_t height = G.tiles_m - 8 * band < 8 ? G.tiles_m - 8 * band : 8;
  const uint32_t mt = 8 * band + in % height, nt = in / height;

  const int64_t N = kBack ? P.k : P.n;                 // outputs of a row
  const int64_t m0 = (int64_t)mt * T::BM, n0 = (int64_t)nt * OUT;
  const int rows_m = (int)(P.m - m0 < T::BM ? P.m - m0 : T::BM);
  const int cols_n = (int)(N - n0 < OUT ? N - n0 : OUT);
  const uint32_t half = (uint32_t)(P.k >> 1), blocks = (uint32_t)(P.k >> 5);
  const uint32_t sum = (uint32_t)(kBack ? P.n : P.k);  // terms of an output
  const uint32_t steps = (sum + 63) / 64;
  const uint32_t t0 = (uint32_t)((uint64_t)split * steps / G.splits);
  const uint32_t t1 = (uint32_t)((uint64_t)(split + 1) * steps / G.splits);

  // where a step's slots start, in units: ring slot s
  auto slot_a = [](uint32_t s) { return s * T::A; };
  auto slot_w = [](uint32_t s) { return NS * T::A + s * T::W; };
  auto slot_s = [](uint32_t s) { return NS * (T::A + T::W) + s * T::S; };
  auto slot_p = [](uint32_t t) { return NS * (T::A + T::W + T::S) + (t & 1) * T::P; };
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
      const int c = (i >> 6) * 32 + (i & 31);
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
    return kBack ? u & 63 : u & 1;
  };
  const uint8_t* wp[T::IW];
#pragma unroll
  for (int i = 0; i < T::IW; ++i) {
    const int u = (wave * T::IW + i) * 64 + lane;
    if constexpr (kBack) {
      const uint32_t c = (uint32_t)(n0 >> 5) + ((u % U) ^ swizzle_wt<U>(u / U));
      wp[i] = P.w + (int64_t)(u / U) * half + 16 * (int64_t)(c < blocks ? c : blocks - 1);
    } else {
      wp[i] = P.w + weight_row(u >> 1) * half + 16 * at_w(lane, i);
    }
  }
  const uint8_t* sp[T::IS];
#pragma unroll
  for (int i = 0; i < T::IS; ++i) {
    const int u = (wave * T::IS + i) * 64 + lane;
    if constexpr (kBack) {
      const uint32_t c = (uint32_t)(n0 >> 5) + (u >> 6);
      sp[i] = P.w_scales + (int64_t)(u & 63) * blocks + (c < blocks ? c : blocks - 1);
    } else {
      sp[i] = P.w_scales + weight_row(u >> 1) * blocks + (u & 1);
    }
  }
  const int64_t step_w = kBack ? 64 * (int64_t)half : 32, step_s = kBack ? 64 * (int64_t)blocks : 2;
  auto inside = [&](uint32_t t, int at) {  // row or block `at` of step t lies before the end of the sum
    return kBack ? 64 * t + at < sum : 2 * t + at < blocks;
  };
  auto copy_scales = [&](uint32_t t, uint32_t s, auto WHOLE) {
#pragma unroll
    for (int i = 0; i < T::IS; ++i) {
      const uint8_t* from = sp[i] + t * step_s;
      if (!decltype(WHOLE)::value) from = inside(t, at_s(lane, i)) ? from : zeros;
      copy_byte(from, lds0 + 16 * slot_s(s) + (wave * T::IS + i) * 256);
    }
  };
  // step t to ring slot s (backward: with the scales of step t + 1, to the next slot);
  // WHOLE: all of it lies before the end of the sum
  auto copy = [&](uint32_t t, uint32_t s, auto WHOLE) {
    constexpr bool whole = decltype(WHOLE)::value;
    const uint32_t to_a = lds0 + 16 * (slot_a(s) + wave * T::IA * 64);
    const uint32_t to_w = lds0 + 16 * (slot_w(s) + wave * T::IW * 64);
    const uint8_t* const xs = uniform(xb + (uint64_t)t * 128);
#pragma unroll
    for (int i = 0; i < T::IA; ++i) {
      if constexpr (whole)
        copy16(xs, xv[i], to_a + i * 1024);
      else
        copy16(64 * t + 8 * unit_x(lane, i) < sum ? xs + xv[i] : zeros, to_a + i * 1024);
    }
#pragma unroll
    for (int i = 0; i < T::IW; ++i) {
      const uint8_t* from = wp[i] + t * step_w;
      if (!whole) from = inside(t, at_w(lane, i)) ? from : zeros;
      copy16(from, to_w + i * 1024);
    }
    if constexpr (kBack)
      copy_scales(t + 1, s + 1 == NS ? 0 : s + 1, WHOLE);
    else
      copy_scales(t, s, WHOLE);
  };
  // steps t that copy() may take as whole
  const uint32_t whole = kBack ? (sum >= 64 ? sum / 64 - 1 : 0) : sum / 64;

  // ---- backward: the scales of step t, in ring slot s, as bytes [block of columns][row]
  auto turn_scales = [&](uint32_t t, uint32_t s) {
    if (lane < 16 * T::IS) {
      const u32x4 v = lds[slot_s(s) + wave * T::IS * 16 + lane];
      reinterpret_cast<uint32_t*>(lds + slot_p(t))[wave * T::IS * 16 + lane] =
          v.x | v.y << 8 | v.z << 16 | v.w << 24;
    }
  };

  f32x16 acc[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;

  // ---- operands.  Of a step: forward the lane's block and scale of each tile,
  // backward the scales of its 32 rows.  Of a quarter: x, backward the weights.
  struct Step {
    u32x4 w[2];
    uint32_t s[2];
  };
  struct Quarter {
    u32x4 a[MT];
    i32x2 w;
  };
  struct Weights {
    u32x4 b[2];
  };
  auto read_step = [&](Step& v, uint32_t t, uint32_t s) {
    if constexpr (kBack) {
#pragma unroll
      for (int j = 0; j < 2; ++j) v.w[j] = lds[slot_p(t) + (2 * wn + (r >> 4)) * 4 + 2 * h + j];
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = wn * 64 + 32 * j + r;
        v.w[j] = lds[slot_w(s) + 2 * row + (h ^ swizzle_w(row))];
        v.s[j] = reinterpret_cast<const uint32_t*>(lds + slot_s(s))[2 * row + h];
      }
    }
  };
  auto read = [&](Quarter& v, uint32_t s, auto Q) {
    constexpr int q = decltype(Q)::value;
    if constexpr (kBack) {
      // of the sixteen lanes' addresses, two neighbours give a row's 16 bytes
      const int p = lane & 15, row = 32 * h + 8 * q + (p >> 1);
      const int unit = (2 * wn + ((lane >> 4) & 1)) ^ swizzle_wt<U>(row);
      const uint8_t* const at = reinterpret_cast<const uint8_t*>(lds + slot_w(s) + row * U + unit) + 8 * (p & 1);
      v.w = __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2*)at);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int row = wm * (32 * MT) + 32 * i + r;
      v.a[i] = lds[slot_a(s) + 8 * row + ((4 * h + q) ^ swizzle_x(row))];
    }
  };
  // a scale byte b at the conversion: its operand's exponent field (it reads no
  // other bit; 0 stands for 2^-127 there, 255 gives NaN)
  auto pair = [](uint32_t d, uint32_t scale, auto SEL) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(
                                            d, __builtin_bit_cast(float, scale), decltype(SEL)::value));
  };
  auto rebuild = [&](Weights& v, const Step& st, const Quarter& o, auto Q) {
    constexpr int q = decltype(Q)::value;
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    if constexpr (kBack) {
#pragma unroll
      for (int d = 0; d < 2; ++d) {  // four rows: scale bytes 8 q + 4 d .. + 3
        const uint32_t s = st.w[q >> 1][2 * (q & 1) + d], w = (uint32_t)o.w[d];
        const uint32_t p0 = pair(w, s << 23, I0{}), p1 = pair(w, s << 15, I1{});
        const uint32_t p2 = pair(w, s << 7, I2{}), p3 = pair(w, s >> 1, I3{});
        v.b[0][2 * d] = perm(p1, p0, 0x05040100u);
        v.b[0][2 * d + 1] = perm(p3, p2, 0x05040100u);
        v.b[1][2 * d] = perm(p1, p0, 0x07060302u);
        v.b[1][2 * d + 1] = perm(p3, p2, 0x07060302u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t d = st.w[j][q], s = st.s[j] << 23;
        v.b[j] = (u32x4){pair(d, s, I0{}), pair(d, s, I1{}), pair(d, s, I2{}), pair(d, s, I3{})};
      }
    }
  };
  auto multiply = [&](const Quarter& o, const Weights& v) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma32x32x16(o.a[i], v.b[j], acc[i][j]);
  };
  using Q0 = std::integral_constant<int, 0>;
  using Q1 = std::integral_constant<int, 1>;
  using Q2 = std::integral_constant<int, 2>;
  using Q3 = std::integral_constant<int, 3>;

  // ---- the loop.  A quarter's operands are read while the one before is
  // multiplied.  The barrier of a step comes before its last quarter: by then
  // every wave holds that in registers, so the step's slot can take the copies
  // of step t + NS, and the next step's first operands are read, while it is
  // multiplied.
  Step st;
  Quarter o0, o1;
  Weights b;
  uint32_t cur = t0 % NS;
  auto step = [&](uint32_t t, auto FAST) {
    constexpr bool fast = decltype(FAST)::value;  // step t + NS exists and is whole
    const uint32_t next = cur + 1 == NS ? 0 : cur + 1;
    if constexpr (kBack) turn_scales(t + 1, next);
    read(o1, cur, Q1{});
    rebuild(b, st, o0, Q0{});
    multiply(o0, b);
    __builtin_amdgcn_sched_barrier(0);
    read(o0, cur, Q2{});
    rebuild(b, st, o1, Q1{});
    multiply(o1, b);
    __builtin_amdgcn_sched_barrier(0);
    read(o1, cur, Q3{});
    rebuild(b, st, o0, Q2{});
    multiply(o0, b);
    rebuild(b, st, o1, Q3{});
    __builtin_amdgcn_sched_barrier(0);
    // the last operands (on every path here: after the branch the compiler's
    // own wait would be for the next step's reads too)
    __builtin_amdgcn_s_waitcnt(kWaitLds);
    if (fast || t + 1 < t1) {
      // the next step's copies: all but those of the NS - 2 steps after it
      if (fast || t + NS <= t1)
        __builtin_amdgcn_s_waitcnt(wait_vm((NS - 2) * T::COPIES));
      else
        __builtin_amdgcn_s_waitcnt(wait_vm(0));
      lds_barrier();
      if constexpr (fast) {
        copy(t + NS, cur, std::true_type{});
      } else {
        if (t + NS < t1) copy(t + NS, cur, std::false_type{});
      }
      read_step(st, t + 1, next);
      read(o0, next, Q0{});
    }
    __builtin_amdgcn_sched_barrier(0);
    multiply(o1, b);
    __builtin_amdgcn_sched_barrier(0);
    cur = next;
  };
  if constexpr (kBack) copy_scales(t0, cur, std::false_type{});
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    if (kBack && i == NS - 1) {
      // this step's copies bring scales to the slot of t0's, which are turned
      // first (behind a barrier: nothing else keeps their reads below the wait)
      if (t0 + NS - 1 <= t1)
        __builtin_amdgcn_s_waitcnt(wait_vm((NS - 1) * T::COPIES));
      else
        __builtin_amdgcn_s_waitcnt(wait_vm(0));
      lds_barrier();
      turn_scales(t0, cur);
      __builtin_amdgcn_s_waitcnt(kWaitLds);
      lds_barrier();
    }
    if (t0 + i < t1) copy(t0 + i, (t0 + i) % NS, std::false_type{});
  }
  if (t0 + NS <= t1)
    __builtin_amdgcn_s_waitcnt(wait_vm((NS - 1) * T::COPIES));
  else
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
  lds_barrier();
  read_step(st, t0, cur);
  read(o0, cur, Q0{});
  const uint32_t tw = whole < t1 ? whole : t1;  // steps t with t + NS < tw are fast
  uint32_t t = t0;
  for (; t + NS < tw; ++t) step(t, std::true_type{});
  for (; t < t1; ++t) step(t, std::false_type{});

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
  const bool part = G.partial != nullptr;
  if constexpr (kGate) {
    const int c = wn * 32 + r;
    auto gate = [&](int i, int q) -> float { return acc[i][0][q]; };
    auto up = [&](int i, int q) -> float { return acc[i][1][q]; };
    if (part) {
      float* const p = G.partial + (int64_t)split * P.m * 2 * N;
      put_f32(resource(p, 2 * N, n0, 4), (uint32_t)N * 8, c, gate);
      put_f32(resource(p, 2 * N, N + n0, 4), (uint32_t)N * 8, c, up);
      return;
    }
    const bool even = (N & 1) == 0;
    if (P.gu) {
      const bool pairs = even && (reinterpret_cast<uintptr_t>(P.gu) & 3) == 0;
      put_bf16(resource(P.gu, 2 * N, n0, 2), (uint32_t)N * 4, c, pairs, gate);
      put_bf16(resource(P.gu, 2 * N, N + n0, 2), (uint32_t)N * 4, c, pairs, up);
    }
    with_activation(P.act, [&](auto ACT) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][0][q] = activate<decltype(ACT)::value>(acc[i][0][q]) * acc[i][1][q];
    });
    if (P.y_bf16)
      put_bf16(resource(P.y, N, n0, 2), (uint32_t)N * 2, c, even && (reinterpret_cast<uintptr_t>(P.y) & 3) == 0, gate);
    else
      put_f32(resource(P.y, N, n0, 4), (uint32_t)N * 4, c, gate);
  } else {
    const int c = wn * 64 + 2 * r;
    void* const y = part ? G.partial + (int64_t)split * P.m * N : P.y;
    const int size = P.y_bf16 && !part ? 2 : 4;
    const __amdgpu_buffer_rsrc_t d = resource(y, N, n0, size);
    const uint32_t pitch = (uint32_t)N * size;
    if (size == 2 && (N & 1) == 0 && (reinterpret_cast<uintptr_t>(y) & 3) == 0) {
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

// y = the sum of the parts in order (gated: act(g) * u of the sums, and gu), one
// row's values of four columns a thread.
template <bool GATE>
__global__ __launch_bounds__(256) void mx_bf16_join_kernel(MxBf16Problem P, const float* __restrict__ partial,
                                                           uint32_t splits, int64_t N, int64_t count) {
  const int64_t first = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  const int64_t part = P.m * N * (GATE ? 2 : 1);
  for (int64_t j = first; j < first + 4 && j < count; ++j) {
    int64_t at = j;
    if constexpr (GATE) at = j + j / N * N;  // row j / N of 2 N
    float v = partial[at];
    for (uint32_t s = 1; s < splits; ++s) v += partial[s * part + at];
    if constexpr (GATE) {
      float u = partial[at + N];
      for (uint32_t s = 1; s < splits; ++s) u += partial[s * part + at + N];
      if (P.gu) {
        P.gu[at] = (uint16_t)f32_to_bf16_bits(v);
        P.gu[at + N] = (uint16_t)f32_to_bf16_bits(u);
      }
      with_activation(P.act, [&](auto ACT) { v = activate<decltype(ACT)::value>(v) * u; });
    }
    if (P.y_bf16)
      reinterpret_cast<uint16_t*>(P.y)[j] = (uint16_t)f32_to_bf16_bits(v);
    else
      reinterpret_cast<float*>(P.y)[j] = v;
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

struct Plan {
  int tile;
  uint32_t splits;
  int64_t tiles_m, tiles_n;
  int64_t blocks() const { return (tiles_m * tiles_n * splits + 7) / 8 * 8; }
};

int64_t outputs(const MxBf16Problem& p) { return p.kind == kMxBackward ? p.k : p.n; }
int64_t steps_of(const MxBf16Problem& p) { return ((p.kind == kMxBackward ? p.n : p.k) + 63) / 64; }

// Tile number t with the sum in s parts; tile < 0 where they do not fit the
// problem: a tile's rows of x and of outputs stay below 2^31 bytes, each part has
// a step, and a launch holds the blocks (of the join, too).
template <typename T>
Plan plan_on(const MxBf16Problem& p, int t, uint32_t s) {
  const int64_t N = outputs(p), wide = p.kind == kMxGated ? 2 * N : N;
  const int64_t cols = p.kind == kMxGated ? T::BN / 2 : T::BN;
  Plan q{t, s, (p.m + T::BM - 1) / T::BM, (N + cols - 1) / cols};
  constexpr int64_t kTileBytes = (INT64_C(1) << 31) - 1;
  if (4 * wide > kTileBytes / T::BM || 2 * p.x_pitch > kTileBytes / T::BM) q.tile = -1;
  if ((int64_t)s > steps_of(p)) q.tile = -1;
  if ((q.tiles_m * q.tiles_n * s + 7) * T::THREADS > kMaxLaunchThreads) q.tile = -1;
  if (s > 1 && (p.m * N + 1023) / 1024 * 256 > kMaxLaunchThreads) q.tile = -1;
  return q;
}

// What a tile costs: first + step us for its start and end and per 64 of the
// sum, by the blocks that share a CU.
struct Cost {
  float first, step;
  int per_cu;
};
constexpr Cost kCost[kTiles] = {{7.0f, 1.05f, 1}, {4.0f, 0.60f, 1}, {3.0f, 0.38f, 1}, {2.5f, 0.28f, 1}, {2.0f, 0.22f, 1}};

Plan make_plan(const MxBf16Problem& p) {
  const int64_t cus = device_cus();
  Plan best{4, 1, 0, 0};
  double least = 0;
  for (int t = 0; t < kTiles; ++t)
    for (uint32_t s = 1; s <= kMaxSplits; s *= 2) {
      const Plan q = with_tile(t, [&](auto X) { return plan_on<decltype(X)>(p, t, s); });
      if (q.tile < 0) continue;
      const int64_t n = q.tiles_m * q.tiles_n * s;
      const double k = (double)((steps_of(p) + s - 1) / s);
      double us = (double)((n + cus - 1) / cus) * (kCost[t].first + kCost[t].step * k);
      if (s > 1) us += 3.0 + (double)s * p.m * outputs(p) * 8 / 4e6;
      if (best.tiles_m == 0 || us < least) {
        least = us;
        best = q;
      }
    }
  if (best.tiles_m == 0) best.tiles_m = best.tiles_n = INT64_C(1) << 31;  // too many tiles of every size
  return best;
}

template <int KIND, typename T>
hipError_t launch_tile(const MxBf16Problem& p, const GemmArgs& g, uint32_t blocks, hipStream_t stream) {
  constexpr int lds = T::LDS * 16;
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

hipError_t launch_plan(const MxBf16Problem& p, const Plan& q, float* partial, hipStream_t stream) {
  const GemmArgs g{(uint32_t)q.tiles_m, (uint32_t)q.tiles_n, q.splits, q.splits > 1 ? partial : nullptr};
  const hipError_t e = with_tile(q.tile, [&](auto X) {
    using T = decltype(X);
    const uint32_t blocks = (uint32_t)q.blocks();
    if (p.kind == kMxGated) return launch_tile<kMxGated, T>(p, g, blocks, stream);
    if (p.kind == kMxBackward) return launch_tile<kMxBackward, T>(p, g, blocks, stream);
    return launch_tile<kMxForward, T>(p, g, blocks, stream);
  });
  if (e != hipSuccess || q.splits == 1) return e;
  const int64_t N = outputs(p), count = p.m * N;
  const dim3 grid((uint32_t)((count + 1023) / 1024));
  if (p.kind == kMxGated)
    mx_bf16_join_kernel<true><<<grid, dim3(256), 0, stream>>>(p, partial, q.splits, N, count);
  else
    mx_bf16_join_kernel<false><<<grid, dim3(256), 0, stream>>>(p, partial, q.splits, N, count);
  return hipGetLastError();
}

size_t partial_bytes(const MxBf16Problem& p, const Plan& q) {
  return q.splits == 1 ? 0 : (size_t)q.splits * p.m * outputs(p) * (p.kind == kMxGated ? 2 : 1) * sizeof(float);
}

}  // namespace

bool mx_bf16_fits(const MxBf16Problem& p) { return make_plan(p).blocks() <= 0x7FFFFFFF; }

size_t mx_bf16_workspace_bytes(const MxBf16Problem& p) { return partial_bytes(p, make_plan(p)); }

hipError_t launch_mx_bf16_on(const MxBf16Problem& p, char* ws, hipStream_t stream) {
  return launch_plan(p, make_plan(p), reinterpret_cast<float*>(ws), stream);
}

}  // namespace w4
