// MX products for many rows (gfx950): y = x w^T with both operands in
// microscaled form, for one weight and for many weights whose rows of x are
// grouped by expert.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes the stored elements and scale bytes as
// they are: nothing is rebuilt, and the sums are the matrix core's fp32.
//
// Bound by the waves' waits for each other: a step of 256 x 256 x 256 (MXFP4) is
// 2048 cycles of matrix instructions on each SIMD and takes 2.0 us, about 4100
// cycles at the 1.9 to 2.1 GHz that the card's power leaves under this load.
// Counters of 4096 x 11008 x 4096: matrix cores busy 42% of the cycles, LDS 20%,
// and the eight waves of a CU, which meet at one barrier a step, 27% of their time
// in waits (1.4% for the LDS to take an instruction).  In the 64 x 128 tiles a
// wave has one 32 x 32 accumulator, and a step's LDS reads, three KB a matrix
// instruction, hold it too.  The copies are no bound: global to LDS reaches 64
// bytes a cycle and CU from L2, the steps need 20 to 30.
//
// Measured (HIP graph replays, three sets of operands in turn, by machine): 4096
// x 11008 x 4096, MXFP4 to fp32, 124 to 127 us (2.9 to 3.0 PFLOP/s), MXFP8 to
// bf16 181 us (2.0); 256 x 8192 x 8192, MXFP8 to bf16, 22 to 23 us (1.5); 8192
// rows over 32 experts of 4096 x 2048, MXFP8, 106 to 113 us (1.2 to 1.3); 3001
// rows over 7 experts of 2048 x 5632, MXFP4, 32 to 35 us (2.0 to 2.1).  A k that is
// no multiple of 128 has no steps without conditions: 4096 x 2880 x 2880, MXFP8,
// 59 us (1.1), at 2816 46 us (1.4).  Short k is held
// by a tile's 4 to 8 us of start and end (the walk of the offsets, the first
// copies, the stores, the next block's launch).
//
// Measured and slower or the same: loads to L2 ahead of the copies; copies
// issued between the products; blocks that stay and copy the next tile's first
// steps before they store; 128 x 128 of the tile a wave (one wave a SIMD; the
// accumulators move between the two register files); a step's quarters split
// over four waves that each hold the whole tile.
#include <atomic>
#include <type_traits>

#include "w4_launch.h"
#include "w4_lds_copy.h"
#include "w4_mx_device.h"
#include "w4_mx_group.h"

namespace w4 {
namespace {

// A block of BM rows of x by BN weight rows: WM x WN waves, each with its part
// of the tile as 32 x 32 accumulators.  A step is 256 of k: BM rows of 256 (fp8)
// or 128 (fp4) bytes and BN rows of 128 bytes, copied straight to LDS in whole
// lines, NS - 1 steps ahead.
template <int AF, int BM_, int BN_, int WM_, int WN_, int NS_>
struct Tile {
  static constexpr int NS = NS_;           // steps in LDS: one read, NS - 1 arriving
  static constexpr int CS = NS == 4 ? 4 : 2;  // scale slots, at least NS / 2 + 1
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int NW = WM * WN, THREADS = 64 * NW;
  static constexpr int MT = BM / WM / 32, NT = BN / WN / 32;
  static constexpr int XU = AF == kMxFp8 ? 16 : 8;  // 16-byte units of a row of x in a step
  static constexpr int A = BM * XU, B = BN * 8;     // units of a step's slots
  static constexpr int S = BM + BN;                 // units of a scale slot: 16 bytes a row, two steps
  static constexpr int LDS = NS * (A + B) + CS * S;
  static_assert(LDS * 16 <= 160 * 1024 - 64, "the LDS of a CU");
  static constexpr int PER_CU = LDS * 16 <= 80 * 1024 ? 2 : 1;  // blocks of a CU
  static constexpr int IA = A / THREADS, IB = B / THREADS;     // copies of a wave per step
  static constexpr int IS = (S + THREADS - 1) / THREADS;       // scale rows of a thread
  // quarters of a step whose operands are read ahead: two, where the registers
  // hold them beside the accumulators
  static constexpr int AHEAD = MT * NT < 8 ? 2 : 1;
  static_assert(IA * THREADS == A && IB * THREADS == B, "the waves share the copies");
};

// Where unit c of a row lies in its LDS row: XOR-swizzled, so that the units c
// of 16 consecutive rows lie on different banks (64 of 4 bytes).
template <int UNITS>
__device__ __forceinline__ int swizzle(int row, int c) {
  return c ^ (UNITS == 16 ? row & 15 : (row >> 1) & 7);
}

constexpr uint32_t kMaxSplits = 8;

// An offset past the resource of a tile's y (below 2^31 bytes), also with the
// offset of a row added.
constexpr uint32_t kStoreOOB = 0x80000000u;

struct GemmArgs {
  uint32_t tiles_m, tiles_n;  // tiles_m: most tiles of rows, grouped
  uint32_t splits;            // parts of k, each to its own fp32 y at partial
  float* partial;
};

template <int AF, typename T, bool GROUPED>
__global__ __launch_bounds__(T::THREADS) __attribute__((amdgpu_waves_per_eu(T::PER_CU * T::NW / 4, T::PER_CU * T::NW / 4))) void mx_gemm_kernel(
    MxProblem P, GemmArgs G) {
  extern __shared__ u32x4 lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % T::WM, wn = wave / T::WM;
  const int r = lane & 31, h = lane >> 5;

  // Blocks are dealt to the 8 XCDs round robin; each XCD takes a contiguous
  // range of the tiles, whose rows of x and w meet in its L2.  Grouped, the
  // launch has a block for every tile that the groups could make; the tiles
  // that they do make are dealt out.
  // (The grid is a multiple of 8.)
  uint32_t total = G.tiles_m * G.tiles_n * G.splits;
  GroupScan<T::BM> scan(P.offsets, P.experts, (int32_t)P.m);
  if constexpr (GROUPED) {
    scan.read();
    total = scan.count() * G.tiles_n;
  }
  const uint32_t range = (total + 7) / 8, L = blockIdx.x % 8 * range + blockIdx.x / 8;
  if (blockIdx.x / 8 >= range || L >= total) return;
  uint32_t mt, nt, split = 0;
  GroupTile E{0, 0, (int32_t)P.m};
  if constexpr (GROUPED) {
    nt = L % G.tiles_n;
    E = scan.find(L / G.tiles_n);
    if (E.e < 0) return;
  } else {
    // eight tiles of rows beside each other, then the next tile of columns
    const uint32_t tiles = G.tiles_m * G.tiles_n, t = L % tiles;
    split = L / tiles;
    const uint32_t band = t / (8 * G.tiles_n), in = t % (8 * G.tiles_n);
    const uint32_t height = G.tiles_m - 8 * band < 8 ? G.tiles_m - 8 * band : 8;
    mt = 8 * band + in % height;
    nt = in / height;
    E.lo = (int32_t)(mt * T::BM);
  }
  const int64_t N = P.n, K = P.k, n0 = (int64_t)nt * T::BN;
  const int rows_n = (int)(N - n0 < T::BN ? N - n0 : T::BN);
  const int rows_m = E.hi - E.lo < T::BM ? E.hi - E.lo : T::BM;
  const bool none = GROUPED && E.e == P.experts;  // rows of no expert

  f32x16 acc[T::MT][T::NT];
#pragma unroll
  for (int i = 0; i < T::MT; ++i)
#pragma unroll
    for (int j = 0; j < T::NT; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
  // rows that are stored as zeros, by their index or for want of an expert
  __shared__ uint64_t dead[T::BM / 64];
  if (GROUPED && wave < T::BM / 64) {
    bool d = none;
    if (P.row_index && !none) {
      const int64_t src = P.row_index[E.lo + (tid < rows_m ? tid : rows_m - 1)];
      d = src < 0 || src >= P.tokens;
    }
    const uint64_t mask = __ballot(d);
    if (lane == 0) dead[wave] = mask;
  }
  if (GROUPED && none) __syncthreads();

  if (!none) {
    const uint32_t half = (uint32_t)(K >> 1), blocks = (uint32_t)(K >> 5);
    const uint32_t x_bytes = AF == kMxFp8 ? (uint32_t)K : half;
    const uint32_t steps = (blocks + 7) / 8;
    const uint32_t t0 = (uint32_t)((uint64_t)split * steps / G.splits) & ~1u;
    const uint32_t t1 = split + 1 == G.splits ? steps : (uint32_t)((uint64_t)(split + 1) * steps / G.splits) & ~1u;
    // where a step's slots start, in units: ring of x and w by s = t % NS
    auto slot_a = [](uint32_t s) { return s * T::A; };
    auto slot_b = [](uint32_t s) { return T::NS * T::A + s * T::B; };
    auto slot_s = [](uint32_t t) { return T::NS * (T::A + T::B) + (t >> 1) % T::CS * T::S; };
    const uint32_t lds0 = lds_address(lds);

    // rows of the tile past the last one repeat it and are never stored
    auto row_of_x = [&](int i) {
      const int64_t row = E.lo + (i < rows_m ? i : rows_m - 1);
      if (!(GROUPED && P.row_index)) return row;
      const int64_t src = P.row_index[row];
      return src < 0 || src >= P.tokens ? 0 : src;  // stored as zeros
    };
    const int64_t w0 = (int64_t)E.e * N + n0;
    const uint8_t* const wb = uniform(P.w + w0 * half);
    auto row_of_w = [&](int i) { return (uint32_t)(i < rows_n ? i : rows_n - 1); };

    // A copy moves 64 units of 16 bytes to consecutive LDS; within a row the
    // units are XOR-swizzled by the row, on the source's side, so that the
    // operand reads (eight rows, one unit each) are free of bank conflicts.
    // Past the end of k a row's last unit is copied again: its scales are 0
    // there on both sides, and 2^-254 of anything finite adds nothing (a NaN
    // element is its row's already).
    // 16-byte unit `lane` of a wave's copy i of x (w) in its row
    auto unit_x = [&](int l, int i) {
      const int u = (wave * T::IA + i) * 64 + l;
      return 16u * swizzle<T::XU>(u / T::XU, u % T::XU);
    };
    auto unit_w = [&](int l, int i) {
      const int u = (wave * T::IB + i) * 64 + l;
      return 16u * swizzle<8>(u / 8, u % 8);
    };
    const uint8_t* xp[T::IA];
#pragma unroll
    for (int i = 0; i < T::IA; ++i)
      xp[i] = P.x + row_of_x(((wave * T::IA + i) * 64 + lane) / T::XU) * x_bytes + unit_x(lane, i);
    uint32_t wp[T::IB];  // (a block's rows: below 2^30 bytes)
#pragma unroll
    for (int i = 0; i < T::IB; ++i)
      wp[i] = row_of_w(((wave * T::IB + i) * 64 + lane) / 8) * half + unit_w(lane, i);
    // this wave's copies of step t, to ring slot s; WHOLE: all of it lies before
    // the end of k
    constexpr int C = T::IA + T::IB;
    auto copy = [&](uint32_t t, uint32_t s, auto WHOLE) {
      const uint32_t to_a = lds0 + 16 * (slot_a(s) + wave * T::IA * 64);
      const uint32_t to_b = lds0 + 16 * (slot_b(s) + wave * T::IB * 64);
      const uint32_t ox = t * (16 * T::XU), ow = t * 128;
      int l = lane;
      if (!decltype(WHOLE)::value) asm volatile("" : "+v"(l));  // (not worth registers from here on)
#pragma unroll
      for (int i = 0; i < T::IA; ++i) {
        const uint32_t u = unit_x(l, i);
        // (signed: a row can be shorter than the unit's offset)
        const int32_t o = (int32_t)(decltype(WHOLE)::value || u + ox < x_bytes ? ox : x_bytes - 16 - u);
        copy16(xp[i] + o, to_a + i * 1024);
      }
#pragma unroll
      for (int i = 0; i < T::IB; ++i) {
        const uint32_t u = unit_w(l, i);
        if constexpr (decltype(WHOLE)::value)
          copy16(uniform(wb + ow), wp[i], to_b + i * 1024);
        else
          copy16(wb, wp[i] + (u + ow < half ? ow : half - 16 - u), to_b + i * 1024);
      }
    };
    // Scales: 16 bytes (two steps) of a row at a time, a lane a row, copied like
    // the elements where they lie on whole dwords; otherwise, and at the end of
    // k, through registers, with zeros past the end.
    const uint8_t* sp[T::IS];
#pragma unroll
    for (int i = 0; i < T::IS; ++i) {
      const int row = i * T::THREADS + tid;
      sp[i] = row < T::BM ? P.x_scales + row_of_x(row) * blocks
                          : P.w_scales + (w0 + row_of_w(row - T::BM)) * blocks;
    }
    const bool dwords = (blocks & 3) == 0;
    auto copied = [&](uint32_t t) { return dwords && 8 * t + 16 <= blocks; };
    auto copy_scales = [&](uint32_t t) {
#pragma unroll
      for (int i = 0; i < T::IS; ++i)
        if (i * T::THREADS + wave * 64 < T::S)
          copy16(sp[i] + 8 * t, lds0 + 16 * (slot_s(t) + i * T::THREADS + wave * 64));
    };
    // (the last 16 bytes of a row, where fewer are left, and shifted when put)
    u32x4 sv[T::IS];
    auto load_scales = [&](uint32_t t) {
      const uint32_t c = 8 * t;
#pragma unroll
      for (int i = 0; i < T::IS; ++i) {
        if (blocks >= 16) {
          __builtin_memcpy(&sv[i], sp[i] + (c + 16 <= blocks ? c : blocks - 16), 16);
        } else {
          uint32_t d[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const uint32_t e = sp[i][c + q < blocks ? c + q : c];
            d[q / 4] |= (c + q < blocks ? e : 0u) << (8 * (q % 4));
          }
          sv[i] = (u32x4){d[0], d[1], d[2], d[3]};
        }
      }
    };
    auto put_scales = [&](uint32_t t) {
      const uint32_t over = blocks >= 16 && 8 * t + 16 > blocks ? 8 * t + 16 - blocks : 0;  // bytes, the same in every lane
#pragma unroll
      for (int i = 0; i < T::IS; ++i) {
        u32x4 v = sv[i];
        if (over) {
          if (over & 8) v = (u32x4){v.z, v.w, 0u, 0u};
          if (over & 4) v = (u32x4){v.y, v.z, v.w, 0u};
          const uint32_t n = over & 3;
          v = (u32x4){__builtin_amdgcn_alignbyte(v.y, v.x, n), __builtin_amdgcn_alignbyte(v.z, v.y, n),
                      __builtin_amdgcn_alignbyte(v.w, v.z, n), __builtin_amdgcn_alignbyte(0u, v.w, n)};
        }
        if (i * T::THREADS + wave * 64 < T::S) lds[slot_s(t) + i * T::THREADS + tid] = v;
      }
    };

    // operands of 64 of k (a quarter of a step), and a step's scales
    struct Operands {
      u32x4 a[T::MT][AF == kMxFp8 ? 2 : 1], b[T::NT];
    };
    Operands o[2 * T::AHEAD];
    u32x2 sa[T::MT], sb[T::NT], na[T::MT], nb[T::NT];
    auto read = [&](Operands& v, uint32_t s, auto Q) {
      constexpr int q = decltype(Q)::value;
      const u32x4* const a = lds + slot_a(s);
      const u32x4* const w = lds + slot_b(s);
#pragma unroll
      for (int j = 0; j < T::NT; ++j) {
        const int row = wn * (32 * T::NT) + 32 * j + r;
        v.b[j] = w[row * 8 + swizzle<8>(row, 2 * q + h)];
      }
#pragma unroll
      for (int i = 0; i < T::MT; ++i) {
        const int row = wm * (32 * T::MT) + 32 * i + r;
        if constexpr (AF == kMxFp8) {
          v.a[i][0] = a[row * 16 + swizzle<16>(row, 4 * q + h)];
          v.a[i][1] = a[row * 16 + swizzle<16>(row, 4 * q + 2 + h)];
        } else {
          v.a[i][0] = a[row * 8 + swizzle<8>(row, 2 * q + h)];
        }
      }
    };
    // the scale bytes of a row's eight blocks; lane half h needs blocks 2 q + h
    auto read_scales = [&](uint32_t t) {
      const u32x2* const s = reinterpret_cast<const u32x2*>(lds + slot_s(t)) + (t & 1);
#pragma unroll
      for (int i = 0; i < T::MT; ++i) na[i] = s[2 * (wm * (32 * T::MT) + 32 * i + r)];
#pragma unroll
      for (int j = 0; j < T::NT; ++j) nb[j] = s[2 * (T::BM + wn * (32 * T::NT) + 32 * j + r)];
    };
    auto shift_scales = [&]() {
#pragma unroll
      for (int i = 0; i < T::MT; ++i) sa[i] = na[i] >> (8u * h);
#pragma unroll
      for (int j = 0; j < T::NT; ++j) sb[j] = nb[j] >> (8u * h);
    };
    auto multiply = [&](const Operands& v, auto Q) {
      constexpr int q = decltype(Q)::value, op = 2 * (q & 1);
#pragma unroll
      for (int i = 0; i < T::MT; ++i)
#pragma unroll
        for (int j = 0; j < T::NT; ++j) {
          acc[i][j] = mx_mfma32<AF, op, op>(mx_operand<AF>(v.a[i][0], v.a[i][AF == kMxFp8 ? 1 : 0]),
                                            mx_operand<kMxFp4>(v.b[j], v.b[j]), acc[i][j], sa[i][q >> 1], sb[j][q >> 1]);
          // keeps the product here (it would sink past the branches below, and
          // every quarter's operands would have to live till then)
          asm volatile("" : "+v"(acc[i][j]));
        }
    };
    // A quarter's products and the next one's reads by turns: the reads of eight
    // waves issued together would fill the LDS queue, and the products would
    // wait behind them.
    auto interleave = [&]() {
      constexpr int reads = T::AHEAD * (T::NT + T::MT * (AF == kMxFp8 ? 2 : 1)), products = T::AHEAD * T::MT * T::NT;
#pragma unroll
      for (int n = 0; n < products; ++n) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
        for (int m = n * reads / products; m < (n + 1) * reads / products; ++m)
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
    };
    using Q0 = std::integral_constant<int, 0>;
    using Q1 = std::integral_constant<int, 1>;
    using Q2 = std::integral_constant<int, 2>;
    using Q3 = std::integral_constant<int, 3>;

    // A quarter's operands (AHEAD = 2: a half's) are read while the one before
    // is multiplied.  The barrier of a step comes before its last quarter
    // (half): by then every wave holds that in registers, so the step's slot can
    // take the copies of step t + NS, and the next step's first operands are
    // read, while it is multiplied.
    // FAST: step t + NS and the scales of steps t + NS and t + 3 lie whole before
    // the end of k, or k is a multiple of 512, and so all are copied: no conditions, and only x's addresses to add up.
    uint32_t cur = t0 % T::NS;
    auto step = [&](uint32_t t, auto FAST) {
      constexpr bool fast = decltype(FAST)::value;
      if constexpr (T::AHEAD == 2) {
        read(o[2], cur, Q2{});
        read(o[3], cur, Q3{});
        multiply(o[0], Q0{});
        multiply(o[1], Q1{});
        interleave();
      } else {
        read(o[1], cur, Q1{});
        multiply(o[0], Q0{});
        interleave();
        __builtin_amdgcn_sched_barrier(0);
        read(o[0], cur, Q2{});
        multiply(o[1], Q1{});
        interleave();
        __builtin_amdgcn_sched_barrier(0);
        read(o[1], cur, Q3{});
        multiply(o[0], Q2{});
        interleave();
      }
      __builtin_amdgcn_sched_barrier(0);
      // the last operands (on every path here: after the branch the compiler's
      // own wait would be for the next step's reads too)
      __builtin_amdgcn_s_waitcnt(kWaitLds);
      const uint32_t next = cur + 1 == T::NS ? 0 : cur + 1;
      if (fast || t + 1 < t1) {
        // the next step's copies: all but those of the NS - 2 steps after it
        if (fast || t + T::NS <= t1)
          __builtin_amdgcn_s_waitcnt(wait_vm((T::NS - 2) * C));
        else
          __builtin_amdgcn_s_waitcnt(wait_vm(0));
        if (!fast && (t & 1) == 1 && !copied(t + 1)) put_scales(t + 1);
        lds_barrier();
        if (fast || t + T::NS < t1) {
          if (((t + T::NS) & 1) == 0 && (fast || copied(t + T::NS))) copy_scales(t + T::NS);
          if (fast || (T::AHEAD == 1 && 8 * (t + T::NS) + 8 <= blocks))
            copy(t + T::NS, cur, std::true_type{});
          else
            copy(t + T::NS, cur, std::false_type{});
        }
        if (!fast && (t & 1) == 1 && t + 3 < t1 && !copied(t + 3)) load_scales(t + 3);
        read_scales(t + 1);
        read(o[0], next, Q0{});
        if constexpr (T::AHEAD == 2) read(o[1], next, Q1{});
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (T::AHEAD == 2) {
        multiply(o[2], Q2{});
        multiply(o[3], Q3{});
      } else {
        multiply(o[1], Q3{});
      }
      __builtin_amdgcn_sched_barrier(0);
      shift_scales();
      cur = next;
    };
#pragma unroll
    for (int i = 0; i < T::NS; ++i) {
      if (i % 2 == 0 && t0 + i < t1 && copied(t0 + i)) copy_scales(t0 + i);
      if (t0 + i < t1) copy(t0 + i, (t0 + i) % T::NS, std::false_type{});
    }
    if (!copied(t0)) {
      load_scales(t0);
      put_scales(t0);
    }
    if (t0 + T::NS <= t1)
      __builtin_amdgcn_s_waitcnt(wait_vm((T::NS - 1) * C));
    else
      __builtin_amdgcn_s_waitcnt(wait_vm(0));
    lds_barrier();
    if (t0 + 2 < t1 && !copied(t0 + 2)) load_scales(t0 + 2);
    read_scales(t0);
    read(o[0], cur, Q0{});
    if constexpr (T::AHEAD == 2) read(o[1], cur, Q1{});
    shift_scales();
    // steps t with t + NS < t1 and, unless every pair of steps is whole,
    // 8 (t + max(NS, 3)) + 16 <= blocks
    constexpr uint32_t reach = T::NS > 3 ? T::NS : 3;
    const uint32_t inside = blocks % 16 == 0 ? steps
                            : dwords && blocks >= 8 * reach + 16 ? (blocks - 16) / 8 - reach + 1 : 0;
    const uint32_t tf = t1 < T::NS ? 0 : t1 - T::NS < inside ? t1 - T::NS : inside;
    uint32_t t = t0;
    if constexpr (T::AHEAD == 2)  // (else a second loop's addresses would not fit the registers)
      for (; t < tf; ++t) step(t, std::true_type{});
    for (; t < t1; ++t) step(t, std::false_type{});
  }

  if (GROUPED && (none || P.row_index)) {
#pragma unroll
    for (int i = 0; i < T::MT; ++i)
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int row = wm * (32 * T::MT) + 32 * i + 8 * (q >> 2) + 4 * h + (q & 3);
        if (dead[row >> 6] >> (row & 63) & 1) {
#pragma unroll
          for (int j = 0; j < T::NT; ++j) acc[i][j][q] = 0.f;
        }
      }
  }

  // D[row of x][weight row]: lane half h, register q hold row 8 (q / 4) + 4 h +
  // q % 4 of column r.  Stores go through a resource that ends with the last
  // row; columns past the last take an offset past it.
  const bool part = G.partial != nullptr;
  const int size = P.y_bf16 && !part ? 2 : 4;
  uint8_t* const y0 = const_cast<uint8_t*>(uniform(
      (part ? reinterpret_cast<uint8_t*>(G.partial + (int64_t)split * P.m * N) : reinterpret_cast<uint8_t*>(P.y)) +
      ((int64_t)E.lo * N + n0) * size));
  const uint32_t pitch = (uint32_t)N * size;
  const __amdgpu_buffer_rsrc_t yr = mx_rsrc(y0, (uint32_t)(rows_m - 1) * pitch + (uint32_t)rows_n * size);
  const int row0 = wm * (32 * T::MT), col0 = wn * (32 * T::NT) + r;
  if (size == 4) {
    uint32_t at[T::NT];
#pragma unroll
    for (int j = 0; j < T::NT; ++j)
      at[j] = col0 + 32 * j < rows_n ? (uint32_t)(row0 + 4 * h) * pitch + 4u * (col0 + 32 * j) : kStoreOOB;
#pragma unroll
    for (int i = 0; i < T::MT; ++i)
#pragma unroll
      for (int q = 0; q < 16; ++q)
#pragma unroll
        for (int j = 0; j < T::NT; ++j)
          __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, (float)acc[i][j][q]), yr,
                                                at[j] + (32 * i + 8 * (q >> 2) + (q & 3)) * pitch, 0, 0);
  } else if ((N & 1) == 0 && (reinterpret_cast<uintptr_t>(P.y) & 3) == 0) {
    // pairs of columns: of rows q and q + 1, a lane and its neighbour keep one
    // each and swap the other
    const int odd = lane & 1;
    uint32_t at[T::NT];
#pragma unroll
    for (int j = 0; j < T::NT; ++j)
      at[j] = col0 + 32 * j < rows_n ? (uint32_t)(row0 + 4 * h + odd) * pitch + 2u * ((col0 & ~1) + 32 * j) : kStoreOOB;
#pragma unroll
    for (int i = 0; i < T::MT; ++i)
#pragma unroll
      for (int q = 0; q < 16; q += 2)
#pragma unroll
        for (int j = 0; j < T::NT; ++j) {
          const float e = acc[i][j][q], f = acc[i][j][q + 1];
          // quad_perm [1,0,3,2]
          const float got = __builtin_bit_cast(
              float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, odd ? e : f), 0xB1, 0xF, 0xF, true));
          __builtin_amdgcn_raw_buffer_store_b32(cvt_pk_bf16(odd ? got : e, odd ? f : got), yr,
                                                at[j] + (32 * i + 8 * (q >> 2) + (q & 3)) * pitch, 0, 0);
        }
  } else {
    uint32_t at[T::NT];
#pragma unroll
    for (int j = 0; j < T::NT; ++j)
      at[j] = col0 + 32 * j < rows_n ? (uint32_t)(row0 + 4 * h) * pitch + 2u * (col0 + 32 * j) : kStoreOOB;
#pragma unroll
    for (int i = 0; i < T::MT; ++i)
#pragma unroll
      for (int q = 0; q < 16; ++q)
#pragma unroll
        for (int j = 0; j < T::NT; ++j)
          __builtin_amdgcn_raw_buffer_store_b16((uint16_t)f32_to_bf16_bits(acc[i][j][q]), yr,
                                                at[j] + (32 * i + 8 * (q >> 2) + (q & 3)) * pitch, 0, 0);
  }
}

// y = the sum of the splits' y in split order, four values a thread (the last
// ones singly).
__global__ __launch_bounds__(256) void mx_join_kernel(const float* __restrict__ partial, uint32_t splits,
                                                      int64_t count, void* y, int y_bf16) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= count) return;
  if (i + 4 <= count && (count & 3) == 0) {
    f32x4 p[kMaxSplits];
#pragma unroll
    for (uint32_t s = 0; s < kMaxSplits; ++s)
      if (s < splits) p[s] = *reinterpret_cast<const f32x4*>(partial + s * count + i);
    f32x4 v = p[0];
#pragma unroll
    for (uint32_t s = 1; s < kMaxSplits; ++s)
      if (s < splits) v += p[s];
    mx_store4(y, y_bf16, i, 0, 4, v);
    return;
  }
  for (int64_t j = i; j < i + 4 && j < count; ++j) {
    float v = partial[j];
    for (uint32_t s = 1; s < splits; ++s) v += partial[s * count + j];
    if (y_bf16)
      reinterpret_cast<uint16_t*>(y)[j] = (uint16_t)f32_to_bf16_bits(v);
    else
      reinterpret_cast<float*>(y)[j] = v;
  }
}

int device_cus() {
  int dev = 0, cus = 256;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    cus = 256;
  return cus;
}

// Tiles, largest first, with what they cost: a block alone on its CU takes
// first + step us for its start and end and per 256 of k, two blocks that
// share one (where they fit) first2 + step2.  Measured: 2048 to 4096 rows and
// columns that give one block (or two) a CU, k = 2048 and 8192.
struct Cost {
  float first, step, first2, step2;
};
template <int AF>
struct Tiles;
template <>
struct Tiles<kMxFp8> {
  using T0 = Tile<kMxFp8, 128, 256, 2, 4, 2>;
  using T1 = Tile<kMxFp8, 128, 128, 2, 4, 3>;
  using T2 = Tile<kMxFp8, 64, 256, 1, 8, 3>;
  using T3 = Tile<kMxFp8, 64, 128, 2, 4, 4>;
  using T4 = Tile<kMxFp8, 64, 128, 2, 4, 2>;
  static constexpr Cost cost[5] = {
      {5.6f, 1.58f, 0, 0}, {3.0f, 1.01f, 0, 0}, {2.2f, 1.06f, 0, 0}, {1.9f, 0.60f, 0, 0}, {1.2f, 0.69f, 4.0f, 1.05f}};
};
template <>
struct Tiles<kMxFp4> {
  using T0 = Tile<kMxFp4, 256, 256, 2, 4, 2>;
  using T1 = Tile<kMxFp4, 128, 256, 2, 4, 3>;
  using T2 = Tile<kMxFp4, 128, 128, 2, 4, 4>;
  using T3 = Tile<kMxFp4, 64, 256, 1, 8, 3>;
  using T4 = Tile<kMxFp4, 64, 128, 2, 4, 3>;
  static constexpr Cost cost[5] = {
      {6.7f, 2.04f, 0, 0}, {5.8f, 1.10f, 0, 0}, {3.0f, 0.70f, 0, 0}, {2.5f, 0.76f, 0, 0}, {1.0f, 0.46f, 3.3f, 0.80f}};
};

template <int AF, typename F>
auto with_tile(int tile, F&& f) {
  using S = Tiles<AF>;
  switch (tile) {
    case 0: return f(typename S::T0{});
    case 1: return f(typename S::T1{});
    case 2: return f(typename S::T2{});
    case 3: return f(typename S::T3{});
    default: return f(typename S::T4{});
  }
}

struct Plan {
  int tile;
  uint32_t splits;
  int64_t tiles_m, tiles_n;  // tiles_m: most tiles of rows, grouped
  int64_t blocks() const { return (tiles_m * tiles_n * splits + 7) / 8 * 8; }
};

// Groups that have rows, the rows of no expert among them, at most.
int64_t most_groups(const MxProblem& p) { return p.m < p.experts + 1 ? p.m : p.experts + 1; }

// Tile number t with k in s parts; tile < 0 where they do not fit the problem:
// a tile of y stays below 2^31 bytes, grouped products do not split k, each part
// has two steps of k, and a launch holds the blocks.
template <typename T>
Plan plan_on(const MxProblem& p, int t, uint32_t s) {
  Plan q{t, s, (p.m + T::BM - 1) / T::BM, (p.n + T::BN - 1) / T::BN};
  if (p.offsets) q.tiles_m = most_groups(p) + (p.m - most_groups(p)) / T::BM;
  if (p.n > ((INT64_C(1) << 31) - 1) / 4 / T::BM) q.tile = -1;
  if (s > 1 && (p.offsets || 2 * (int64_t)s > (p.k + 255) / 256)) q.tile = -1;
  if ((q.tiles_m * q.tiles_n * s + 7) * T::THREADS > kMaxLaunchThreads) q.tile = -1;
  return q;
}

// The tile and, for one weight, the parts of k that the costs above say take
// the least time; the parts' sums cost a launch (3 us) and their bytes, written
// and read, at 4 TB/s.  Examples (us, graph replays, the five tiles, each
// with its best of 1, 2 and 4 parts): 256 x 8192 x 8192, MXFP8, 34 / 30 / 30 / 22 /
// 25, the fourth is taken; 4096 x 11008 x 4096, MXFP4, 127 / 152 / 185 / 210 / 202;
// 3001 rows over 7 experts of 2048 x 5632, MXFP4, 46 / 34 / 43 / 44 / 44; 8192 rows
// over 32 experts of 4096 x 2048, MXFP8, 113 / 141 / 126 / 168 / 130.
template <int AF>
Plan make_plan(const MxProblem& p) {
  const int64_t steps = (p.k + 255) / 256, cus = device_cus();
  Plan best{4, 1, 0, 0};
  double least = 0;
  for (int t = 0; t < 5; ++t) {
    with_tile<AF>(t, [&](auto X) {
      using T = decltype(X);
      const Cost c = Tiles<AF>::cost[t];
      const double G = (double)most_groups(p);
      const double rows = p.offsets ? (double)p.m / T::BM + 0.5 * G  // half a tile lost to each group
                                    : (double)((p.m + T::BM - 1) / T::BM);
      for (uint32_t s = 1; s <= kMaxSplits; s *= 2) {
        const Plan q = plan_on<T>(p, t, s);
        if (q.tile < 0) continue;
        const int64_t n = (int64_t)(rows * (double)q.tiles_n + 0.5) * s;
        const double k = (double)((steps + s - 1) / s), find = p.offsets ? 2.0 : 0.0;  // the walk of the offsets
        const double alone = find + c.first + c.step * k, pair = find + c.first2 + c.step2 * k;
        const int64_t round = cus * T::PER_CU, full = n / round, rest = n % round;
        double us = full * (T::PER_CU == 2 ? pair : alone);
        if (rest) us += rest <= cus ? alone : pair;
        if (s > 1) us += 3.0 + (double)s * p.m * p.n * 8 / 4e6;
        if (best.tiles_m == 0 || us < least) {
          least = us;
          best = q;
        }
      }
    });
  }
  if (best.tiles_m == 0) best.tiles_m = best.tiles_n = INT64_C(1) << 31;  // too many tiles of every size
  return best;
}

// Products with few rows a weight: one tile of 16, or on average at most five
// (us as tiles of 16 / of 64: 64 rows over 26 experts of 4096 x 2048 30.7 / 32.9,
// 96 rows over 29 of them 32.3 / 34.9, 256 rows over 63 of 4096 x 1024 35 / 43,
// 256 rows over 32 of 2048 x 5632, eight a weight, 53 / 45).
bool skinny(const MxProblem& p) {
  return p.m <= 16 || (p.offsets && p.m <= 5 * (int64_t)p.experts);
}

template <int AF, typename T, bool GROUPED>
hipError_t launch_tile(const MxProblem& p, const GemmArgs& g, uint32_t blocks, hipStream_t stream) {
  constexpr int lds = T::LDS * 16;
  // the LDS limit is raised once per device (one bit each for the first 64);
  // callers racing here all set the same value
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&mx_gemm_kernel<AF, T, GROUPED>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    configured.fetch_or(bit, std::memory_order_release);
  }
  mx_gemm_kernel<AF, T, GROUPED><<<dim3(blocks), dim3(T::THREADS), lds, stream>>>(p, g);
  return hipGetLastError();
}

template <int AF>
hipError_t launch_gemm_format(const MxProblem& p, const Plan& q, hipStream_t stream) {
  GemmArgs g{(uint32_t)q.tiles_m, (uint32_t)q.tiles_n, q.splits, nullptr};
  std::unique_lock<std::mutex> turn;
  if (q.splits > 1) {
    turn = stream_turn(stream);
    char* ws = nullptr;
    const hipError_t e =
        stream_workspace(kWorkspaceMx, stream, (size_t)q.splits * p.m * p.n * sizeof(float), &ws);
    if (e != hipSuccess) return e;
    g.partial = reinterpret_cast<float*>(ws);
  }
  const hipError_t e = with_tile<AF>(q.tile, [&](auto X) {
    using T = decltype(X);
    return p.offsets ? launch_tile<AF, T, true>(p, g, (uint32_t)q.blocks(), stream)
                     : launch_tile<AF, T, false>(p, g, (uint32_t)q.blocks(), stream);
  });
  if (e != hipSuccess || q.splits == 1) return e;
  const int64_t count = p.m * p.n;
  mx_join_kernel<<<dim3((uint32_t)((count + 1023) / 1024)), dim3(256), 0, stream>>>(g.partial, q.splits, count, p.y,
                                                                                    p.y_bf16);
  return hipGetLastError();
}

}  // namespace

int64_t mx_linear_blocks(int x_fmt, const MxProblem& p) {
  if (skinny(p)) return mx_skinny_blocks(x_fmt, p);
  // No tile is smaller than 64 x 128 (nor has more threads) and k has at most
  // kMaxSplits parts: where a launch holds the blocks of that, it holds any
  // plan's, and the costs are computed by the launch only.
  const int64_t groups = p.offsets ? most_groups(p) : 1;
  const int64_t most = (groups + p.m / 64) * ((p.n + 127) / 128) * (p.offsets ? 1 : kMaxSplits);
  if ((most + 7) * 512 <= kMaxLaunchThreads) return most;
  return (x_fmt == kMxFp8 ? make_plan<kMxFp8>(p) : make_plan<kMxFp4>(p)).blocks();
}

hipError_t launch_mx_linear(int x_fmt, const MxProblem& p, hipStream_t stream) {
  if (skinny(p)) return launch_mx_skinny(x_fmt, p, mx_skinny_shape(x_fmt, p), stream);
  return x_fmt == kMxFp8 ? launch_gemm_format<kMxFp8>(p, make_plan<kMxFp8>(p), stream)
                         : launch_gemm_format<kMxFp4>(p, make_plan<kMxFp4>(p), stream);
}

extern "C" int32_t w4_mx_kernel_of(int32_t x_fmt, int32_t experts, int64_t n, int64_t k, int64_t m) {
  static const int32_t some = 0;
  const MxProblem p{nullptr, nullptr, nullptr, nullptr, experts ? &some : nullptr, nullptr, nullptr, m, n, k, m,
                    experts ? experts : 1, 0};
  if (skinny(p)) return 256 + mx_skinny_shape(x_fmt, p);
  const Plan q = x_fmt == kMxFp8 ? make_plan<kMxFp8>(p) : make_plan<kMxFp4>(p);
  return 16 * (int32_t)q.splits + q.tile;
}

extern "C" int32_t w4_mx_product_on(int32_t kernel, int32_t x_fmt, int32_t experts, int64_t n, int64_t k,
                                    const uint8_t* w, const uint8_t* w_scales, int64_t tokens, const uint8_t* x,
                                    const uint8_t* x_scales, int64_t rows, const int32_t* offsets,
                                    const int32_t* row_index, void* y, int32_t y_bf16, void* stream) {
  const MxProblem p{w, w_scales, x, x_scales, offsets, row_index, y, rows, n, k, tokens, offsets ? experts : 1, y_bf16};
  const hipStream_t on = static_cast<hipStream_t>(stream);
  if (kernel >= 256) {
    if (kernel > 258 || (!offsets && rows > 16)) return hipErrorInvalidValue;
    return launch_mx_skinny(x_fmt, p, kernel - 256, on);
  }
  const uint32_t parts = (uint32_t)kernel / 16;
  if (kernel % 16 > 4 || parts < 1 || parts > kMaxSplits) return hipErrorInvalidValue;
  auto go = [&](auto AF) -> hipError_t {
    const Plan q = with_tile<decltype(AF)::value>(kernel % 16, [&](auto X) {
      return plan_on<decltype(X)>(p, kernel % 16, parts);
    });
    if (q.tile < 0) return hipErrorInvalidValue;
    return caught([&] { return launch_gemm_format<decltype(AF)::value>(p, q, on); });
  };
  return x_fmt == kMxFp8 ? go(std::integral_constant<int, kMxFp8>{}) : go(std::integral_constant<int, kMxFp4>{});
}

}  // namespace w4
