// Host-side launchers of the gfx950 kernels (internal to libw4; the public
// ABI is include/w4.h).  Arguments are validated by w4_api.cpp before any of
// these is called; each launcher only enqueues on `stream`.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>

namespace w4 {

// A launch holds fewer than 2^32 threads (HIP cuts a larger one without an error).
constexpr int64_t kMaxLaunchThreads = 0xFFFFFFFF;
// What a launcher returns, before it enqueues anything, for a size that needs more.
constexpr hipError_t kTooLarge = hipErrorInvalidConfiguration;
inline bool too_large(int64_t blocks, int threads) { return blocks > kMaxLaunchThreads / threads; }

// f()'s error.  A launcher may allocate on the host (the tables of workspaces); nothing
// that it throws passes the C boundary.
template <typename F>
hipError_t caught(F&& f) {
  try {
    return f();
  } catch (...) {
    return hipErrorOutOfMemory;
  }
}

// f(first, count) over parts of at most `most` of `total`, until one fails: the
// launches of an elementwise call.
template <typename F>
hipError_t in_parts(int64_t total, int64_t most, F&& f) {
  hipError_t e = hipSuccess;
  for (int64_t at = 0; at < total && e == hipSuccess; at += most) e = f(at, total - at < most ? total - at : most);
  return e;
}

// Weights of a launch of the codecs' elementwise kernels: a thread takes eight
// at least.
constexpr int64_t kMaxLaunchWeights = INT64_C(1) << 33;

// Same layout as w4_gemv_problem in include/w4.h.
struct GemvProblem {
  const uint8_t* packed;
  const uint16_t* scales;
  const uint16_t* codebook;
  const uint16_t* x;
  void* y;
  int64_t n;
  int64_t k;
  int64_t tile_begin;
};

hipError_t launch_quantize(int codec, int64_t n, int64_t k, const uint16_t* w, uint8_t* packed,
                           uint16_t* scales, const uint16_t* codebook, hipStream_t stream);

hipError_t launch_quantize_dyadic5(int64_t n, int64_t k, const uint16_t* w, const uint8_t* widths,
                                   uint8_t* packed, uint8_t* msb, uint16_t* scales,
                                   hipStream_t stream);

// W4_LUT16S_IL records (k a multiple of 256) from planar LUT16S arrays
hipError_t launch_lut16s_interleave(int64_t n, int64_t k, const uint8_t* packed,
                                    const uint16_t* scales, uint8_t* out, hipStream_t stream);

hipError_t launch_dequant(int codec, int64_t n, int64_t k, const uint8_t* packed,
                          const uint16_t* scales, const uint16_t* codebook, void* out,
                          hipStream_t stream);

hipError_t launch_lut16_fit(int64_t n, int64_t k, const uint16_t* w, uint16_t* scales,
                            uint16_t* lut, int iters, hipStream_t stream);
hipError_t launch_signmag8_fit(int64_t n, int64_t k, const uint16_t* w, uint16_t* codebook,
                               int iters, hipStream_t stream);
hipError_t launch_signmag8_warm_fit(int64_t n, int64_t k, const uint16_t* w, uint16_t* codebook,
                                    uint8_t* params, int iters, hipStream_t stream);

hipError_t launch_gemv(int codec, const GemvProblem& p, int m, int y_bf16, hipStream_t stream);

// y[0 .. count) = +0 (fp32, or bf16 when y_bf16): the product over k == 0.
hipError_t launch_zero(void* y, int64_t count, int y_bf16, hipStream_t stream);

// The batched GEMV's plan takes 64-row tiles, or for m == 1 halves them (down
// to 16) while the launch would have fewer than this many tiles.
constexpr int64_t kGemvBatchedMinTiles = 1024;
// probs_dev: count problems with tile_begin set by the plan for tiles of
// tile_rows (64; 32 or 16 only with m == 1) rows
// ragged: some problem's k is not a multiple of 256 (its last step is partial)
hipError_t launch_gemv_batched(int codec, const GemvProblem* probs_dev, int count,
                               int64_t total_tiles, int64_t k_max, int tile_rows, int m,
                               int y_bf16, bool ragged, hipStream_t stream);

// Library-owned device buffer of at least `bytes` for (current device, stream,
// user); its contents are undefined.  Growing allocates a new buffer and keeps
// the old one (work already enqueued, or a graph captured earlier, may still
// use it), so it never waits for the stream.
enum { kWorkspaceGemm = 0, kWorkspaceGemv = 1, kWorkspaceMx = 2 };
hipError_t stream_workspace(int user, hipStream_t stream, size_t bytes, char** out);
// The calling thread's turn on a stream (of the current device).  A call that fills a
// workspace in one launch and reads it in a later one holds it from the lookup of the
// workspace to its last launch, so that another host thread's call on the stream comes
// before or behind all of them.  Streams' turns are apart.
[[nodiscard]] std::unique_lock<std::mutex> stream_turn(hipStream_t stream);
// A number of the calling thread from 1 on, never given again (the system gives
// an ended thread's id again, while its last kernels may still run).
uint64_t this_thread();
// A product's sums may be cut into kMxMaxParts parts in all, a tile's into kMxMaxSplits
// (256 MB of sums on the largest tile; more than four blocks a CU are not worth their
// joining).
constexpr int kMxMaxParts = 1024, kMxMaxSplits = 16;
// A counter for each tile that a launch cuts into `splits` parts (2 .. kMxMaxSplits; at
// most kMxMaxParts / splits tiles), of (current device, stream), zeros to begin with:
// every launch that counts in them leaves zeros behind (w4_counters.cpp).
hipError_t stream_counters(hipStream_t stream, uint32_t splits, uint32_t** out);

// ws: a workspace of at least gemm_workspace_bytes(...) bytes, or nullptr for
// the library-kept one of the stream (stream_workspace)
hipError_t launch_gemm(int codec, const GemvProblem& p, int m, int y_bf16, hipStream_t stream,
                       char* ws);
size_t gemm_workspace_bytes(int codec, int64_t n, int64_t k, int m);

// Device address of the current device's copy of the fixed scratch array
// (w4_noalloc.hip), looked up once per device; its size in bytes.
hipError_t noalloc_scratch(char** out);
constexpr size_t kNoallocScratchBytes = size_t{64} << 20;

// ---- MX (microscaled) operators
// One product y[m][n] = x w^T, or with offsets != nullptr the products of
// `experts` weights with the rows of y that offsets gives each of them.
struct MxProblem {
  const uint8_t* w;         // fp4 elements [experts][n][k/2]
  const uint8_t* w_scales;  // [experts][n][k/32]
  const uint8_t* x;         // elements [tokens][k or k/2]
  const uint8_t* x_scales;  // [tokens][k/32]
  const int32_t* offsets;   // [experts + 1], or nullptr
  const int32_t* row_index; // [m] rows of x, or nullptr: row i of y takes row i of x
  void* y;                  // [m][n]
  int64_t m, n, k, tokens;
  int32_t experts, y_bf16;
};

hipError_t launch_mx_quantize(int fmt, int64_t rows, int64_t k, const void* x, int dtype, uint8_t* q,
                              uint8_t* scales, hipStream_t stream);
hipError_t launch_mx_dequant(int fmt, int64_t rows, int64_t k, const uint8_t* q, const uint8_t* scales,
                             void* out, int dtype, hipStream_t stream);
hipError_t launch_mx_rmsnorm(int fmt, int64_t rows, int64_t k, const void* x, const void* residual,
                             const void* gamma, int dtype, float eps, void* residual_out, void* y,
                             uint8_t* q, uint8_t* scales, hipStream_t stream);
// blocks of the product's launch at most; 2^31 or more: too many for a launch
int64_t mx_linear_blocks(int x_fmt, const MxProblem& p);
hipError_t launch_mx_linear(int x_fmt, const MxProblem& p, hipStream_t stream);
// For the tests, which name the kernel that they run: kernel 16 * parts of k +
// tile (w4_mx_gemm.hip), or with few rows a weight 256 + shape (w4_mx_skinny.hip).
// The kernel that a product takes (experts 0: one weight):
extern "C" int32_t w4_mx_kernel_of(int32_t x_fmt, int32_t experts, int64_t n, int64_t k, int64_t m);
// The product on a kernel of the caller's choice, with arguments that
// w4_mx_grouped_linear accepts (offsets == nullptr: w4_mx_linear) and something
// to compute; a hipError_t, an error where the kernel does not fit the product.
extern "C" int32_t w4_mx_product_on(int32_t kernel, int32_t x_fmt, int32_t experts, int64_t n, int64_t k,
                                    const uint8_t* w, const uint8_t* w_scales, int64_t tokens, const uint8_t* x,
                                    const uint8_t* x_scales, int64_t rows, const int32_t* offsets,
                                    const int32_t* row_index, void* y, int32_t y_bf16, void* stream);
// few rows of x a weight (w4_mx_skinny.hip)
int64_t mx_skinny_blocks(int x_fmt, const MxProblem& p);
int mx_skinny_shape(int x_fmt, const MxProblem& p);  // 0 .. 2
hipError_t launch_mx_skinny(int x_fmt, const MxProblem& p, int shape, hipStream_t stream);

// ---- bf16 rows times MXFP4 weights
// kMxForward: y[m][n] = x w^T.  kMxGated: w holds n gate and n up rows, y[m][n] =
// act(x gate^T) * (x up^T).  kMxBackward: y[m][k] = x w, x [m][n].
constexpr int kMxForward = 0, kMxGated = 1, kMxBackward = 2;
struct MxBf16Problem {
  const uint8_t* w;         // fp4 elements [n, gated 2 n][k/2]
  const uint8_t* w_scales;  // [n, gated 2 n][k/32]
  const uint16_t* x;        // bf16 rows of x_pitch values, whole 16-byte units
  void* y;
  uint16_t* gu;             // gated: bf16 [m][2 n], or nullptr
  int64_t m, n, k, x_pitch;
  int32_t y_bf16, act, kind;
};
// Backward of the gated block: dgu[m][2 n] from dh [m][n] and gu [m][2 n], bf16.
struct MxGateGrad {
  const uint16_t* dh;
  const uint16_t* gu;
  uint16_t* dgu;
  int64_t m, n;
  int32_t act;
};
// false: some launch would need more than 2^32 threads
bool mx_bf16_fits(const MxBf16Problem& p);
// (w4_mx_bf16_gemm.hip) with the library's workspace of the stream; `reserve` bytes of
// it (whole 256), before the product's own, are the caller's: fill (or nullptr)
// enqueues what writes them, and may change the problem
struct MxBf16Fill {
  virtual hipError_t operator()(MxBf16Problem& p, char* reserved) = 0;
};
hipError_t launch_mx_bf16_with(const MxBf16Problem& p, size_t reserve, MxBf16Fill* fill, hipStream_t stream);
// at most 16 rows, forward (w4_mx_bf16_skinny.hip)
int mx_bf16_skinny_shape(const MxBf16Problem& p);
hipError_t launch_mx_bf16_skinny(const MxBf16Problem& p, int shape, hipStream_t stream);
// few rows, backward (w4_mx_bf16_narrow.hip): `splits` blocks a tile, whose parts' sums
// and counts (of each tile) are partial and counted
hipError_t launch_mx_bf16_narrow(const MxBf16Problem& p, uint32_t splits, char* partial, uint32_t* counted,
                                 hipStream_t stream);
// For the tests, which name the kernel that they run: 16 * parts of the sum + tile
// (w4_mx_bf16_gemm.hip), 1024 more where only the last tiles are cut into parts, or
// 4096 + shape (w4_mx_bf16_skinny.hip).  The kernel that a product takes:
extern "C" int32_t w4_mx_bf16_kernel_of(int32_t kind, int64_t n, int64_t k, int64_t m);
// The product (kind, sizes and pointers as in MxBf16Problem, x without padding)
// on a kernel of the caller's choice; a hipError_t, an error where it does not fit.
extern "C" int32_t w4_mx_bf16_product_on(int32_t kernel, int32_t kind, int32_t act, int64_t n, int64_t k,
                                         const uint8_t* w, const uint8_t* w_scales, const uint16_t* x, int64_t m,
                                         uint16_t* gu, void* y, int32_t y_bf16, void* stream);
// (w4_mx_bf16.hip) with the library's workspace of the stream.  Backward, x's
// pitch may be any n: rows of no whole 16-byte units are padded into the
// workspace first.
hipError_t launch_mx_bf16(const MxBf16Problem& p, hipStream_t stream);
// dgu, then (where p.k > 0) p, kMxBackward over dgu
hipError_t launch_mx_gated_grad(const MxGateGrad& g, const MxBf16Problem& p, hipStream_t stream);

}  // namespace w4
