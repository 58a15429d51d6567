// Device-side building blocks of the MX (microscaled) kernels of libw4.
//
// An MX block is 32 consecutive values along k: elements of 4 bits (E2M1) or
// 8 bits (E4M3) and one power-of-two scale byte b, 2^(b - 127).
#pragma once

#include "w4_device.h"

namespace w4 {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Formats, as w4_mx_format.
constexpr int kMxFp4 = 0, kMxFp8 = 1;

// Largest binary exponent of an element: 6 = 1.5 * 2^2, 448 = 1.75 * 2^8.
template <int FMT>
constexpr uint32_t kMxEmax = FMT == kMxFp4 ? 2u : 8u;

// 2^(b - 127) of a scale byte as fp32, exact (b = 0 is a subnormal); 255 is NaN.
__device__ __forceinline__ float mx_scale_value(uint32_t b) {
  const uint32_t u = b == 0 ? 0x00400000u : b == 255u ? 0x7FC00000u : b << 23;
  return __builtin_bit_cast(float, u);
}

// Maximum of v over each aligned quad of lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  // quad_perm [1,0,3,2] and [2,3,0,1]
  const uint32_t a = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
  v = v > a ? v : a;
  const uint32_t b = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);
  return v > b ? v : b;
}

// Quantize one MX block held by an aligned quad of lanes, eight values each.
// b: the block's scale byte; e: the lane's eight element codes (one dword of
// nibbles, or two dwords of bytes).
//
// The magnitudes compare as their bit patterns (NaN above infinity above every
// number), so the block's largest is an integer maximum and its exponent field
// E is floor(log2) + 127.  A block with a NaN or an infinity has no scale: it
// becomes scale 255 (NaN) with zero codes.  Otherwise b = E - emax, at least 0
// (a subnormal or zero maximum has E = 0), at most 252, so 2^(127 - b) is a
// normal fp32 number and the product is exact except where it falls far below
// half the smallest element and becomes 0 either way.  The conversions round
// to nearest even; values that the scaled maximum's binade leaves above the
// largest element become the largest (the fp4 conversion saturates by itself).
template <int FMT>
__device__ __forceinline__ void mx_quantize8(const float (&v)[8], uint32_t& b, uint32_t (&e)[2]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu;
    top = top > u ? top : u;
  }
  const uint32_t E = quad_max(top) >> 23;
  const bool bad = E == 255u;
  b = bad ? 255u : E > kMxEmax<FMT> ? E - kMxEmax<FMT> : 0u;
  const float s = __builtin_bit_cast(float, (bad ? 127u : 254u - b) << 23);
  if constexpr (FMT == kMxFp4) {
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0] * s, v[1] * s, 1.0f, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2] * s, v[3] * s, 1.0f, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4] * s, v[5] * s, 1.0f, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6] * s, v[7] * s, 1.0f, 3);
    e[0] = bad ? 0u : r;
    e[1] = 0u;
  } else {
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = __builtin_amdgcn_fmed3f(v[i] * s, -448.0f, 448.0f);
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], hi, true);
    e[0] = bad ? 0u : (uint32_t)lo;
    e[1] = bad ? 0u : (uint32_t)hi;
  }
}

// Stores a lane's eight element codes at group of eight `g` of the array.
template <int FMT>
__device__ __forceinline__ void mx_store8(uint8_t* q, int64_t g, const uint32_t (&e)[2]) {
  if constexpr (FMT == kMxFp4)
    reinterpret_cast<uint32_t*>(q)[g] = e[0];
  else
    reinterpret_cast<u32x2*>(q)[g] = (u32x2){e[0], e[1]};
}

// Input types by w4_dtype: eight consecutive values <-> fp32.
constexpr int kF32 = 0, kBf16 = 1, kF16 = 2;

template <int DT>
struct Raw8 {
  u32x4 a;
};
template <>
struct Raw8<kF32> {
  u32x4 a, b;
};

template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const void* x, int64_t g) {
  Raw8<DT> r;
  if constexpr (DT == kF32) {
    r.a = reinterpret_cast<const u32x4*>(x)[2 * g];
    r.b = reinterpret_cast<const u32x4*>(x)[2 * g + 1];
  } else {
    r.a = reinterpret_cast<const u32x4*>(x)[g];
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void to_f32(const Raw8<DT>& r, float (&v)[8]) {
  if constexpr (DT == kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (a bit cast of a vector's element itself reads element 0)
      v[i] = __builtin_bit_cast(float, (uint32_t)r.a[i]);
      v[4 + i] = __builtin_bit_cast(float, (uint32_t)r.b[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == kBf16) {
        v[2 * i] = bf16_bits_to_f32(r.a[i] & 0xFFFFu);
        v[2 * i + 1] = __builtin_bit_cast(float, r.a[i] & 0xFFFF0000u);
      } else {
        const f16x2 h = __builtin_bit_cast(f16x2, (uint32_t)r.a[i]);
        v[2 * i] = (float)h.x;
        v[2 * i + 1] = (float)h.y;
      }
    }
  }
}

// fp32 -> the type, to nearest even.
template <int DT>
__device__ __forceinline__ Raw8<DT> from_f32(const float (&v)[8]) {
  Raw8<DT> r;
  if constexpr (DT == kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.a[i] = __builtin_bit_cast(uint32_t, v[i]);
      r.b[i] = __builtin_bit_cast(uint32_t, v[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == kBf16) {
        r.a[i] = cvt_pk_bf16(v[2 * i], v[2 * i + 1]);
      } else {
        const f16x2 h = {(_Float16)v[2 * i], (_Float16)v[2 * i + 1]};
        r.a[i] = __builtin_bit_cast(uint32_t, h);
      }
    }
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void store8(void* x, int64_t g, const Raw8<DT>& r) {
  if constexpr (DT == kF32) {
    reinterpret_cast<u32x4*>(x)[2 * g] = r.a;
    reinterpret_cast<u32x4*>(x)[2 * g + 1] = r.b;
  } else {
    reinterpret_cast<u32x4*>(x)[g] = r.a;
  }
}

// Orders one lane's LDS accesses with another lane's of the same wave.  The
// hardware runs a wave's LDS instructions in order; this keeps the compiler
// from taking a value that this lane has not written to be the one it read
// before.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// A pointer that is the same in every lane, kept in scalar registers.
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
  return reinterpret_cast<const uint8_t*>((uint64_t)hi << 32 | lo);
}

// Buffer resource over `bytes` from base: loads at an offset past it return zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes,
                                           0x00020000);
}
// An offset past every resource (a block's rows hold at most 2^31 bytes).
constexpr uint32_t kMxOOB = 0xFFFFFF00u;

__device__ __forceinline__ u32x4 mx_load16(__amdgpu_buffer_rsrc_t r, uint32_t offset) {
  const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, 0);
  return (u32x4){v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ uint32_t mx_load1(__amdgpu_buffer_rsrc_t r, uint32_t offset) {
  return (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(r, offset, 0, 0);
}

// Matrix operand registers: fp4 takes the first 16 bytes, fp8 both.
template <int FMT>
__device__ __forceinline__ i32x8 mx_operand(const u32x4& a, const u32x4& b) {
  if constexpr (FMT == kMxFp4)
    return (i32x8){(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  else
    return (i32x8){(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// Four consecutive outputs of one row from column c on, where c + i < n.
__device__ __forceinline__ void mx_store4(void* y, int y_bf16, int64_t row_base, int64_t c, int64_t n,
                                          const f32x4& v) {
  if (y_bf16) {
    uint16_t* const p = reinterpret_cast<uint16_t*>(y) + row_base + c;
    if (c + 4 <= n && (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
      *reinterpret_cast<u32x2*>(p) = (u32x2){cvt_pk_bf16(v.x, v.y), cvt_pk_bf16(v.z, v.w)};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < n) p[i] = (uint16_t)f32_to_bf16_bits(v[i]);
    }
  } else {
    float* const p = reinterpret_cast<float*>(y) + row_base + c;
    if (c + 4 <= n && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
      *reinterpret_cast<f32x4*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < n) p[i] = v[i];
    }
  }
}

// D[16][16] += A[16][128] B[128][16] with block scales.  Lane l: row (A) or
// column (B) l % 16; with g = l / 16, fp4 registers 0-3 hold k = 32 g .. + 31,
// fp8 registers 0-3 k = 16 g .. + 15 and registers 4-7 k = 64 + 16 g .. + 15;
// the scale (low byte) is that of k block g.  D: row 4 (l / 16) + i, column
// l % 16.
template <int AF, int BF>
__device__ __forceinline__ f32x4 mx_mfma16(const i32x8& a, const i32x8& b, const f32x4& c, uint32_t sa,
                                           uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
      a, b, c, AF == kMxFp8 ? 0 : 4, BF == kMxFp8 ? 0 : 4, 0, (int)sa, 0, (int)sb);
}

// D[32][32] += A[32][64] B[64][32] with block scales.  AF: format of A; B is
// fp4.  Lane l: row (A) or column (B) l % 32.  With g = l / 32:
//   fp4: registers 0-3 hold k = 32 g .. 32 g + 31, low nibble first;
//   fp8: registers 0-3 hold k = 16 g .. + 15, registers 4-7 k = 32 + 16 g .. + 15;
//   byte OPS of the scale register is the scale of k block g (32 g .. 32 g + 31).
// D as of mfma32x32x16.  fp4 x fp4 products add exactly (to the fp32
// accumulator's own rounding); with fp8 the matrix core aligns the products of
// eight neighbours along k (8 i .. 8 i + 7) to the largest of their exponents and
// drops what lies 2^-13 and more below it (both instructions, found by placing
// one large and one small product at every pair of places).  That is at most
// 7 * 2^-13 of the magnitudes, and 4.2e-6 of the result in the 2-norm on normal
// data at k = 4096, far below the elements' own rounding (2^-4).
template <int AF, int OPA, int OPB>
__device__ __forceinline__ f32x16 mx_mfma32(const i32x8& a, const i32x8& b, const f32x16& c, uint32_t sa,
                                            uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, AF == kMxFp8 ? 0 : 4, 4, OPA,
                                                         (int)sa, OPB, (int)sb);
}

}  // namespace w4
