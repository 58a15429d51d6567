// Copies from global memory straight to LDS, and the waits that go with them.
#pragma once

#include "w4_device.h"

namespace w4 {

// 64 x 16 bytes, one unit a lane, from global memory to consecutive LDS at
// `to` (the same in every lane), without registers between.  Written as
// assembly because after the builtin form the compiler makes every LDS read
// wait for all copies in flight, the next step's too; the waits are placed by
// hand instead.  It has no register outputs.  It writes m0, which this compiler
// reserves and does not let a statement declare as written: in these kernels
// nothing else may read or set m0 (no builtin that moves to or from LDS or
// indexes registers through it; the assembly holds no other use).
__device__ __forceinline__ uint32_t lds_address(const u32x4* p) {
  return __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p);
}
__device__ __forceinline__ void copy16(const uint8_t* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from)
               : "memory");
}
__device__ __forceinline__ void copy16(const uint8_t* base, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset),
               "s"(base)
               : "memory");
}
// 64 bytes, one a lane, each to a dword of its own (zeros above it).
__device__ __forceinline__ void copy_byte(const uint8_t* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, off" ::"s"(to), "v"(from)
               : "memory");
}
__device__ __forceinline__ void copy_byte(const uint8_t* base, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, %2" ::"s"(to), "v"(offset),
               "s"(base)
               : "memory");
}

// s_waitcnt for at most n vector memory operations in flight, the others free.
constexpr int wait_vm(int n) { return (n & 15) | (n >> 4) << 14 | 0x0F70; }
// s_waitcnt for every LDS operation, the others free.
constexpr int kWaitLds = 0xC07F;

}  // namespace w4
