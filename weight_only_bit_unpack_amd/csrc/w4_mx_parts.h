// Sums that blocks share: each block of a tile writes its part, and the one that
// counts last adds the parts in order, so that the bits are the same whichever is
// last.  Nobody waits.
//
// Parts are written and read with device scope, past the caches that belong to one
// XCD: then a wave's wait for its stores is all that the count needs before it (a
// release of the device would write back an XCD's whole cache; products of one row
// took 13 instead of 9 us with it).
#pragma once

#include "w4_device.h"

namespace w4 {

// pairs v = 0 .. N - 1 of a thread, get(v), to at[v * stride]
template <int N, typename F>
__device__ __forceinline__ void put_part(uint64_t* at, int stride, F&& get) {
#pragma unroll
  for (int v = 0; v < N; ++v)
    __hip_atomic_store(at + v * stride, __builtin_bit_cast(uint64_t, (f32x2)get(v)), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}

// Every thread of the block calls this when its part is put; true in the block
// that is the last of `splits`, whose count is then back at zero.  `before` is a dword of
// LDS that nobody reads or writes any more.
__device__ __forceinline__ bool last_part(uint32_t* counted, uint32_t splits, uint32_t* before) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) {
    *before = atomicInc(counted, splits - 1);  // (after splits - 1 comes 0)
  }
  __syncthreads();
  return *before + 1 == splits;
}

// set(v, sum of pair v over the parts, in order): part p's at from[p * part + v *
// stride]; AHEAD parts' loads in flight
template <int N, int AHEAD, typename F>
__device__ __forceinline__ void add_parts(const uint64_t* from, int64_t part, int stride, uint32_t splits, F&& set) {
  f32x2 total[N];
  for (uint32_t p0 = 0; p0 < splits; p0 += AHEAD) {
    uint64_t x[AHEAD][N];
#pragma unroll
    for (uint32_t p = 0; p < AHEAD; ++p)
      if (p0 + p < splits) {
#pragma unroll
        for (int v = 0; v < N; ++v)
          x[p][v] = __hip_atomic_load(from + (int64_t)(p0 + p) * part + v * stride, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT);
      }
#pragma unroll
    for (uint32_t p = 0; p < AHEAD; ++p)
      if (p0 + p < splits) {
#pragma unroll
        for (int v = 0; v < N; ++v) {
          const f32x2 y = __builtin_bit_cast(f32x2, x[p][v]);
          total[v].x = p0 + p == 0 ? y.x : total[v].x + y.x;
          total[v].y = p0 + p == 0 ? y.y : total[v].y + y.y;
        }
      }
  }
#pragma unroll
  for (int v = 0; v < N; ++v) set(v, total[v]);
}

}  // namespace w4
