// A HIP runtime for the CPU: the program that includes this defines the runtime's
// functions that libw4.so calls, so the library as it is built runs its host side
// against them.  Kernels do not run; on_launch gets the name, the arguments and the
// stream of each.  Device memory is host memory, zeros at first.
#pragma once

#define __HIP_PLATFORM_AMD__ 1
#include <hip/hip_runtime_api.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <functional>
#include <map>
#include <string>

namespace fake {
inline std::map<const void*, std::string>& names() {  // (the library registers before main's file is set up)
  static std::map<const void*, std::string> m;
  return m;
}
inline std::function<void(const std::string& kernel, void** args, hipStream_t stream)> on_launch;
struct Call {
  dim3 grid, block;
  size_t shared;
  hipStream_t stream;
};
inline thread_local Call call;
inline int failures = 0;
}  // namespace fake

#define EXPECT(c)                                          \
  do {                                                     \
    if (!(c)) {                                            \
      fprintf(stderr, "FAIL line %d: %s\n", __LINE__, #c); \
      ++fake::failures;                                    \
    }                                                      \
  } while (0)

extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* module;
  return &module;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* stub, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
  fake::names()[stub] = name;
}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t stream) {
  fake::call = {grid, block, shared, stream};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
  *grid = fake::call.grid;
  *block = fake::call.block;
  *shared = fake::call.shared;
  *stream = fake::call.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* stub, dim3, dim3, void** args, size_t, hipStream_t stream) {
  const auto at = fake::names().find(stub);
  if (at == fake::names().end()) return hipErrorInvalidDeviceFunction;
  if (fake::on_launch) fake::on_launch(at->second, args, stream);
  return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipGetDevice(int* dev) {
  *dev = 0;
  return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* value, hipDeviceAttribute_t, int) {
  *value = 256;  // compute units
  return hipSuccess;
}
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* status) {
  *status = hipStreamCaptureStatusNone;
  return hipSuccess;
}
hipError_t hipMalloc(void** p, size_t bytes) {
  *p = calloc(bytes, 1);
  return *p ? hipSuccess : hipErrorOutOfMemory;
}
hipError_t hipFree(void* p) {
  free(p);
  return hipSuccess;
}
hipError_t hipGetSymbolAddress(void** p, const void*) {
  static char scratch[256];  // (nothing runs in it)
  *p = scratch;
  return hipSuccess;
}
}
