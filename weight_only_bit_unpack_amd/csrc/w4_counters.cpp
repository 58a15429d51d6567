// Device counters kept by the library per (device, stream): the parts of a
// product's tiles that are done.  They are zeroed once, by a kernel on the stream
// that they belong to, and every launch that counts in them leaves zeros behind,
// so no call has to clear them.  Calls on one stream are ordered and share the
// counters; calls on different streams never do, and hipStreamPerThread is a
// stream of its own in each thread under one handle.  They are never freed, as
// the workspaces (w4_workspace.cpp).
#include "w4_launch.h"

#include <map>
#include <mutex>
#include <tuple>

namespace w4 {

hipError_t stream_counters(hipStream_t stream, uint32_t** out) {
  static std::mutex mu;
  static std::map<std::tuple<int, hipStream_t, uint64_t>, uint32_t*> kept;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t thread = stream == hipStreamPerThread ? this_thread() : 0;
  std::lock_guard<std::mutex> g(mu);
  uint32_t*& slot = kept[std::make_tuple(dev, stream, thread)];
  if (!slot) {
    // (a captured kernel would zero them at replays only)
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    e = hipStreamIsCapturing(stream, &capture);
    if (e != hipSuccess) return e;
    if (capture != hipStreamCaptureStatusNone) return hipErrorStreamCaptureUnsupported;
    uint32_t* p = nullptr;
    e = hipMalloc(reinterpret_cast<void**>(&p), kMxCounters * sizeof(uint32_t));
    if (e != hipSuccess) return e;
    e = launch_zero(p, kMxCounters, 0, stream);
    if (e != hipSuccess) {
      (void)hipFree(p);  // (nothing uses it yet)
      return e;
    }
    slot = p;
  }
  *out = slot;
  return hipSuccess;
}

}  // namespace w4
