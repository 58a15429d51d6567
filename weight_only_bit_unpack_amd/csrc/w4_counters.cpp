// Device counters kept by the library per (device, stream): the parts of a
// product's tiles that are done.  They are zeroed once, by a kernel on the stream
// that they belong to, and every launch that counts in them leaves zeros behind,
// so no call has to clear them.  Calls on one stream are ordered and share the
// counters; calls on different streams never do, and hipStreamPerThread is a
// stream of its own in each thread under one handle.  They are never freed, as
// the workspaces (w4_workspace.cpp).
//
// Each number of parts has counters of its own.  A count goes round modulo the number
// of parts, and a launch counts each of its tiles as often as that: so it is back at
// zero when all launches have ended, in whatever order their blocks counted.  Were a
// counter shared by launches of several numbers of parts, replays of captured calls
// that overlap would leave counts behind, and every later sum in parts on the stream
// would be joined too early.
#include "w4_launch.h"

#include <map>
#include <mutex>
#include <tuple>

namespace w4 {

namespace {
constexpr int kSet = kMxMaxParts / 2, kCounters = (kMxMaxSplits - 1) * kSet;  // of a number of parts, all
}  // namespace

hipError_t stream_counters(hipStream_t stream, uint32_t splits, uint32_t** out) {
  if (splits < 2 || splits > (uint32_t)kMxMaxSplits) return hipErrorInvalidValue;
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
    e = hipMalloc(reinterpret_cast<void**>(&p), kCounters * sizeof(uint32_t));
    if (e != hipSuccess) return e;
    e = launch_zero(p, kCounters, 0, stream);
    if (e != hipSuccess) {
      (void)hipFree(p);  // (nothing uses it yet)
      return e;
    }
    slot = p;
  }
  *out = slot + (splits - 2) * kSet;
  return hipSuccess;
}

}  // namespace w4
