// Device workspaces kept by the library per (device, stream, user).
//
// A matrix-product call that needs scratch memory (packed activations, k-split
// partial sums) takes it from here: the buffer is allocated on first use and
// replaced by a larger one when a call needs more.  A replaced buffer is
// never freed: kernels enqueued earlier on the stream, and HIP graphs captured
// earlier, may still read and write it, and freeing it would need a wait for
// the stream.  Each replacement at least doubles the size, so the buffers a
// (device, stream, user) ever holds add up to less than twice the largest.
// Calls on one stream are ordered and share the current buffer (calls of several
// host threads too: those of more than one launch take turns); calls on
// different streams never share one: hipStreamPerThread is a stream of its own
// in each thread under one handle, so its buffers are the thread's.  Nothing is
// released before the process ends, also for streams the caller has destroyed
// and threads that have ended.
#include "w4_launch.h"

#include <atomic>
#include <map>
#include <mutex>
#include <tuple>

namespace w4 {

uint64_t this_thread() {
  static std::atomic<uint64_t> threads{0};
  thread_local const uint64_t id = ++threads;
  return id;
}

std::unique_lock<std::mutex> stream_turn(hipStream_t stream) {
  static std::mutex mu;
  // (kept to the end: a thread may still enqueue while the process ends)
  static auto& turns = *new std::map<std::tuple<int, hipStream_t, uint64_t>, std::mutex>;
  int dev = -1;
  (void)hipGetDevice(&dev);  // (where it fails, so does the lookup of the workspace)
  const uint64_t thread = stream == hipStreamPerThread ? this_thread() : 0;
  std::mutex* turn;
  {
    std::lock_guard<std::mutex> g(mu);
    turn = &turns[std::make_tuple(dev, stream, thread)];  // (a map's elements stay where they are)
  }
  return std::unique_lock<std::mutex>(*turn);
}

hipError_t stream_workspace(int user, hipStream_t stream, size_t bytes, char** out) {
  static std::mutex mu;
  static std::map<std::tuple<int, hipStream_t, uint64_t, int>, std::pair<char*, size_t>> cache;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t thread = stream == hipStreamPerThread ? this_thread() : 0;
  std::lock_guard<std::mutex> g(mu);
  auto& slot = cache[std::make_tuple(dev, stream, thread, user)];
  if (slot.second < bytes) {
    size_t want = bytes;
    if (want < 2 * slot.second) want = 2 * slot.second;
    char* p = nullptr;
    e = hipMalloc(reinterpret_cast<void**>(&p), want);
    if (e != hipSuccess) return e;
    slot = {p, want};  // the old buffer stays allocated (see above)
  }
  *out = slot.first;
  return hipSuccess;
}

}  // namespace w4
