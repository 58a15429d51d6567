// Calls of two host threads on one stream: a call that fills a workspace and reads it
// in a later launch has nothing of another call between its launches.  Calls on
// different streams do not wait for one another.
#include "fake_hip.h"

#include <chrono>
#include <condition_variable>
#include <mutex>
#include <thread>
#include <utility>
#include <vector>

#include "w4.h"

namespace {
uint16_t* H(uintptr_t a) { return reinterpret_cast<uint16_t*>(a); }
uint8_t* P(uintptr_t a) { return reinterpret_cast<uint8_t*>(a); }
const uintptr_t A = 0x100000;

struct Kind {
  const char* name;
  w4_status (*call)(hipStream_t);
};
// sizes at which each takes two launches or three
const Kind kinds[] = {
    {"w4_gemm", [](hipStream_t s) { return w4_gemm(W4_DYADIC, 256, 4096, P(A), H(A), nullptr, H(A), 64, P(A), W4_F32, s); }},
    {"w4_gemm_noalloc",
     [](hipStream_t s) { return w4_gemm_noalloc(W4_DYADIC, 256, 4096, P(A), H(A), nullptr, H(A), 64, P(A), W4_F32, s); }},
    {"w4_gemv", [](hipStream_t s) { return w4_gemv(W4_DYADIC, 4096, 4096, P(A), H(A), nullptr, H(A), 16, P(A), W4_F32, s); }},
    {"w4_mx_linear",
     [](hipStream_t s) { return w4_mx_linear(W4_MXFP8, 256, 8192, P(A), P(A), P(A), P(A), 64, P(A), W4_F32, s); }},
    {"w4_mx_linear_grad",
     [](hipStream_t s) { return w4_mx_linear_grad(1001, 512, P(A), P(A), H(A), 40, P(A), W4_F32, s); }},
    {"w4_mx_gated_linear_grad",
     [](hipStream_t s) {
       return w4_mx_gated_linear_grad(W4_SILU, 1001, 512, P(A), P(A), H(A), H(A), 40, H(A), P(A), W4_F32, s);
     }},
};

std::mutex mu;
thread_local int this_call = 0;  // a number for each call
std::vector<std::pair<std::thread::id, int>> log_;

void one_stream(const Kind& kind) {
  log_.clear();
  fake::on_launch = [](const std::string&, void**, hipStream_t) {
    {
      std::lock_guard<std::mutex> g(mu);
      log_.push_back({std::this_thread::get_id(), this_call});
    }
    std::this_thread::sleep_for(std::chrono::microseconds(200));
  };
  const hipStream_t s = reinterpret_cast<hipStream_t>(0x10000);
  constexpr int kCalls = 20;
  auto work = [&] {
    for (this_call = 0; this_call < kCalls; ++this_call) EXPECT(kind.call(s) == W4_OK);
  };
  std::thread a(work), b(work);
  a.join();
  b.join();
  EXPECT(log_.size() >= 2 * 2 * kCalls);
  int runs = 0;  // of launches of one call
  for (size_t i = 0; i < log_.size(); ++i) runs += i == 0 || log_[i] != log_[i - 1];
  if (runs != 2 * kCalls) fprintf(stderr, "%s: %d runs of launches for %d calls\n", kind.name, runs, 2 * kCalls);
  EXPECT(runs == 2 * kCalls);
}

void two_streams(const Kind& kind) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(0x10000), t = reinterpret_cast<hipStream_t>(0x20000);
  static std::condition_variable other;
  static bool seen, started;
  seen = started = false;
  fake::on_launch = [=](const std::string&, void**, hipStream_t on) {
    std::unique_lock<std::mutex> g(mu);
    if (on == t) {
      seen = true;
    } else {  // inside its call until the other stream's is enqueued
      started = true;
      other.notify_all();
      EXPECT(other.wait_for(g, std::chrono::seconds(10), [] { return seen; }));
    }
    other.notify_all();
  };
  std::thread a([&] { EXPECT(kind.call(s) == W4_OK); });
  std::thread b([&] {
    {
      std::unique_lock<std::mutex> g(mu);
      other.wait_for(g, std::chrono::seconds(10), [] { return started; });
    }
    EXPECT(kind.call(t) == W4_OK);
  });
  a.join();
  b.join();
}
}  // namespace

int main() {
  // (a stream's first call makes its workspace and counters)
  for (const Kind& k : kinds)
    for (uintptr_t s : {0x10000, 0x20000}) EXPECT(k.call(reinterpret_cast<hipStream_t>(s)) == W4_OK);
  for (const Kind& k : kinds) {
    one_stream(k);
    two_streams(k);
  }
  if (fake::failures) {
    fprintf(stderr, "%d failures\n", fake::failures);
    return 1;
  }
  printf("turns_check ok\n");
  return 0;
}
