// Host-side check of the library's stream workspaces (w4_workspace.cpp), built
// with AddressSanitizer and UndefinedBehaviorSanitizer on the CPU with stubs of
// the HIP calls: who shares a buffer with whom.  Built and run by
// tests/test_workspace.py.
#include <stdio.h>
#include <stdlib.h>

#include <atomic>
#include <thread>

#include "w4_launch.h"

namespace {
std::atomic<int> g_allocations{0};
}  // namespace

extern "C" hipError_t hipGetDevice(int* dev) {
  *dev = 0;
  return hipSuccess;
}
extern "C" hipError_t hipMalloc(void** p, size_t) {
  *p = reinterpret_cast<void*>((uintptr_t)0x1000 * (uintptr_t)++g_allocations);
  return hipSuccess;
}

namespace {
int failures = 0;
#define EXPECT(c)                                            \
  do {                                                       \
    if (!(c)) {                                              \
      fprintf(stderr, "FAIL line %d: %s\n", __LINE__, #c);   \
      ++failures;                                            \
    }                                                        \
  } while (0)

char* get(hipStream_t s, size_t bytes, int user = w4::kWorkspaceMx) {
  char* p = nullptr;
  EXPECT(w4::stream_workspace(user, s, bytes, &p) == hipSuccess && p);
  return p;
}
char* get_on_thread(hipStream_t s, size_t bytes) {
  char* p = nullptr;
  std::thread([&] { p = get(s, bytes); }).join();
  return p;
}
}  // namespace

int main() {
  const hipStream_t a = reinterpret_cast<hipStream_t>(0x10000), b = reinterpret_cast<hipStream_t>(0x20000);
  char* const pa = get(a, 100);
  EXPECT(get(a, 50) == pa && get(a, 100) == pa);
  EXPECT(get(b, 50) != pa && get(nullptr, 50) != pa);
  EXPECT(get(a, 100, w4::kWorkspaceGemv) != pa);
  char* const grown = get(a, 101);
  EXPECT(grown != pa && get(a, 200) == grown);  // (at least doubled)
  EXPECT(get_on_thread(a, 200) == grown);       // a stream's buffer, whoever calls
  // one handle, another stream in each thread: in one that has ended, too
  char* const mine = get(hipStreamPerThread, 64);
  char* const first = get_on_thread(hipStreamPerThread, 64);
  char* const second = get_on_thread(hipStreamPerThread, 64);
  EXPECT(mine != first && mine != second && first != second);
  EXPECT(get(hipStreamPerThread, 64) == mine);
  if (failures) {
    fprintf(stderr, "%d failures\n", failures);
    return 1;
  }
  printf("workspace_check ok\n");
  return 0;
}
