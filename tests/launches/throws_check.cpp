// Where memory runs out on the host, in a stream's first call (which enters it in the
// library's tables) or in a plan, no exception passes the C boundary: the call returns
// a status, and the same call works when memory is back.
#include "fake_hip.h"

#include <new>

#include "w4.h"
#include "w4_launch.h"

namespace {
bool g_empty = false;
int g_refused = 0;
}  // namespace

void* operator new(size_t bytes) {
  if (g_empty) {
    ++g_refused;
    throw std::bad_alloc();
  }
  if (void* p = malloc(bytes ? bytes : 1)) return p;
  throw std::bad_alloc();
}
void operator delete(void* p) noexcept { free(p); }
void operator delete(void* p, size_t) noexcept { free(p); }

namespace {
uint16_t* H(uintptr_t a) { return reinterpret_cast<uint16_t*>(a); }
uint8_t* P(uintptr_t a) { return reinterpret_cast<uint8_t*>(a); }
const uintptr_t A = 0x100000;
w4_gemv_problem problems[2];

struct Kind {
  const char* name;
  int (*call)(hipStream_t);
};
const Kind kinds[] = {
    {"w4_gemm",
     [](hipStream_t s) -> int { return w4_gemm(W4_DYADIC, 256, 4096, P(A), H(A), nullptr, H(A), 64, P(A), W4_F32, s); }},
    {"w4_gemm_noalloc",
     [](hipStream_t s) -> int {
       return w4_gemm_noalloc(W4_DYADIC, 256, 4096, P(A), H(A), nullptr, H(A), 64, P(A), W4_F32, s);
     }},
    {"w4_gemv",
     [](hipStream_t s) -> int { return w4_gemv(W4_DYADIC, 4096, 4096, P(A), H(A), nullptr, H(A), 16, P(A), W4_F32, s); }},
    {"w4_linear",
     [](hipStream_t s) -> int {
       return w4_linear(W4_DYADIC, 256, 4096, P(A), H(A), nullptr, H(A), 64, P(A), W4_F32, s);
     }},
    {"w4_gemv_batched_plan",
     [](hipStream_t) -> int {
       for (w4_gemv_problem& p : problems) p = {P(A), H(A), nullptr, H(A), P(A), 256, 4096, 0};
       w4_gemv_batch_info info;
       return w4_gemv_batched_plan(W4_DYADIC, 1, W4_F32, problems, 2, &info);
     }},
    {"w4_mx_linear",
     [](hipStream_t s) -> int { return w4_mx_linear(W4_MXFP8, 256, 8192, P(A), P(A), P(A), P(A), 64, P(A), W4_F32, s); }},
    {"w4_mx_linear_grad",
     [](hipStream_t s) -> int { return w4_mx_linear_grad(1001, 512, P(A), P(A), H(A), 40, P(A), W4_F32, s); }},
    {"w4_mx_gated_linear_grad",
     [](hipStream_t s) -> int {
       return w4_mx_gated_linear_grad(W4_SILU, 1001, 512, P(A), P(A), H(A), H(A), 40, H(A), P(A), W4_F32, s);
     }},
    // calls that name the kernel
    {"w4_mx_product_on",
     [](hipStream_t s) -> int {
       return w4::w4_mx_product_on(16 * 2 + 1, 1, 0, 256, 8192, P(A), P(A), 64, P(A), P(A), 64, nullptr, nullptr, P(A), 1, s);
     }},
    {"w4_mx_bf16_product_on",
     [](hipStream_t s) -> int {
       return w4::w4_mx_bf16_product_on(16 * 2 + 3, w4::kMxForward, 0, 256, 8192, P(A), P(A), H(A), 64, nullptr, P(A), 1, s);
     }},
};
}  // namespace

int main() {
  uintptr_t stream = 0x10000;
  for (const Kind& k : kinds) {
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream += 0x100);  // new to the library
    int launches = 0;
    fake::on_launch = [&](const std::string&, void**, hipStream_t) { ++launches; };
    g_refused = 0;
    g_empty = true;
    int status = 0;
    bool thrown = false;
    try {
      status = k.call(s);
    } catch (...) {
      thrown = true;
    }
    g_empty = false;
    if (thrown || !g_refused || !status || launches)
      fprintf(stderr, "%s: thrown %d, refused %d, status %d, launches %d\n", k.name, thrown, g_refused, status, launches);
    EXPECT(!thrown);
    EXPECT(g_refused > 0);  // (it did ask for memory)
    EXPECT(status != 0 && launches == 0);
    EXPECT(k.call(s) == 0);
  }
  if (fake::failures) {
    fprintf(stderr, "%d failures\n", fake::failures);
    return 1;
  }
  printf("throws_check ok\n");
  return 0;
}
