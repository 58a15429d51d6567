// The counters of sums in parts (w4_counters.cpp), whose launches on one stream share
// them: where launches overlap, which replays of captured calls can, whatever order
// their blocks count in, every counter is back at zero when they have all ended.
// (The overlapping calls' own results are lost; later calls' must not be.)
#include "fake_hip.h"

#include <algorithm>
#include <random>
#include <utility>
#include <vector>

#include "w4_launch.h"

namespace {
// as in w4_mx_bf16_gemm.hip and w4_mx_bf16_narrow.hip
struct GemmArgs {
  uint32_t tiles_m, tiles_n, whole, splits;
  uint64_t* partial;
  uint32_t* counted;
};
struct NarrowArgs {
  uint32_t tiles_m, tiles_n, splits;
  uint64_t* partial;
  uint32_t* counted;
};

struct Counts {
  uint32_t* first;
  uint32_t tiles, splits;
};
std::vector<Counts> launched;

void note(const std::string& kernel, void** args, hipStream_t) {
  if (kernel.find("mx_bf16_gemm_kernel") != std::string::npos) {
    const GemmArgs& g = *static_cast<GemmArgs*>(args[1]);
    if (g.splits > 1) launched.push_back({g.counted, g.tiles_m * g.tiles_n - g.whole, g.splits});
  } else if (kernel.find("mx_bf16_narrow_kernel") != std::string::npos) {
    const NarrowArgs& g = *static_cast<NarrowArgs*>(args[1]);
    if (g.splits > 1) launched.push_back({g.counted, g.tiles_m * g.tiles_n, g.splits});
  }
}

uint16_t* H(uintptr_t a) { return reinterpret_cast<uint16_t*>(a); }
uint8_t* P(uintptr_t a) { return reinterpret_cast<uint8_t*>(a); }

// the counting of the launches, their blocks' turns drawn at random
void count(const std::vector<Counts>& launches, std::mt19937& rng) {
  std::vector<std::pair<uint32_t*, uint32_t>> turns;
  for (const Counts& c : launches)
    for (uint32_t t = 0; t < c.tiles; ++t)
      for (uint32_t s = 0; s < c.splits; ++s) turns.push_back({c.first + t, c.splits - 1});
  std::shuffle(turns.begin(), turns.end(), rng);
  for (const auto& t : turns) *t.first = *t.first >= t.second ? 0 : *t.first + 1;  // atomicInc
}
}  // namespace

int main() {
  fake::on_launch = note;
  const uintptr_t A = 0x100000;
  const hipStream_t s = reinterpret_cast<hipStream_t>(0x10000), other = reinterpret_cast<hipStream_t>(0x20000);
  std::mt19937 rng(1);
  auto product = [&](int kernel, int kind, int64_t n, int64_t k, int64_t m, hipStream_t on) {
    return w4::w4_mx_bf16_product_on(kernel, kind, 0, n, k, P(A), P(A), H(A), m, nullptr, P(A), 1, on);
  };
  for (int a = 2; a <= 16; ++a)
    for (int b = 2; b <= 16; ++b) {
      launched.clear();
      // forward on 64 x 128 tiles, backward on the narrow kernel's, and a tail
      EXPECT(product(16 * a + 3, w4::kMxForward, 1000, 2080, 300, s) == 0);
      EXPECT(product(16 * b + 4, w4::kMxBackward, 2080, 1024, 96, s) == 0);
      EXPECT(product(1024 + 16 * a + 2, w4::kMxGated, 1100, 1312, 600, s) == 0);
      EXPECT(launched.size() == 3);
      for (int i = 0; i < 4; ++i) {
        count(launched, rng);
        uint32_t left = 0;
        for (const Counts& c : launched)
          for (uint32_t t = 0; t < c.tiles; ++t) left += c.first[t];
        if (left) fprintf(stderr, "%d and %d parts leave counts behind\n", a, b);
        EXPECT(left == 0);
      }
    }
  // one stream's counters are its own
  const Counts here = launched.back();
  launched.clear();
  EXPECT(product(1024 + 16 * here.splits + 2, w4::kMxGated, 1100, 1312, 600, other) == 0);
  EXPECT(launched.size() == 1 && launched[0].first != here.first);
  // as many tiles in parts as a launch may have: sets lie apart, inside the allocation
  launched.clear();
  EXPECT(product(16 * 2 + 4, w4::kMxForward, 64 * 512, 4096, 32, s) == 0);
  EXPECT(launched.size() == 1 && launched[0].tiles == 512);
  if (fake::failures) {
    fprintf(stderr, "%d failures\n", fake::failures);
    return 1;
  }
  printf("counters_check ok\n");
  return 0;
}
