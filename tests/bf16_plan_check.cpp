// Which kernel the bfloat16 linears' rule (csrc/launch_bf16.h) chooses, for tests/test_bf16_plans.py.
// Reads lines "T N K groups gated" (0 groups: a dense product), prints the kernel's number for
// each; after the line "sweep" prints "number gated grouped" of every kernel that sizes spread
// over the supported range reach.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <random>
#include <set>
#include <tuple>

#include "launch_bf16.h"

namespace {

int plan(long T, long N, long K, int groups, bool gated) {
  static const int32_t some[1] = {0};
  moe::Bf16Args a{};
  a.T = (int)T;
  a.N = (int)N;
  a.K = (int)K;
  a.E = groups > 0 ? groups : 1;
  a.offsets = groups > 0 ? some : nullptr;
  return moe::bf16_plan(gated, a);
}

}  // namespace

int main() {
  char line[256];
  while (fgets(line, sizeof line, stdin)) {
    if (strncmp(line, "sweep", 5) == 0) {
      std::mt19937_64 rng(1);
      auto spread = [&](double high) { return (long)lround(exp(log(high) * (double)(rng() >> 11) * 0x1p-53)); };
      std::set<std::tuple<int, bool, bool>> seen;
      for (int i = 0; i < 400000; ++i) {
        const bool gated = rng() & 1, grouped = rng() & 1;
        const int groups = grouped ? (int)spread(512) : 0;
        const long K = 8 * spread(8192), N = spread(1 << 18), T = spread(1 << 24);
        seen.insert({plan(T, N, K, groups, gated), gated, grouped});
      }
      for (const auto& [p, gated, grouped] : seen) printf("%d %d %d\n", p, gated, grouped);
      return 0;
    }
    long T, N, K;
    int groups, gated;
    if (sscanf(line, "%ld %ld %ld %d %d", &T, &N, &K, &groups, &gated) != 5) return 1;
    printf("%d\n", plan(T, N, K, groups, gated != 0));
  }
  return 0;
}
