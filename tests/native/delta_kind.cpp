// Launches of the gated delta rule's single positions on 256 CUs: for every head size and
// heads up to the most that the calls take, prints the largest thread count, whether each
// wave has its part of a head and each head all its parts, and the passes of some sizes.
#include <cstdio>
#include <initializer_list>

#include "ssd_delta_kind.hpp"

int main() {
  int64_t most = 0;
  bool whole = true;
  for (const int P : {16, 32, 64, 128})
    for (const int N : {16, 32, 64, 128})
      for (const int64_t L : {0, 1, 8, 16})
        for (int bit = 0; bit <= 23; ++bit)
          for (int64_t heads = ((int64_t)1 << bit) - 3; heads < ((int64_t)1 << bit) + 3; ++heads) {
            if (heads < 1 || heads >= (int64_t)1 << 23) continue;
            const int el = ssd::delta_step_passes(heads, L, P, N, 256), all = P * N / 256;
            const int64_t wgs = ssd::delta_step_wgs(ssd::delta_step_items(heads, P, N, el));
            whole = whole && el >= 1 && el <= 8 && all % el == 0 && wgs * ssd::kDeltaStepWaves * el >= heads * all;
            const int64_t threads = wgs * ssd::kDeltaStepWaves * 64;
            most = threads > most ? threads : most;
          }
  std::printf("%lld %d", (long long)most, whole);
  for (const int64_t heads : {64, 320, 20480, 1 << 22})
    std::printf(" %d", ssd::delta_step_passes(heads, 1, 64, 128, 256));
  std::printf(" %d\n", ssd::delta_step_passes((1 << 22) + 1, 1, 128, 128, 256));
  return 0;
}
