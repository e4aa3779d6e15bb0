// The gated delta rule's launch of single positions (without HIP: a test asks it for its
// thread counts).
#pragma once

#include <cstdint>

namespace ssd {

constexpr int kDeltaStepWaves = 4;  // of a workgroup

// Passes of a wave (256 elements of the state each): four, fewer where that leaves CUs
// without 8 waves (us of a step at 1, 2, 4, 8 and 16 passes, heads of 64 x 128: 64 heads 4.1,
// 4.0, 4.1, 4.6 and 5.6; 320 heads 8.9, 6.8, 5.7, 6.1 and 6.6; 20480 heads 362, 220, 221, 241
// and 234); eight for more than one position where waves are many, which share a position's
// loads and sums (5120 heads, 8 positions: 132 at 4, 111 at 8, 134 at 16; 640 heads 21.4,
// 21.8 and 27), and where four would come to 2^32 threads, which is more than a launch holds
// (2^22 heads of 128 x 128 without a state before or after; at eight 2^23 heads stay below it).
inline int delta_step_passes(int64_t heads, int64_t L, int P, int N, int64_t ncu) {
  const int all = P * N / 256;  // passes of a head: 1 to 64
  int el = (L > 1 && heads * (all / 8) >= 32 * ncu) || heads * all >= (int64_t)1 << 28 ? 8 : 4;
  while (el > 1 && (el > all || heads * (all / el) < 8 * ncu)) el /= 2;
  return el;
}
// Waves, each of them el passes of a head, and their workgroups.
inline int64_t delta_step_items(int64_t heads, int P, int N, int el) { return heads * (P * N / 256 / el); }
inline int64_t delta_step_wgs(int64_t items) { return (items + kDeltaStepWaves - 1) / kDeltaStepWaves; }

}  // namespace ssd
