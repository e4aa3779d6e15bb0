// The 8-bit product's choice of kernel (host code without HIP: a test lists what its
// sizes reach).
#pragma once

#include <cstdint>

namespace ssd {

// Which kernel takes a product: the one whose time, a + rounds (b + c K / 1024)
// us, comes out least. A round is as many workgroups as the chip holds at once
// (256 CUs, or twice that where two fit a CU's LDS); the few-rows kernels of two
// workgroups a CU fill in between rounds, the others finish whole rounds. K is
// taken up to whole rounds of a kernel's buffers. The constants are fits to 300
// products over 1 to 16384 rows, N from 17 to 18000 and K from 64 to 8192, of
// which half have odd sizes; over 200 others the choice is 1.1 % above the best
// kernel's time in the geometric mean, 30 % at most. Where they cross, for
// example (us, the chosen first): 8 x 2560 x 5120 4.4 at 16 x 16, 5.7 at 32 x 32;
// 64 x 10576 x 2560 9.5 at 32 x 32, 16.4 at 16 x 16, 10.0 at 64 x 64; 333 x 2560 x 5120 12.0
// at 64 x 64, 16.4 at 32 x 32, 20.5 at 128; 333 x 8512 x 2048 12.6 at 128, 22.6
// at 32 x 32, 27 at 256; 4096 x 2048 x 1024 15.8 at 128 with two workgroups a CU,
// 18.5 with one, 22 at 256; 4096 x 4096 x 4096 62 at 256, 71 and 75 at 128;
// 16384 x 2560 x 5120 224 at 256, 257 at 128.
struct MatmulKind {
  int rows, cols;  // of a workgroup's block
  int per_cu;      // workgroups
  int round;       // of K: what a round of the buffers holds, or one piece of all waves
  float a, b, c;
};
constexpr int kMatmulKinds = 7;
constexpr MatmulKind kMatmulKind[kMatmulKinds] = {
    {16, 16, 2, 1024, 2.2f, 1.7f, 0.45f},  {16, 32, 2, 512, 2.8f, 1.2f, 1.12f},
    {32, 32, 2, 512, 3.3f, 0.8f, 1.61f},   {64, 64, 1, 512, 0.4f, 5.5f, 1.40f},
    {128, 128, 1, 512, 2.3f, 3.8f, 3.70f}, {128, 128, 2, 256, 0.2f, 4.4f, 6.35f},
    {256, 256, 1, 256, 1.7f, 11.3f, 9.58f},
};

inline int pick_matmul_kind(int64_t M, int64_t N, int64_t K, int64_t ncu) {
  int best = 0;
  float least = 0.f;
  for (int i = 0; i < kMatmulKinds; ++i) {
    const MatmulKind& q = kMatmulKind[i];
    if (q.rows >= 128 && (M < q.rows || N < q.cols)) continue;  // tiles lie inside the matrix
    const int64_t blocks = ((M + q.rows - 1) / q.rows) * ((N + q.cols - 1) / q.cols);
    const int64_t slots = ncu * q.per_cu;
    const float rounds = q.rows < 64 ? (float)blocks / (float)slots : (float)((blocks + slots - 1) / slots);
    const float us = q.a + rounds * (q.b + q.c * (float)((K + q.round - 1) / q.round * q.round) / 1024.f);
    if (i == 0 || us < least) {
      best = i;
      least = us;
    }
  }
  return best;
}

}  // namespace ssd
