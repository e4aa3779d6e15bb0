// The kernel that the 8-bit product takes on 256 CUs, for sizes "M N K" a line on
// stdin: its index, block rows and columns, and round of K.
#include <cstdio>

#include "ssd_matmul_kind.hpp"

int main() {
  long long m, n, k;
  while (std::scanf("%lld %lld %lld", &m, &n, &k) == 3) {
    const int i = ssd::pick_matmul_kind(m, n, k, 256);
    const ssd::MatmulKind& q = ssd::kMatmulKind[i];
    std::printf("%d %d %d %d\n", i, q.rows, q.cols, q.round);
  }
  return 0;
}
