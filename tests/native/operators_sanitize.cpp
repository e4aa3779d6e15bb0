// Host code of the operators' entry points under AddressSanitizer and UBSan: every
// call's checks on extreme sizes and fake device addresses (the launchers below only
// count). Prints the failures.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>

#include "ssd.h"
#include "ssd_launch.hpp"

namespace {
int launches = 0, failures = 0, checks = 0;
}

namespace ssd {
hipError_t launch_delta_steps(const Dims&, int, const DeltaArgs&, hipStream_t) { return ++launches, hipSuccess; }
hipError_t launch_delta_chunks(const Dims&, int, const DeltaArgs&, void*, hipStream_t) { return ++launches, hipErrorUnknown; }
size_t delta_workspace_bytes(const Dims&, int) { return 1000; }
hipError_t launch_matmul(int, int, const MatmulArgs&, void*, hipStream_t) { return ++launches, hipSuccess; }
size_t matmul_workspace_bytes(int64_t, int64_t, int64_t, int) { return 1000; }
hipError_t launch_block_norm(int, int, const BlockNormArgs&, hipStream_t) { return ++launches, hipErrorUnknown; }
}  // namespace ssd

#define EXPECT(call, rc_, n_)                                                          \
  do {                                                                                 \
    launches = 0;                                                                      \
    const int got = (call);                                                            \
    ++checks;                                                                          \
    if (got != (rc_) || launches != (n_)) {                                            \
      ++failures;                                                                      \
      std::printf("line %d: status %d, launches %d\n", __LINE__, got, launches);       \
    }                                                                                  \
  } while (0)

template <typename T = void>
T* at(uintptr_t a) { return reinterpret_cast<T*>(a); }

int main() {
  const uintptr_t A = 0x10000;
  const int64_t huge[] = {INT64_MAX, INT64_MAX / 2, (int64_t)1 << 62, (int64_t)1 << 40, INT64_MIN, -1};
  ssd_shape sh{};
  sh.batch = 2; sh.seqlen = 64; sh.nheads = 4; sh.headdim = 128; sh.dstate = 16; sh.ngroups = 1; sh.chunk = 64;
  sh.dtype = SSD_DTYPE_F16;
  auto fwd = [&](const ssd_shape& s, int64_t ld, float scale, void* ws, size_t wsb, float* fin) {
    return ssd_delta_forward(&s, 3, at(A), at(A), at<float>(A), at(A), at(A), at(A), ld, scale, 1e-6f, at(A), nullptr, fin,
                             ws, wsb, nullptr);
  };
  EXPECT(fwd(sh, 4, 1.f, at(A), 1000, nullptr), SSD_E_HIP, 1);
  EXPECT(fwd(sh, 4, 1.f, at(A), 999, nullptr), SSD_E_WORKSPACE, 0);
  EXPECT(fwd(sh, 4, NAN, at(A), 1000, nullptr), SSD_E_SHAPE, 0);
  EXPECT(fwd(sh, 4, std::numeric_limits<float>::infinity(), at(A), 1000, nullptr), SSD_E_SHAPE, 0);
  ssd_shape s = sh;
  s.seqlen = 16;
  EXPECT(fwd(s, 4, 1.f, nullptr, 0, nullptr), SSD_OK, 1);
  s.seqlen = 0;
  EXPECT(fwd(s, 4, 1.f, nullptr, 0, at<float>(A)), SSD_OK, 1);
  EXPECT(fwd(s, 4, 1.f, nullptr, 0, nullptr), SSD_OK, 0);
  s.batch = 0;
  EXPECT(fwd(s, 4, 1.f, nullptr, 0, at<float>(A)), SSD_OK, 0);
  for (int64_t v : huge) {
    for (int k = 0; k < 7; ++k) {
      s = sh;
      int64_t* const f[] = {&s.batch, &s.seqlen, &s.nheads, &s.headdim, &s.dstate, &s.ngroups, &s.chunk};
      *f[k] = v;
      launches = 0;
      const int rc = fwd(s, 4, 1.f, at(A), 1000, nullptr);
      ++checks;
      if (rc == SSD_OK || launches) ++failures, std::printf("shape field %d: %d\n", k, rc);
      ssd_delta_workspace_bytes(&s);
    }
    EXPECT(fwd(sh, v, 1.f, at(A), 1000, nullptr), SSD_E_SHAPE, 0);
    launches = 0;
    EXPECT(ssd_matmul(v, 16, 64, 1, at(A), 64, at(A), nullptr, 0, nullptr, 1, at(A), nullptr, 0, nullptr), SSD_E_SHAPE, 0);
    EXPECT(ssd_matmul(16, v, 64, 1, at(A), 64, at(A), nullptr, 0, nullptr, 1, at(A), nullptr, 0, nullptr), SSD_E_SHAPE, 0);
    EXPECT(ssd_matmul(16, 16, v, 1, at(A), 64, at(A), nullptr, 0, nullptr, 1, at(A), nullptr, 0, nullptr), SSD_E_SHAPE, 0);
    EXPECT(ssd_matmul(16, 16, 64, 1, at(A), v, at(A), nullptr, 0, nullptr, 1, at(A), nullptr, 0, nullptr), SSD_E_SHAPE, 0);
    ssd_matmul_workspace_bytes(v, v, v, 1);
    EXPECT(ssd_block_norm(v, 64, 1, at(A), 64, at<float>(A), nullptr, 0, 1, 0, nullptr, 1.f, 1, nullptr, at<float>(A), 0.f,
                          at(A), nullptr, nullptr, nullptr), SSD_E_SHAPE, 0);
    if (v < (int64_t)1 << 50) continue;
    EXPECT(ssd_block_norm(1 << 20, 64, 1, at(A), v, at<float>(A), nullptr, 0, 1, 0, nullptr, 1.f, 1, nullptr, at<float>(A),
                          0.f, at(A), nullptr, nullptr, nullptr), SSD_E_SHAPE, 0);
    EXPECT(ssd_block_norm(1 << 20, 64, 1, at(A), 64, at<float>(A), at(A), v, 1, 0, nullptr, 1.f, 1, nullptr, at<float>(A),
                          0.f, at(A), nullptr, nullptr, nullptr), SSD_E_SHAPE, 0);
  }
  ssd_shape one = sh;
  one.seqlen = 1;
  EXPECT(ssd_delta_step(&one, 0, at(A), at(A), at<float>(A), at(A), at(A), at(A), 4, 1.f, 0.f, at<float>(A), at(A), nullptr),
         SSD_OK, 1);
  EXPECT(ssd_delta_step(&sh, 0, at(A), at(A), at<float>(A), at(A), at(A), at(A), 4, 1.f, 0.f, at<float>(A), at(A), nullptr),
         SSD_E_SHAPE, 0);
  EXPECT(ssd_matmul(16, 16, 65, 1, at(A), 65, at(A), nullptr, 0, nullptr, 1, at(A), at(A), 999, nullptr), SSD_E_WORKSPACE, 0);
  EXPECT(ssd_matmul(16, 16, 65, 1, at(A), 65, at(A), nullptr, 0, nullptr, 1, at(A), at(A), 1000, nullptr), SSD_OK, 1);
  EXPECT(ssd_matmul(16, 16, 64, 1, at(A), 64, at(A), nullptr, 0, nullptr, 1, at(A), at(A), 0, nullptr), SSD_OK, 1);
  EXPECT(ssd_block_norm(5, 64, 1, at(A), 64, at<float>(A), at(A), 64, INT64_MAX, 3, nullptr, 1.f, 1, nullptr, at<float>(A),
                        0.f, at(A), nullptr, nullptr, nullptr), SSD_E_HIP, 1);
  std::printf("%d checks, %d failures\n", checks, failures);
  return failures != 0;
}
