// Host code of the layer entry points under AddressSanitizer and UBSan: every
// call's checks on extreme sizes and fake device addresses (the launchers below
// only count), and the weight packing on real memory. Prints the failures.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>
#include <vector>

#include "ssd.h"
#include "ssd_launch.hpp"

namespace {
int launches = 0, failures = 0, checks = 0;
}

namespace ssd {
hipError_t launch_conv_forward(const Dims&, int, const ConvPtrs&, const int32_t*, void*, void*, void*, void*,
                               hipStream_t) {
  return ++launches, hipSuccess;
}
hipError_t launch_conv_decode_step(const Dims&, int, bool, const ConvPtrs&, const float*, const float*,
                                   const ScalePtrs&, void*, void*, hipStream_t) {
  return ++launches, hipSuccess;
}
hipError_t launch_norm(int, int, const NormArgs&, hipStream_t) { return ++launches, hipErrorUnknown; }
hipError_t launch_matmul_i8(int, const MatmulI8Args&, hipStream_t) { return ++launches, hipSuccess; }
}  // namespace ssd

// 0: refused, nothing launched; 1: exactly one launch (whatever it returned)
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
  sh.batch = 2; sh.seqlen = 64; sh.nheads = 4; sh.headdim = 16; sh.dstate = 16; sh.ngroups = 1; sh.chunk = 64;
  sh.dtype = SSD_DTYPE_F16;
  ssd_conv cv{at<float>(A), nullptr, nullptr, 4};
  ssd_scales sc{};
  sc.s_B = sc.s_C = sc.s_X = sc.s_S = sc.inv_B = sc.inv_C = sc.inv_X = at<float>(A);
  const int64_t cd = 96;

  auto fwd = [&](const ssd_shape& s, int64_t ldx, int64_t ldt) {
    return ssd_conv_forward(&s, &cv, at(A), ldx, at(A), ldt, nullptr, nullptr, nullptr, at(A), at(A), at(A), at(A),
                            nullptr);
  };
  EXPECT(fwd(sh, cd, 4), SSD_OK, 1);
  EXPECT(fwd(sh, ((int64_t)1 << 28) - 1, ((int64_t)1 << 28) - 1), SSD_OK, 1);
  for (int64_t v : huge) {
    EXPECT(fwd(sh, v, 4), SSD_E_SHAPE, 0);
    EXPECT(fwd(sh, cd, v), SSD_E_SHAPE, 0);
  }
  for (int k = 0; k < 6; ++k) {
    ssd_shape s = sh;
    s.batch = s.seqlen = std::numeric_limits<decltype(s.batch)>::max();
    if (k & 1) s.nheads = std::numeric_limits<decltype(s.nheads)>::max();
    if (k & 2) s.ngroups = std::numeric_limits<decltype(s.ngroups)>::max();
    if (k & 4) s.batch = std::numeric_limits<decltype(s.batch)>::min();
    launches = 0;
    ++checks;
    if (fwd(s, ((int64_t)1 << 28) - 1, ((int64_t)1 << 28) - 1) == SSD_OK || launches) ++failures;
  }

  auto step = [&](const ssd_shape& s, int path, const ssd_scales* q) {
    return ssd_conv_decode_step(&s, path, &cv, at(A), ((int64_t)1 << 28) - 1, at(A), ((int64_t)1 << 28) - 1,
                                at<float>(A), at<float>(A), q, at(A), at<int32_t>(A), at(A), at(A), nullptr);
  };
  ssd_shape one = sh;
  one.seqlen = 1;
  EXPECT(step(one, SSD_PATH_FLOAT, nullptr), SSD_OK, 1);
  EXPECT(step(one, SSD_PATH_INT8, nullptr), SSD_E_NULL, 0);
  EXPECT(step(sh, SSD_PATH_FLOAT, nullptr), SSD_E_SHAPE, 0);
  one.batch = 32768; one.nheads = 512;
  EXPECT(step(one, SSD_PATH_FLOAT, nullptr), SSD_E_SHAPE, 0);
  one.nheads = 511;
  EXPECT(step(one, SSD_PATH_FLOAT, nullptr), SSD_OK, 1);

  auto norm = [&](int64_t rows, int64_t cols, int64_t ld, int64_t groups) {
    return groups ? ssd_gated_norm(rows, cols, groups, SSD_DTYPE_BF16, at(A), at(A), ld, at<float>(A), 1e-5f, at(A),
                                   nullptr, nullptr, nullptr)
                  : ssd_add_norm(rows, cols, SSD_DTYPE_BF16, at(A), ld, nullptr, 0, nullptr, at<float>(A), 1e-5f,
                                 at(A), nullptr, nullptr, nullptr);
  };
  EXPECT(norm(3, 64, 64, 0), SSD_E_HIP, 1);  // the launch's own error comes back
  EXPECT(norm(INT32_MAX, 16384, 16384, 1), SSD_E_HIP, 1);
  EXPECT(norm(0, 64, 64, 0), SSD_OK, 0);
  for (int64_t v : huge) {
    EXPECT(norm(v, 64, 64, 0), SSD_E_SHAPE, 0);
    EXPECT(norm(3, v, v, 0), SSD_E_SHAPE, 0);
    if (v > (int64_t)1 << 41 || v < 0) EXPECT(norm(INT32_MAX, 64, v, 0), SSD_E_SHAPE, 0);
    if (v > (int64_t)1 << 41 || v < 0) EXPECT(norm(INT32_MAX, 64, v, 1), SSD_E_SHAPE, 0);
    EXPECT(norm(3, 64, 64, v), SSD_E_SHAPE, 0);
  }

  auto mm = [&](int64_t m, int64_t n, int64_t k) {
    return ssd_matmul_i8(m, n, k, at<int8_t>(A), at<float>(A), at<int8_t>(A), at<float>(A), nullptr, SSD_DTYPE_F32,
                         at(A), nullptr, 0, nullptr);
  };
  EXPECT(mm(7, 9, 16), SSD_OK, 1);
  EXPECT(mm(((int64_t)1 << 26) - 1, 1 << 13, 131056), SSD_OK, 1);
  EXPECT(mm((int64_t)1 << 25, 1 << 15, 16), SSD_E_SHAPE, 0);
  EXPECT(mm(0, 9, 16), SSD_OK, 0);
  EXPECT(mm(7, 9, 24), SSD_E_UNSUPPORTED, 0);
  EXPECT(mm(7, 9, 131072), SSD_E_SHAPE, 0);
  for (int64_t v : huge) {
    EXPECT(mm(v, 9, 16), SSD_E_SHAPE, 0);
    EXPECT(mm(7, v, 16), SSD_E_SHAPE, 0);
    EXPECT(mm(7, 9, v), SSD_E_SHAPE, 0);
    EXPECT(mm(v, v, v), SSD_E_SHAPE, 0);
    ++checks;
    if (ssd_matmul_i8_workspace_bytes(v, v, v) != 0) ++failures;
  }

  // packing: rows of ordinary, subnormal, largest and zero values; buffers of the exact size
  const float kMax = std::numeric_limits<float>::max(), kSub = std::numeric_limits<float>::denorm_min();
  const std::vector<float> w = {1.f, -2.f, 0.5f, kSub, -kSub, 0.f, kMax, -kMax, 1.f, 0.f, -0.f, 0.f, 200 * kSub, kSub, -99 * kSub};
  std::vector<int8_t> q(15);
  std::vector<float> s(5);
  EXPECT(ssd_pack_weight_i8(5, 3, w.data(), q.data(), s.data()), SSD_OK, 0);
  for (size_t i = 0; i < w.size(); ++i) {
    ++checks;
    if (q[i] == -128 || std::abs(q[i] * (double)s[i / 3] - w[i]) > 0.5 * s[i / 3] * (1 + 1e-6) + 127 * kSub) {
      ++failures;
      std::printf("weight %zu: code %d step %g\n", i, q[i], s[i / 3]);
    }
  }
  std::vector<float> bad = w;
  bad[14] = std::numeric_limits<float>::infinity();
  EXPECT(ssd_pack_weight_i8(5, 3, bad.data(), q.data(), s.data()), SSD_E_VALUE, 0);
  for (int64_t v : huge) {
    if (v != (int64_t)1 << 40) EXPECT(ssd_pack_weight_i8(v, 3, w.data(), q.data(), s.data()), SSD_E_SHAPE, 0);
    EXPECT(ssd_pack_weight_i8(v, v, w.data(), q.data(), s.data()), SSD_E_SHAPE, 0);
  }
  std::printf("%d checks, %d failures\n", checks, failures);
  return failures != 0;
}
