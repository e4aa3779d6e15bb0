// Bounds of the gated delta rule's scales over all of fp32: prints what a scale brings a
// largest value to at least and at most, and the largest state that a chunk can leave.
#include <cmath>
#include <cstdio>
#include <initializer_list>

#include "ssd_delta_scale.hpp"

int main() {
  float least = 1e30f, most = 0.f, state = 0.f;
  bool inverse = true;
  for (int e = -149; e < 128; ++e)
    for (const float f : {1.f, 1.0001f, 1.5f, 1.9999f, 2.f - 0x1p-23f}) {
      const float m = std::ldexp(f, e);
      if (m == 0.f || std::isinf(m)) continue;
      for (const bool wide : {false, true}) {
        const ssd::Scale s = wide ? ssd::Scale(m, ssd::kWide) : ssd::Scale(m);
        inverse = inverse && s.by * s.inv == 1.f;
        const float v = m * s.by;
        if (m >= (wide ? 0x1p-110f : 0x1p-82f)) least = std::fmin(least, v);
        most = std::fmax(most, v);
      }
      // a chunk whose changes and keys are the largest, on a state that is as large as they allow
      for (const float keeps : {0.f, 0.25f, 0.5f, 1.f}) {
        if (m > 0x1p100f) continue;
        const float before = keeps / ssd::kStateDown * m;
        const ssd::Scale sc(std::fmax(before * ssd::kStateDown, m), ssd::kWide);
        const float key = (2.f - 0x1p-23f) * ssd::Scale(2.f - 0x1p-23f).by;
        state = std::fmax(state, (before * sc.by + 64.f * (m * sc.by) * key) * ssd::kStateDown);
      }
    }
  std::printf("%d %.9g %.9g %.9g %.9g %.9g\n", inverse, least, most, ssd::kScaledMost, state, ssd::kStateMost);
  return 0;
}
