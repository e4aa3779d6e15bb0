// The powers of two that bring the gated delta rule's operands into fp16's range (without
// HIP as well: a test asks them for their bounds).
#pragma once

#include <cstdint>

#ifdef __HIPCC__
#define SSD_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SSD_HOST_DEVICE inline
#endif

namespace ssd {

// The power of two that brings m to [2^8, 2^9), and its inverse; from 2^-82 on down it
// is 2^90, so that products of two of them stay in fp32's range. Values and states, whose
// scales are not multiplied, have theirs (kWide) down to 2^-110.
constexpr int kWide = 127 + 118;
struct Scale {
  float by, inv;
  SSD_HOST_DEVICE explicit Scale(float m, int most = 127 + 90) {
    const int up = 262 - (int)((__builtin_bit_cast(uint32_t, m) >> 23) & 255), e = up < most ? up : most;
    by = __builtin_bit_cast(float, (uint32_t)e << 23);
    inv = __builtin_bit_cast(float, (uint32_t)(254 - e) << 23);
  }
  // of by: -120 to 90
  SSD_HOST_DEVICE int exponent() const { return (int)(__builtin_bit_cast(uint32_t, by) >> 23) - 127; }
};
// What a scaled value is below, and at most once it is rounded to fp16.
constexpr float kScaledMost = 512.f;

// The scaled state takes the products of a chunk as they come: 64 terms, each a key times a
// change, both at most kScaledMost. Before them it is at most kScaledMost / kStateDown, and
// times kStateDown it is an operand of the next chunk, which has to stay below fp16's 65504:
// 2^9 + 64 * 2^18 * 2^-9 = 33280. (Changes scaled to 1 instead, so that the state needs no
// factor, would lose what is below 2^-25 of a column's largest, not 2^-33; the factor costs 2 %
// of the scan.)
constexpr float kStateDown = 1.f / 512.f;
constexpr float kStateMost = kScaledMost + 64 * kScaledMost * kScaledMost * kStateDown;
static_assert(kStateMost < 65504.f, "the state leaves fp16's range");

}  // namespace ssd
