// Shared by the gated delta rule's kernels (k_delta.hip, k_delta_step.hip).
#pragma once

#include "ssd_device.hpp"
#include "ssd_launch.hpp"

namespace ssd {

// The write strength of a position: beta, or the logistic function of it.
template <int DT>
__device__ __forceinline__ float delta_beta(const DeltaArgs& a, int64_t row, int h) {
  const float b = ld_f<DT>(a.beta, row * a.ld_beta + h);
  return a.logit ? 1.f / (1.f + expf(-b)) : b;
}

// Sums over aligned groups of R lanes, in every lane: exchanges inside the vector
// unit up to 16 lanes, then across.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int R>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr (R >= 2) v = dpp_add<0xB1>(v);   // lanes 1 0 3 2
  if constexpr (R >= 4) v = dpp_add<0x4E>(v);   // lanes 2 3 0 1
  if constexpr (R >= 8) v = dpp_add<0x141>(v);  // mirrored in 8
  if constexpr (R >= 16) v = dpp_add<0x140>(v); // mirrored in 16
  if constexpr (R >= 32) v += __int_as_float(swz<16>(__float_as_int(v)));
  if constexpr (R >= 64) v += __shfl_xor(v, 32);
  return v;
}

}  // namespace ssd
