// Activations of a product's epilogue and of gates, in fp32.
#pragma once

#include "ssd_conv.hpp"

namespace ssd {

// The values equal the C ABI's SSD_ACT_* codes.
enum { kActNone = 0, kActRelu = 1, kActRelu2 = 2, kActSilu = 3, kActSigmoid = 4, kActGelu = 5, kActGeluTanh = 6 };

// Infinities have their limits, and NaN stays NaN: what is held inside a range is
// compared and selected, as a minimum would drop NaN.
__device__ __forceinline__ float at_most(float v, float most) { return v > most ? most : v; }
__device__ __forceinline__ float at_least(float v, float least) { return v < least ? least : v; }

// 1 / (1 + exp(-u)), as silu() forms it: nothing overflows, 9 roundings for any u.
__device__ __forceinline__ float sigmoid(float u) {
  const float a = at_most(fabsf(u), 104.f);
  const float h = a * -1.44269502f;
  const float l = fmaf(a, -1.92596299e-8f, fmaf(a, -1.44269502f, -h));
  const float t = __builtin_amdgcn_exp2f(h) * fmaf(l, 0.693147182f, 1.f);
  return (u < 0.f ? t : 1.f) * __builtin_amdgcn_rcpf(1.f + t);
}

// u Phi(u) with the normal distribution's Phi, as u (1 - q) or u q with
// q = erfc(|u| / sqrt 2) / 2. With z = |u| / sqrt 2 and t = 1 / (1 + z / 2),
// erfc(z) = t exp(-z^2 + p(t)) (the form of Press et al., Numerical Recipes): p is a
// polynomial of degree 9, fitted here to log(exp(z^2) erfc(z) / t) on 0 <= z <= 11 for the
// least largest error (5.5e-8). To u^2 / 2 + 12 roundings.
__device__ __forceinline__ float gelu(float u) {
  constexpr float p[10] = {
      -1.26546233f, 0.998917351f, 0.384254506f, 0.0457367484f, -0.0307324845f, -0.0213053197f,
      -0.766202087f, 1.20839332f, -0.70244627f, 0.148846621f};
  const float a = at_most(fabsf(u), 15.f);
  const float t = __builtin_amdgcn_rcpf(fmaf(a, 0.353553391f, 1.f));
  float e = p[9];
#pragma unroll
  for (int i = 8; i >= 0; --i) e = fmaf(e, t, p[i]);
  const float q = 0.5f * t * __expf(fmaf(-0.5f * a, a, e));
  return u > 0.f ? fmaf(-a, q, u) : -a * q;
}

// The same with the approximation Phi(u) = (1 + tanh(sqrt(2 / pi) (u + 0.044715 u^3))) / 2,
// which is a logistic function of twice that.
__device__ __forceinline__ float gelu_tanh(float u) {
  const float v = at_least(u, -30.f);  // the function is 0 from there on down
  return v * sigmoid(1.59576912f * fmaf(0.044715f * v * v, v, v));
}

template <int N>
__device__ __forceinline__ void activate(int act, float (&y)[N]) {
  switch (act) {  // the same for all lanes
    case kActRelu:
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] = y[e] < 0.f ? 0.f : y[e];
      break;
    case kActRelu2:
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] = y[e] < 0.f ? 0.f : y[e] * y[e];
      break;
    case kActSilu:
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] = silu(at_least(y[e], -104.f));
      break;
    case kActSigmoid:
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] = sigmoid(y[e]);
      break;
    case kActGelu:
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] = gelu(y[e]);
      break;
    case kActGeluTanh:
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] = gelu_tanh(y[e]);
      break;
    default: break;
  }
}

}  // namespace ssd
