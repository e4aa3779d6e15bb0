// Device helpers of the causal convolution (k_conv.hip, k_conv_decode.hip) and
// of the row norms (k_norm.hip).
#pragma once

#include "ssd_device.hpp"

namespace ssd {

// u / (1 + exp(-u)) in fp32, to 9 roundings for any u down to -87 (below, where it is
// less than 2^-119, it may be 0). With t = exp(-|u|) it is u / (1 + t) or u t / (1 + t):
// nothing overflows. -|u| log2(e) is held to twice fp32's bits, as h + l, because an
// exponent's absolute error is the power's relative one (rounded once, it would cost
// |u| roundings); exp2 and the reciprocal are the hardware's, one unit each.
__device__ __forceinline__ float silu(float u) {
  const float a = fminf(fabsf(u), 104.f);  // exp(-104) is 0
  const float h = a * -1.44269502f;
  const float l = fmaf(a, -1.92596299e-8f, fmaf(a, -1.44269502f, -h));
  const float t = __builtin_amdgcn_exp2f(h) * fmaf(l, 0.693147182f, 1.f);
  return (u < 0.f ? u * t : u) * __builtin_amdgcn_rcpf(1.f + t);
}

// The same to about |u| + 8 roundings (2^-17 at u = -87), eight operations fewer: for
// what is 16 bits wide next, or was before.
__device__ __forceinline__ float silu_16(float u) {
  return u * __builtin_amdgcn_rcpf(1.0f + __expf(-u));
}

// Rows in storage type DT. fp32 rows take the exact form, which the memory covers
// (8192 x 5376 channels fp32 73 us with either; gated norm of 8192 x 5120 fp32 96).
// 16-bit rows take the short one: a convolution's result is rounded to 16 bits at
// once (a half step is 2^-12 of it or more), and a gate was read from 16 bits; there
// the exact form would cost 5 to 19 % (16384 x 5120 gated, rows and codes 107 us
// and 113, codes only 86 and 103).
template <int DT>
__device__ __forceinline__ float silu_rows(float u) {
  return DT == DT_F32 ? silu(u) : silu_16(u);
}

// log(1 + exp(v)) as max(v, 0) + log1p(exp(-|v|)): step sizes of 1e-3 keep
// their relative precision (log(1 + x) of a small x would lose it).
__device__ __forceinline__ float softplus(float v) {
  return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v)));
}

// 16 bytes of consecutive elements as loaded, at a 16-byte aligned address (AL)
// or at any element's: the memory pipe takes both in one access.
template <int DT>
struct RawVec {
  static constexpr int V = DT == DT_F32 ? 4 : 8;
  typedef uint32_t v4 __attribute__((ext_vector_type(4)));
  typedef uint32_t v4_any __attribute__((ext_vector_type(4), aligned(2)));
  v4 w;
  __device__ __forceinline__ void zero() { w = (v4){0, 0, 0, 0}; }
  template <bool AL>
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const typename Store<DT>::T* const q = (const typename Store<DT>::T*)p + i;
    if constexpr (AL) w = *(const v4*)q;
    else w = *(const v4_any*)q;
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    *(v4*)((typename Store<DT>::T*)p + i) = w;
  }
  // past the caches' reach: written once and read, if at all, by a later kernel
  template <bool AL>
  __device__ __forceinline__ void store_nt(void* p, int64_t i) const {
    typename Store<DT>::T* const q = (typename Store<DT>::T*)p + i;
    if constexpr (AL) __builtin_nontemporal_store(w, (v4*)q);
    else __builtin_nontemporal_store(w, (v4_any*)q);
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (DT == DT_F32) return __uint_as_float(w[e]);
    else if constexpr (DT == DT_BF16) return __uint_as_float((e & 1) ? (w[e >> 1] & 0xffff0000u) : (w[e >> 1] << 16));
    else return (float)__builtin_bit_cast(_Float16, (u16)((e & 1) ? (w[e >> 1] >> 16) : (w[e >> 1] & 0xffffu)));
  }
  __device__ __forceinline__ void set(const float* v) {
    if constexpr (DT == DT_F32) {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = pack2<DT>(v[2 * e], v[2 * e + 1]);
    }
  }
};

}  // namespace ssd
