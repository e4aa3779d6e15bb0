// Shared by the row norms (k_norm.hip, k_block_norm.hip): rows in pieces of 8 channels,
// sums and maxima over a row, means of squares that leave fp32's range, 8-bit rows.
#pragma once

#include "ssd_conv.hpp"

namespace ssd {
namespace {

constexpr int kMaxWaves = 8;
constexpr int VEC = 8;  // channels of a piece

// A piece of a row as loaded: VEC channels, of which the last piece of a row that
// is no multiple of 8 long has fewer (n; the rest are zeros, and are not written).
template <int DT>
struct RawPiece {
  static constexpr int V = RawVec<DT>::V;
  RawVec<DT> v[VEC / V];
  template <bool AL>
  __device__ __forceinline__ void load(const void* p, int64_t i, int n) {
    if (AL || n >= VEC) {
#pragma unroll
      for (int k = 0; k < VEC / V; ++k) v[k].template load<AL>(p, i + k * V);
    } else {
      float f[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = e < n ? ld_f<DT>(p, i + e) : 0.f;
#pragma unroll
      for (int k = 0; k < VEC / V; ++k) v[k].set(f + k * V);
    }
  }
  __device__ __forceinline__ float get(int e) const { return v[e / V].get(e % V); }
};
// Four whole numbers of [-127, 127] as bytes: the conversions write their low
// bytes straight into place.
__device__ __forceinline__ uint32_t pack4_codes(const float* v) {
  uint32_t d = (uint32_t)(int)v[0];
  asm("v_cvt_i32_f32_sdwa %0, %1 dst_sel:BYTE_1 dst_unused:UNUSED_PRESERVE src0_sel:DWORD" : "+v"(d) : "v"(v[1]));
  asm("v_cvt_i32_f32_sdwa %0, %1 dst_sel:BYTE_2 dst_unused:UNUSED_PRESERVE src0_sel:DWORD" : "+v"(d) : "v"(v[2]));
  asm("v_cvt_i32_f32_sdwa %0, %1 dst_sel:BYTE_3 dst_unused:UNUSED_PRESERVE src0_sel:DWORD" : "+v"(d) : "v"(v[3]));
  return d;
}

template <int DT, bool AL>
__device__ __forceinline__ void st_piece(void* p, int64_t i, int n, const float* v) {
  constexpr int V = RawVec<DT>::V;
  if (AL || n >= VEC) {
#pragma unroll
    for (int k = 0; k < VEC / V; ++k) {
      RawVec<DT> r;
      r.set(v + k * V);
      r.template store_nt<AL>(p, i + k * V);
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < n) ((typename Store<DT>::T*)p)[i + e] = to_store<DT>(v[e]);
  }
}

// v + copysign(0.5 - 2^-25, v), truncated, is v rounded half away from zero.
__device__ __forceinline__ float code(float v) { return truncf(v + __builtin_copysignf(0.49999997f, v)); }

// The codes of VEC values v in steps; |v| is at most 127 (1 + 2^-22), so there is
// nothing to clamp. On return v holds the codes.
template <bool AL>
__device__ __forceinline__ void st_codes(int8_t* p, int n, float* v) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = code(v[e]);
  typedef uint32_t v2 __attribute__((ext_vector_type(2)));
  typedef uint32_t v2_any __attribute__((ext_vector_type(2), aligned(1)));
  const uint32_t lo = pack4_codes(v), hi = pack4_codes(v + 4);
  if constexpr (AL) {
    __builtin_nontemporal_store((v2){lo, hi}, (v2*)p);
  } else if (n >= VEC) {
    __builtin_nontemporal_store((v2_any){lo, hi}, (v2_any*)p);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < n) p[e] = (int8_t)(int)v[e];
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = kWave / 2; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int m = kWave / 2; m >= 1; m >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
  return v;
}

// Whether a mean of squares (and eps) was formed without a loss: neither infinite
// nor so small that squares fell below fp32's normal range. NaN is not.
__device__ __forceinline__ bool in_range(float m) { return m >= 0x1p-100f && m <= 0x1p127f; }
// The power of two that takes the values of such a row to where their squares are
// well inside fp32's range: the largest to 2^48, the smallest subnormal to 2^-53.
__device__ __forceinline__ float scale_for(float m) { return m > 1.f ? 0x1p-80f : 0x1p96f; }
// 1 / sqrt(m), 0 for m = 0 (a row of zeros without eps is zeros, not NaN).
__device__ __forceinline__ float inv_root(float m) { return m > 0.f ? rsqrtf(m) : 0.f; }

// The step of a row whose largest magnitude has these bits: most / 127, 1 where that
// rounds to zero. The codes are those of the quotient y / scale as fp32 rounds it: a
// product with 1 / scale, and its remainder (exact in one multiply-add) brought in,
// which costs no time (16384 rows of 5120 fp16, gated, codes only: 83 us; 87 with
// y * (127 / most), some of whose codes next to a border were the neighbours'; 8 rows
// of 2560 3.47 us and 3.39, as the two divisions follow one another). Rows of steps
// below 2^-64 are scaled up with them (up), exactly, so that the remainder is no
// subnormal; a subnormal step may be well below most / 127: codes end at 127.
struct Step {
  float scale, unit, inv;
  bool tiny;
  __device__ __forceinline__ explicit Step(uint32_t most) {
    scale = __uint_as_float(most) / 127.f;
    if (scale == 0.f) scale = 1.f;
    tiny = scale < 0x1p-64f;
    unit = tiny ? scale * 0x1p64f : scale;
    inv = 1.f / unit;
  }
  __device__ __forceinline__ float up(float y) const {
    return fminf(fmaxf(y * 0x1p64f, -127.f * unit), 127.f * unit);
  }
  __device__ __forceinline__ float quotient(float y) const {
    const float v = y * inv;
    return fmaf(fmaf(-v, unit, y), inv, v);
  }
};

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace
}  // namespace ssd
