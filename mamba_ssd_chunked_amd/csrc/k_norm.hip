// Row norms around the projections, with the rows in 8 bits:
//
//   r = x + residual  (ssd_add_norm)   or   r = y * z / (1 + exp(-z))  (ssd_gated_norm)
//   n = r / sqrt(mean(r^2) + eps) * weight,  the mean over each of G runs of channels
//   scale = max|n| / 127,  q = round half away(n / scale)
//
// Memory bound: every input is read once and every output written once, a row
// stays in fp32 registers in between. A workgroup computes one row; thread i
// holds the row's pieces i, i + blockDim, ... (8 consecutive channels, or one
// channel where the rows are not a multiple of 8 long). Two reductions over
// the row (the sum of squares, the largest magnitude) cross the waves in LDS.
//
// The largest magnitude is found on bit patterns (unsigned order), in which
// NaN is above infinity and infinity above every number: a row that holds
// either gets a scale that is not finite, instead of codes that look sound.
#include "ssd_conv.hpp"
#include "ssd_launch.hpp"

namespace ssd {
namespace {

constexpr int kMaxWaves = 16;

template <int DT, int VEC, bool AL>
__device__ __forceinline__ void ld_piece(const void* p, int64_t i, float* v) {
  if constexpr (VEC == 1) {
    v[0] = ld_f<DT>(p, i);
  } else {
    constexpr int V = RawVec<DT>::V;
#pragma unroll
    for (int k = 0; k < VEC / V; ++k) {
      RawVec<DT> r;
      r.template load<AL>(p, i + k * V);
#pragma unroll
      for (int e = 0; e < V; ++e) v[k * V + e] = r.get(e);
    }
  }
}

template <int DT, int VEC>
__device__ __forceinline__ void st_piece(void* p, int64_t i, const float* v) {
  if constexpr (VEC == 1) {
    ((typename Store<DT>::T*)p)[i] = to_store<DT>(v[0]);
  } else {
    constexpr int V = RawVec<DT>::V;
#pragma unroll
    for (int k = 0; k < VEC / V; ++k) {
      RawVec<DT> r;
      r.set(v + k * V);
      r.store(p, i + k * V);
    }
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

// Codes of values n in steps of most / 127. inv = 127 / most overflows for rows
// below 2^-120; such rows are scaled up by 2^100 first (exactly).
struct Coder {
  float scale, inv, up;
  __device__ __forceinline__ explicit Coder(uint32_t most_bits) {
    const float most = __uint_as_float(most_bits);
    scale = most_bits == 0 ? 1.f : most / 127.f;
    up = most < 0x1p-100f ? 0x1p100f : 1.f;
    inv = most_bits == 0 ? 0.f : 127.f / (most * up);
  }
  __device__ __forceinline__ float code(float n) const { return truncf(q8_pre((n * up) * inv)); }
};

template <int DT, int RT, bool GATED, int VEC, int V, bool AL>
__global__ __launch_bounds__(1024) void k_norm(NormArgs a) {
  extern __shared__ float s_part[];  // groups > 1: the sum of squares of each piece, then 1/rms of each group
  __shared__ float s_sum[kMaxWaves];
  __shared__ uint32_t s_max[kMaxWaves];
  const int nt = blockDim.x, nw = nt / kWave;
  const int np = a.cols / VEC;  // pieces of the row
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t base = row * (int64_t)a.cols;

    float r[V][VEC];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = threadIdx.x + i * nt;
      if (p < np) ld_piece<DT, VEC, GATED || AL>(a.x, row * (GATED ? (int64_t)a.cols : a.ld_x) + p * VEC, r[i]);
    }
    if constexpr (GATED) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int p = threadIdx.x + i * nt;
        if (p < np) {
          float z[VEC];
          ld_piece<DT, VEC, AL>(a.z, row * a.ld_z + p * VEC, z);
#pragma unroll
          for (int e = 0; e < VEC; ++e) r[i][e] *= silu(z[e]);
        }
      }
    } else {
      if (a.residual) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int p = threadIdx.x + i * nt;
          if (p < np) {
            float o[VEC];
            ld_piece<RT, VEC, true>(a.residual, base + p * VEC, o);
#pragma unroll
            for (int e = 0; e < VEC; ++e) r[i][e] += o[e];
          }
        }
      }
      if (a.residual_out) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int p = threadIdx.x + i * nt;
          if (p < np) st_piece<RT, VEC>(a.residual_out, base + p * VEC, r[i]);
        }
      }
    }

    // sums of squares
    float ss[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ss[i] = 0.f;
      if ((int)threadIdx.x + i * nt < np) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss[i] = fmaf(r[i][e], r[i][e], ss[i]);
      }
    }
    const int gp = np / a.groups;  // pieces of a group
    float rs0 = 0.f;
    if (!GATED || a.groups == 1) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) t += ss[i];
      t = wave_sum(t);
      if (lane_id() == 0) s_sum[wave_id()] = t;
      __syncthreads();
      t = 0.f;
      for (int i = 0; i < nw; ++i) t += s_sum[i];
      rs0 = rsqrtf(t / (float)a.cols + a.eps);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int p = threadIdx.x + i * nt;
        if (p < np) s_part[p] = ss[i];
      }
      __syncthreads();
      float* const s_rs = s_part + np;
      for (int g = wave_id(); g < a.groups; g += nw) {
        float t = 0.f;
        for (int k = lane_id(); k < gp; k += kWave) t += s_part[g * gp + k];
        t = wave_sum(t);
        if (lane_id() == 0) s_rs[g] = rsqrtf(t / (float)(gp * VEC) + a.eps);
      }
      __syncthreads();
    }

    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = threadIdx.x + i * nt;
      if (p < np) {
        float w[VEC];
        ld_piece<DT_F32, VEC, true>(a.weight, p * VEC, w);
        const float rs = (!GATED || a.groups == 1) ? rs0 : s_part[np + p / gp];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          r[i][e] = r[i][e] * rs * w[e];
          most = max(most, __float_as_uint(r[i][e]) & 0x7fffffffu);
        }
      }
    }
    if (a.q) {
      most = wave_max(most);
      if (lane_id() == 0) s_max[wave_id()] = most;
      __syncthreads();
      most = 0;
      for (int i = 0; i < nw; ++i) most = max(most, s_max[i]);
      const Coder cd(most);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int p = threadIdx.x + i * nt;
        if (p < np) {
          float c[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            c[e] = cd.code(r[i][e]);
            r[i][e] = c[e] * cd.scale;
          }
          if constexpr (VEC == 1) {
            a.q[base + p] = (int8_t)(int)c[0];
          } else {
            const uint2 v = make_uint2(pack4((int)c[0], (int)c[1], (int)c[2], (int)c[3]),
                                       pack4((int)c[4], (int)c[5], (int)c[6], (int)c[7]));
            *(uint2*)(a.q + base + p * VEC) = v;
          }
        }
      }
      if (threadIdx.x == 0) a.scale[row] = cd.scale;
    }
    if (a.out) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int p = threadIdx.x + i * nt;
        if (p < np) st_piece<DT, VEC>(a.out, base + p * VEC, r[i]);
      }
    }
    // the next row's sums overwrite this one's: with codes, the barrier of the
    // maximum has separated them already
    if (!a.q) __syncthreads();
  }
}

template <int DT, int RT, bool GATED, int VEC, int V, bool AL>
hipError_t go(const NormArgs& a, int nt, hipStream_t st) {
  const size_t lds = GATED && a.groups > 1 ? (size_t)(a.cols / VEC + a.groups) * sizeof(float) : 0;
  hipLaunchKernelGGL((k_norm<DT, RT, GATED, VEC, V, AL>), dim3((unsigned)min(a.rows, (int64_t)1 << 20)),
                     dim3(nt), lds, st, a);
  return hipGetLastError();
}

template <int DT, int RT, bool GATED>
hipError_t pick(const NormArgs& a, hipStream_t st) {
  constexpr int esize = DT == DT_F32 ? 4 : 2;
  const int group = a.cols / a.groups;
  if (group % 8 == 0) {
    const int np = a.cols / 8;
    const int v = (np + 511) / 512;  // pieces of a thread, 1 .. 4
    const int nt = ((np + v - 1) / v + kWave - 1) / kWave * kWave;
    const bool al = GATED ? (uintptr_t)a.z % 16 == 0 && a.ld_z * esize % 16 == 0
                          : (uintptr_t)a.x % 16 == 0 && a.ld_x * esize % 16 == 0;
#define GO_(V_) return al ? go<DT, RT, GATED, 8, V_, true>(a, nt, st) : go<DT, RT, GATED, 8, V_, false>(a, nt, st)
    switch (v) {
      case 1: GO_(1);
      case 2: GO_(2);
      case 3: GO_(3);
      default: GO_(4);
    }
#undef GO_
  }
  // single channels, 1 .. 16 of a thread in powers of two
  int v = 1;
  while (a.cols > v * 1024) v *= 2;
  const int nt = ((a.cols + v - 1) / v + kWave - 1) / kWave * kWave;
  switch (v) {
    case 1: return go<DT, RT, GATED, 1, 1, false>(a, nt, st);
    case 2: return go<DT, RT, GATED, 1, 2, false>(a, nt, st);
    case 4: return go<DT, RT, GATED, 1, 4, false>(a, nt, st);
    case 8: return go<DT, RT, GATED, 1, 8, false>(a, nt, st);
    default: return go<DT, RT, GATED, 1, 16, false>(a, nt, st);
  }
}

}  // namespace

hipError_t launch_norm(int dtype, int res_dtype, const NormArgs& a, hipStream_t st) {
  const bool keep32 = res_dtype == DT_F32;
  switch (dtype) {
    case DT_F32: return a.z ? pick<DT_F32, DT_F32, true>(a, st) : pick<DT_F32, DT_F32, false>(a, st);
    case DT_F16:
      return a.z ? pick<DT_F16, DT_F16, true>(a, st)
                 : keep32 ? pick<DT_F16, DT_F32, false>(a, st) : pick<DT_F16, DT_F16, false>(a, st);
    case DT_BF16:
      return a.z ? pick<DT_BF16, DT_BF16, true>(a, st)
                 : keep32 ? pick<DT_BF16, DT_F32, false>(a, st) : pick<DT_BF16, DT_BF16, false>(a, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ssd
