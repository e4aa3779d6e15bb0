// From one block of a layer to the next: the norm after the block, its gate, the
// residual, and the norm before the next block, with the rows in 8 bits.
//   u = x / sqrt(mean(x^2) + eps) * post
//   r = act(gate) u + res_scale residual
//   y = r / sqrt(mean(r^2) + eps) * weight,  codes as the other norms'
//
// Memory bound: every input is read once and every output written once; between the two
// norms a row stays in fp32 registers. A workgroup computes one row (four of up to 512
// channels, a wave each), as k_norm does, with three reductions over the row instead of
// two. 16384 rows of 2560 bf16 with a gate for each token and an fp32 residual: 114 us for
// 587 MB, 5.2 TB/s, a large copy's rate. 8 rows 5.1 us: a launch, a round trip to memory
// and the reductions.
#include "ssd_act.hpp"
#include "ssd_launch.hpp"
#include "ssd_norm.hpp"

namespace ssd {
namespace {

// 1 / (1 + exp(-z)) to 9 roundings for any z, of a type DT: r may be kept in fp32.
// exp(-z) = 2^(-z c) exp(-z d) with c the first bits of log2(e), as many as leave z c
// exact (z has 8 or 11 bits), and the rest as exp's first terms. Infinities have their
// limits, as the second factor stays near 1, and NaN stays NaN. 16384 rows of 2560, a
// bf16 gate for each token and an fp32 residual: 122 us a call, 128 with fp32's sigmoid()
// and 120 with z log2(e) rounded to fp32, which costs |z| roundings.
template <int DT>
__device__ __forceinline__ float sigmoid_of(float z) {
  if constexpr (DT == DT_F32) {
    return sigmoid(z);
  } else {
    constexpr double kLog2e = 1.4426950408889634, kLn2 = 0.6931471805599453;
    constexpr double c = DT == DT_BF16 ? 47274.0 / 32768 : 5909.0 / 4096, d = (kLog2e - c) * kLn2;
    const float slope = DT == DT_BF16 ? -(float)d : fmaf(z, (float)(d * d / 2), -(float)d);
    const float rest = __builtin_amdgcn_fmed3f(fmaf(slope, z, 1.f), 0.875f, 1.125f);
    return __builtin_amdgcn_rcpf(fmaf(__builtin_amdgcn_exp2f(z * -(float)c), rest, 1.f));
  }
}
// Gates in the place of what they are the functions of.
template <int DT>
__device__ __forceinline__ void gates_of(int act, float (&z)[VEC]) {
  if (act == kActSigmoid) {  // the same for all lanes
#pragma unroll
    for (int e = 0; e < VEC; ++e) z[e] = sigmoid_of<DT>(z[e]);
  } else if (act == kActSilu) {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      z[e] = DT == DT_F32 ? silu(at_least(z[e], -104.f)) : fmaxf(z[e], -104.f) * sigmoid_of<DT>(z[e]);
  }
}

template <int DT, int RT, int V, bool AL, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 512) void k_block_norm(BlockNormArgs a) {
  __shared__ float s_sum[2][kMaxWaves];
  __shared__ uint32_t s_max[kMaxWaves];
  const int nt = WAVE ? kWave : blockDim.x, nw = nt / kWave;
  const int tid = WAVE ? lane_id() : threadIdx.x, wave = WAVE ? 0 : wave_id();
  const int rows_wg = WAVE ? blockDim.x / kWave : 1;
  const int np = (a.cols + VEC - 1) / VEC;  // pieces of the row
  const bool normed = a.out || a.q;
  for (int64_t row = (int64_t)blockIdx.x * rows_wg + (WAVE ? wave_id() : 0); row < a.rows;
       row += (int64_t)gridDim.x * rows_wg) {
    const int64_t base = row * (int64_t)a.cols;
    // everything is requested before anything is used; threads behind the last piece
    // load it too, and what is not there is read from the weights instead
    RawPiece<DT> xr[V], zr[V];
    RawPiece<RT> rr[V];
    RawPiece<DT_F32> pr[V], wr[V];
    const int64_t gate_row = (int64_t)((uint32_t)row / (uint32_t)a.per) * a.ld_gate;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = min(tid + i * nt, np - 1), c = p * VEC, n = a.cols - c;
      xr[i].template load<AL>(a.x, row * a.ld_x + c, n);
      zr[i].template load<AL>(a.gate ? a.gate : (const void*)a.post, a.gate ? gate_row + c : 0, a.gate ? n : a.cols);
      rr[i].template load<AL>(a.residual ? a.residual : (const void*)a.post, a.residual ? base + c : 0,
                              a.residual ? n : a.cols);
      pr[i].template load<AL>(a.post, c, n);
      wr[i].template load<AL>(normed ? a.weight : a.post, c, n);
    }
    float r[V][VEC];
    // 1 / rms of the row in r; where the sum of squares left fp32's range, or they and
    // eps are so small that squares lost bits, r is scaled by a power of two first
    auto inv_rms = [&](float* sums) {
      auto mean = [&] {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < VEC; ++e) ss = fmaf(r[i][e], r[i][e], ss);
          t += tid + i * nt < np ? ss : 0.f;
        }
        t = wave_sum(t);
        if constexpr (!WAVE) {
          if (lane_id() == 0) sums[wave] = t;
          __syncthreads();
          t = 0.f;
          for (int i = 0; i < nw; ++i) t += sums[i];
        }
        return t / (float)a.cols;
      };
      float m = mean() + a.eps;
      if (!in_range(m)) {  // the same in all threads of the row
        if constexpr (!WAVE) __syncthreads();
        const float by = scale_for(m);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) r[i][e] *= by;
        m = mean() + a.eps * by * by;
      }
      return inv_root(m);
    };
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) r[i][e] = xr[i].get(e);
    const float rx = inv_rms(s_sum[0]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = tid + i * nt;
#pragma unroll
      for (int e = 0; e < VEC; ++e) r[i][e] = r[i][e] * rx * pr[i].get(e);
      if (a.gate) {
        float z[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) z[e] = zr[i].get(e);
        gates_of<DT>(a.act, z);
#pragma unroll
        for (int e = 0; e < VEC; ++e) r[i][e] *= z[e];
      }
      if (a.residual) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) r[i][e] = fmaf(a.res_scale, rr[i].get(e), r[i][e]);
      }
      if (a.residual_out && p < np) st_piece<RT, AL>(a.residual_out, base + p * VEC, a.cols - p * VEC, r[i]);
    }
    if (normed) {
      const float rs = inv_rms(s_sum[1]);
      // what threads behind the last piece hold counts for nothing: where residual_out
      // is residual itself, another wave may have written the piece before they read it
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          r[i][e] = r[i][e] * rs * wr[i].get(e);
          m = max(m, __float_as_uint(r[i][e]) & 0x7fffffffu);
        }
        if (tid + i * nt < np) most = max(most, m);
      }
      if (a.q) {
        most = wave_max(most);
        if constexpr (!WAVE) {
          if (lane_id() == 0) s_max[wave] = most;
          __syncthreads();
          most = 0;
          for (int i = 0; i < nw; ++i) most = max(most, s_max[i]);
        }
        const Step st(most);
        if (st.tiny) {
#pragma unroll
          for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) r[i][e] = st.up(r[i][e]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int p = tid + i * nt;
#pragma unroll
          for (int e = 0; e < VEC; ++e) r[i][e] = st.quotient(r[i][e]);
          if (p < np) st_codes<AL>(a.q + base + p * VEC, a.cols - p * VEC, r[i]);
#pragma unroll
          for (int e = 0; e < VEC; ++e) r[i][e] *= st.scale;
        }
        if (tid == 0) a.scale[row] = st.scale;
      }
      if (a.out) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int p = tid + i * nt;
          if (p < np) st_piece<DT, AL>(a.out, base + p * VEC, a.cols - p * VEC, r[i]);
        }
      }
    }
    // the next row's sums overwrite this one's
    if constexpr (!WAVE) __syncthreads();
  }
}

template <int DT, int RT, int V, bool AL, bool WAVE = false>
hipError_t go(const BlockNormArgs& a, int waves, hipStream_t st) {
  const int64_t wgs = WAVE ? (a.rows + waves - 1) / waves : a.rows;
  hipLaunchKernelGGL((k_block_norm<DT, RT, V, AL, WAVE>), dim3((unsigned)min(wgs, (int64_t)1 << 20)),
                     dim3(waves * kWave), 0, st, a);
  return hipGetLastError();
}

// As the other norms: at most 8 waves a row; rows of one wave four to a workgroup.
template <int DT, int RT, bool AL>
hipError_t pick_pieces(const BlockNormArgs& a, hipStream_t st) {
  const int wp = ((a.cols + 7) / 8 + kWave - 1) / kWave;  // pieces of a row, in waves
  const int v = (wp + 7) / 8, waves = (wp + v - 1) / v;
  if (waves == 1) return go<DT, RT, 1, AL, true>(a, 4, st);
  switch (v) {
    case 1: return go<DT, RT, 1, AL>(a, waves, st);
    case 2: return go<DT, RT, 2, AL>(a, waves, st);
    case 3: return go<DT, RT, 3, AL>(a, waves, st);
    default: return go<DT, RT, 4, AL>(a, waves, st);
  }
}

template <int DT, int RT>
hipError_t pick(const BlockNormArgs& a, hipStream_t st) {
  constexpr int64_t esize = DT == DT_F32 ? 4 : 2;
  auto aligned = [&](const void* p, int64_t ld) { return (uintptr_t)p % 16 == 0 && ld * esize % 16 == 0; };
  const bool al = a.cols % 8 == 0 && aligned(a.x, a.ld_x) && (!a.gate || aligned(a.gate, a.ld_gate));
  return al ? pick_pieces<DT, RT, true>(a, st) : pick_pieces<DT, RT, false>(a, st);
}

}  // namespace

hipError_t launch_block_norm(int dtype, int res_dtype, const BlockNormArgs& a, hipStream_t st) {
  const bool keep32 = res_dtype == DT_F32;
  switch (dtype) {
    case DT_F32: return pick<DT_F32, DT_F32>(a, st);
    case DT_F16: return keep32 ? pick<DT_F16, DT_F32>(a, st) : pick<DT_F16, DT_F16>(a, st);
    case DT_BF16: return keep32 ? pick<DT_BF16, DT_F32>(a, st) : pick<DT_BF16, DT_BF16>(a, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ssd
