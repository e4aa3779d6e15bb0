// Row norms around the projections, with the rows in 8 bits:
//
//   r = x + residual  (ssd_add_norm)   or   r = y * z / (1 + exp(-z))  (ssd_gated_norm)
//   n = r / sqrt(mean(r^2) + eps) * weight,  the mean over each of G runs of channels
//   scale = max|n| / 127 (1 where that is 0),  q = round half away(n / scale)
//
// Memory bound: every input is read once and every output written once, a row
// stays in fp32 registers in between. A workgroup computes one row (four of up to
// 512 channels, a wave each); thread i holds the row's pieces i, i + blockDim, ...
// of 8 consecutive channels. Rows that are not aligned, or not a multiple of 8
// long, take the same pieces with unaligned accesses, the last one channel by
// channel (G runs of channels that are no multiple of 8 long: a kernel of single
// channels). Two reductions over the row (the sum of squares, the largest
// magnitude) cross the waves in LDS; short runs of channels are summed side by
// side (4000 rows of 4096 in 64 runs: 35 -> 22 us). Rows leave past the caches: 2 to
// 10 % faster alone (loads that do are slower). With the 8-bit product that reads the
// codes next it is even at 8 rows (9.2 us, gated norm and Out Proj 9.0) and 16384
// (534 against 538 with ordinary stores, gated 275 against 280), but costs 2 to 7 %
// where they would still lie in the caches (2048 rows: 80.7 against 78.7, gated 54.0
// against 50.4).
// Measured: 16384 rows of 2560 bf16 with an fp32 residual, codes and values 98 to
// 101 us, 5.5 TB/s of 545 MB (codes only 86); 16384 of 5120 fp16, gated, 104 to 107
// us, 5.5 TB/s (139 us while the loads waited for one another; codes only 83 to 88);
// 8 rows of 2560 3.5 us, a launch and two memory round trips.
//
// The largest magnitude is found on bit patterns (unsigned order), in which
// NaN is above infinity and infinity above every number: a row that holds
// either gets a scale that is not finite, instead of codes that look sound.
#include "ssd_conv.hpp"
#include "ssd_launch.hpp"

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

// The mean of squares of each group goes to done(g, mean) in one lane. A group has n
// channels, and its squares are at(g gp) .. at(g gp + gp - 1).
//
// A wave takes a group at a time ...
template <class At, class Done>
__device__ __forceinline__ void group_means(int groups, int gp, int n, int wave, int nw, At at, Done done) {
  for (int g = wave; g < groups; g += nw) {
    float t = 0.f;
    for (int k = lane_id(); k < gp; k += kWave) t += at(g * gp + k);
    t = wave_sum(t);
    if (lane_id() == 0) done(g, t / (float)n);
  }
}
// ... or several side by side, with 2^sh lanes each.
template <class At, class Done>
__device__ __forceinline__ void short_group_means(int groups, int gp, int n, int sh, int wave, int nw, At at, Done done) {
  const int lanes = 1 << sh, sub = lane_id() & (lanes - 1);
  for (int g0 = wave * (kWave >> sh); g0 < groups; g0 += nw * (kWave >> sh)) {
    const int g = g0 + (lane_id() >> sh);
    float t = 0.f;
    if (g < groups)
      for (int k = sub; k < gp; k += lanes) t += at(g * gp + k);
    for (int m = lanes / 2; m >= 1; m >>= 1) t += __shfl_xor(t, m);
    if (g < groups && sub == 0) done(g, t / (float)n);
  }
}
// The largest power of two up to v, as its exponent.
__device__ __forceinline__ int log2_down(int v) { return 31 - __builtin_clz(v); }

// One row for each workgroup (of the first 2^20, then on), or (WAVE: rows of one
// piece a lane) for each wave. The mean is over the row (PARTS 0), or over groups
// of at least 64 pieces (1) or fewer (2).
template <int DT, int RT, bool GATED, int PARTS, int V, bool AL, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 512) void k_norm(NormArgs a) {
  extern __shared__ float s_parts[];  // PARTS: the sum of squares of each piece, then 1/rms of each group
  __shared__ float s_sum[kMaxWaves];
  __shared__ uint32_t s_max[kMaxWaves];
  const int nt = WAVE ? kWave : blockDim.x, nw = nt / kWave;
  const int tid = WAVE ? lane_id() : threadIdx.x, wave = WAVE ? 0 : wave_id();
  const int rows_wg = WAVE ? blockDim.x / kWave : 1;
  const int np = (a.cols + VEC - 1) / VEC;  // pieces of the row
  float* const s_part = s_parts + (PARTS && WAVE ? wave_id() * (np + a.groups) : 0);
  auto sync = [] {
    if constexpr (WAVE) wave_sync();
    else __syncthreads();
  };
  for (int64_t row = (int64_t)blockIdx.x * rows_wg + (WAVE ? wave_id() : 0); row < a.rows;
       row += (int64_t)gridDim.x * rows_wg) {
    const int64_t base = row * (int64_t)a.cols;
    const bool add = !GATED && a.residual;

    // everything is requested before anything is used; threads behind the last
    // piece load it too (no load is conditional on the lane)
    RawPiece<DT> xr[V], zr[V];
    RawPiece<RT> rr[V];
    RawPiece<DT_F32> wr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = min(tid + i * nt, np - 1), c = p * VEC, n = a.cols - c;
      xr[i].template load<AL>(a.x, row * (GATED ? (int64_t)a.cols : a.ld_x) + c, n);
      if constexpr (GATED) zr[i].template load<AL>(a.z, row * a.ld_z + c, n);
      else rr[i].template load<AL>(add ? a.residual : (const void*)a.weight, add ? base + c : 0, add ? n : a.cols);
      wr[i].template load<AL>(a.weight, c, n);
    }
    float r[V][VEC], ss[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = tid + i * nt;
      ss[i] = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        r[i][e] = xr[i].get(e);
        if constexpr (GATED) r[i][e] *= silu_rows<DT>(zr[i].get(e));
        else if (add) r[i][e] += rr[i].get(e);
        ss[i] = fmaf(r[i][e], r[i][e], ss[i]);
      }
      if (p >= np) ss[i] = 0.f;
      if constexpr (!GATED)
        if (a.residual_out && p < np) st_piece<RT, AL>(a.residual_out, base + p * VEC, a.cols - p * VEC, r[i]);
    }

    // 1 / rms, of the row or of each group. Where the sum of squares left fp32's range
    // (a value above 2^56 or so), or their mean and eps are so small that squares lost
    // bits, the row is scaled by a power of two and summed again. Ordinary rows pay a
    // comparison (16384 rows of 2560: 100.5 us with, 100.9 without).
    float rs0 = 0.f;
    const int gp = PARTS ? np / a.groups : np;  // pieces of a group
    auto again = [&](int i, float by) {  // piece i, scaled
      ss[i] = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        r[i][e] *= by;
        ss[i] = fmaf(r[i][e], r[i][e], ss[i]);
      }
      if (tid + i * nt >= np) ss[i] = 0.f;
    };
    if constexpr (PARTS == 0) {
      auto mean = [&] {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) t += ss[i];
        t = wave_sum(t);
        if constexpr (!WAVE) {
          if (lane_id() == 0) s_sum[wave] = t;
          __syncthreads();
          t = 0.f;
          for (int i = 0; i < nw; ++i) t += s_sum[i];
        }
        return t / (float)a.cols;
      };
      float m = mean() + a.eps;
      if (!in_range(m)) {  // the same in all threads of the row
        sync();
        const float by = scale_for(m);
#pragma unroll
        for (int i = 0; i < V; ++i) again(i, by);
        m = mean() + a.eps * by * by;
      }
      rs0 = inv_root(m);
    } else {
      float* const s_rs = s_part + np;
      float* const s_out = s_sum + (WAVE ? wave_id() : 0);  // whether a group's mean is out of range
      if (tid == 0) *s_out = 0.f;
      auto groups = [&](auto done) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int p = tid + i * nt;
          if (p < np) s_part[p] = ss[i];
        }
        sync();
        auto at = [&](int k) { return s_part[k]; };
        if constexpr (PARTS == 1) group_means(a.groups, gp, gp * VEC, wave, nw, at, done);
        else short_group_means(a.groups, gp, gp * VEC, log2_down(gp), wave, nw, at, done);
        sync();
      };
      groups([&](int g, float mean) {
        const float m = mean + a.eps;
        const bool in = in_range(m);
        s_rs[g] = in ? inv_root(m) : -scale_for(m);
        if (!in) *s_out = 1.f;
      });
      if (*s_out != 0.f) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float by = s_rs[min(tid + i * nt, np - 1) / gp];
          again(i, by < 0.f ? -by : 1.f);
        }
        groups([&](int g, float mean) {
          const float by = s_rs[g];
          if (by < 0.f) s_rs[g] = inv_root(mean + a.eps * by * by);
        });
      }
    }

    // The normalised rows. What threads behind the last piece hold counts for
    // nothing: where residual_out is residual itself, another wave may have
    // written the last piece before they loaded it.
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = tid + i * nt;
      const float rs = PARTS ? s_part[np + min(p, np - 1) / gp] : rs0;
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        r[i][e] = r[i][e] * rs * wr[i].get(e);
        m = max(m, __float_as_uint(r[i][e]) & 0x7fffffffu);
      }
      if (p < np) most = max(most, m);
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
    // the next row's sums overwrite this one's: with codes, the barrier of the
    // maximum has separated them already
    if (WAVE ? PARTS != 0 : !a.q) sync();
  }
}

// Gated rows in groups whose size is no multiple of 8, channel by channel. The row
// lies in LDS (up to 64 KB, and the groups' 1 / rms as much again) instead of
// registers, of which 16 channels in each of 1024 threads spilled 55. Up to 1024
// channels a wave where rows are many, 512 where they are few; loops unrolled twice
// (once: 458 -> 555 us in the first of these, four times: 64 -> 65 in the second).
// us, and with rows in registers: 4000 x 16380 in groups of 4 bf16 458, 620; 16384 x
// 1400 of 14 fp16 64, 87; 5000 x 4097 of 241 fp16 62, 217; 8 x 5100 of 204 7.8, 15;
// 16384 x 2001 of 87 bf16 92, 103; 16384 x 60 of 12 11.4, 10.1.
template <int DT>
__global__ __launch_bounds__(512) void k_norm_channels(NormArgs a) {
  typedef typename Store<DT>::T T;
  extern __shared__ float s_r[];
  __shared__ uint32_t s_max[kMaxWaves];
  __shared__ int s_out;  // whether a group's mean is out of range
  float* const s_rs = s_r + a.cols;
  const int nt = blockDim.x, nw = nt / kWave, tid = threadIdx.x, gp = a.cols / a.groups;
  // 16 lanes a group at most where that keeps all waves busy: fewer steps of a sum
  const int sh = min(log2_down(gp), a.groups > 2 * nw ? 4 : 6);
  const float per = 1.f / (float)gp;
  // channel c's group: (c + 1/2) / gp lies at least 1 / 2 gp from a whole number, and
  // two roundings of up to 16384 / gp are far less
  auto group = [&](int c) { return (int)(((float)c + 0.5f) * per); };
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t base = row * (int64_t)a.cols;
    const T* const y = (const T*)a.x + base;
    const T* const z = (const T*)a.z + row * a.ld_z;
    if (tid == 0) s_out = 0;
#pragma unroll 2
    for (int c = tid; c < a.cols; c += nt) s_r[c] = Store<DT>::to_f(y[c]) * silu_rows<DT>(Store<DT>::to_f(z[c]));
    auto groups = [&](auto done) {
      __syncthreads();
      short_group_means(a.groups, gp, gp, sh, wave_id(), nw, [&](int k) { return s_r[k] * s_r[k]; }, done);
      __syncthreads();
    };
    groups([&](int g, float mean) {
      const float m = mean + a.eps;
      const bool in = in_range(m);
      s_rs[g] = in ? inv_root(m) : -scale_for(m);
      if (!in) s_out = 1;
    });
    if (s_out) {
      for (int c = tid; c < a.cols; c += nt) {
        const float by = s_rs[group(c)];
        if (by < 0.f) s_r[c] *= -by;
      }
      groups([&](int g, float mean) {
        const float by = s_rs[g];
        if (by < 0.f) s_rs[g] = inv_root(mean + a.eps * by * by);
      });
    }
    uint32_t most = 0;
#pragma unroll 2
    for (int c = tid; c < a.cols; c += nt) {
      const float v = s_r[c] * s_rs[group(c)] * a.weight[c];
      most = max(most, __float_as_uint(v) & 0x7fffffffu);
      if (a.q) s_r[c] = v;
      else ((T*)a.out)[base + c] = to_store<DT>(v);
    }
    if (a.q) {
      most = wave_max(most);
      if (lane_id() == 0) s_max[wave_id()] = most;
      __syncthreads();
      most = 0;
      for (int i = 0; i < nw; ++i) most = max(most, s_max[i]);
      const Step st(most);
#pragma unroll 2
      for (int c = tid; c < a.cols; c += nt) {
        const float v = code(st.quotient(st.tiny ? st.up(s_r[c]) : s_r[c]));
        a.q[base + c] = (int8_t)(int)v;
        if (a.out) ((T*)a.out)[base + c] = to_store<DT>(v * st.scale);
      }
      if (tid == 0) a.scale[row] = st.scale;
    }
    __syncthreads();  // the next row overwrites what this one's threads read
  }
}

template <int DT, int RT, bool GATED, int PARTS, int V, bool AL, bool WAVE = false>
hipError_t go(const NormArgs& a, int waves, hipStream_t st) {
  const size_t lds = PARTS ? (WAVE ? waves : 1) * (size_t)(a.cols / VEC + a.groups) * sizeof(float) : 0;
  const int64_t wgs = WAVE ? (a.rows + waves - 1) / waves : a.rows;
  hipLaunchKernelGGL((k_norm<DT, RT, GATED, PARTS, V, AL, WAVE>), dim3((unsigned)min(wgs, (int64_t)1 << 20)),
                     dim3(waves * kWave), lds, st, a);
  return hipGetLastError();
}

template <int DT, int RT, bool GATED, int PARTS, bool AL>
hipError_t pick_pieces(const NormArgs& a, hipStream_t st) {
  // at most 8 waves a row: more meet at its two barriers more slowly (16384 rows
  // of 5120, gated: 10 waves 174 us, 5 waves 139; 8192 of 8192: 16 waves 120, 8
  // waves 100), fewer hold more registers (2560 columns: 5 waves 101 us, 3 waves
  // 106, 1 wave 116)
  const int wp = ((a.cols + 7) / 8 + kWave - 1) / kWave;  // pieces of a row, in waves
  const int v = (wp + 7) / 8, waves = (wp + v - 1) / v;
  // rows of one wave: four to a workgroup, without barriers (16384 rows of 320 9.2
  // us, one to a workgroup 10.0; 64 rows 3.0 and 3.2)
  if constexpr (PARTS != 1)  // (two groups of them have at most 32 pieces each)
    if (waves == 1) return go<DT, RT, GATED, PARTS, 1, AL, true>(a, 4, st);
  switch (v) {
    case 1: return go<DT, RT, GATED, PARTS, 1, AL>(a, waves, st);
    case 2: return go<DT, RT, GATED, PARTS, 2, AL>(a, waves, st);
    case 3: return go<DT, RT, GATED, PARTS, 3, AL>(a, waves, st);
    default: return go<DT, RT, GATED, PARTS, 4, AL>(a, waves, st);
  }
}

template <int DT>
hipError_t pick_channels(const NormArgs& a, hipStream_t st) {
  const int per = a.rows > 1024 ? 1024 : 512, waves = min((a.cols + per - 1) / per, 8);
  const size_t lds = (size_t)(a.cols + a.groups) * sizeof(float);
  hipLaunchKernelGGL((k_norm_channels<DT>), dim3((unsigned)min(a.rows, (int64_t)1 << 20)), dim3(waves * kWave), lds, st, a);
  return hipGetLastError();
}

template <int DT, int RT, bool GATED>
hipError_t pick(const NormArgs& a, hipStream_t st) {
  constexpr int64_t esize = DT == DT_F32 ? 4 : 2;
  if (a.groups == 1 || a.cols / a.groups % 8 == 0) {
    const void* const p = GATED ? a.z : a.x;
    const int64_t ld = GATED ? a.ld_z : a.ld_x;
    const bool al = a.cols % 8 == 0 && (uintptr_t)p % 16 == 0 && ld * esize % 16 == 0;
    if constexpr (GATED) {
      if (a.groups > 1 && a.cols / 8 / a.groups >= kWave)
        return al ? pick_pieces<DT, RT, true, 1, true>(a, st) : pick_pieces<DT, RT, true, 1, false>(a, st);
      if (a.groups > 1)
        return al ? pick_pieces<DT, RT, true, 2, true>(a, st) : pick_pieces<DT, RT, true, 2, false>(a, st);
    }
    return al ? pick_pieces<DT, RT, GATED, 0, true>(a, st) : pick_pieces<DT, RT, GATED, 0, false>(a, st);
  }
  if constexpr (GATED)
    return pick_channels<DT>(a, st);
  return hipErrorInvalidValue;
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
