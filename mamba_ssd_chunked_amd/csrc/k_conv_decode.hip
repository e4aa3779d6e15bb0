// Single-token step of the causal convolution and the SSD in one launch:
//
//   u[c] = sum_j w[c,j] (the last W inputs of channel c) + b[c],  x | B | C = silu(u)
//   dt = softplus(dt_raw + dt_bias),   then the step of k_decode.hip on x, B, C, dt
//
// with everything between the two kept in fp32 (SiLU and exp(dt A) in their exact
// forms in any storage type: 0.1 us of a step of one sequence). The state is read
// and written once and is by far the most of the traffic (at P = 64, N = 128 in
// fp32 64 KB a head against about 6 KB of the convolution's inputs, which the heads
// of a group share in the caches), so a large batch is bound by HBM and a small one
// by the latency of one pass.
//
// A workgroup of four waves takes HB heads of a group: one where heads are few
// or large, up to 8 otherwise (32 KB of state), so that the
// convolution of B and C is done for all of them and no workgroup is over
// before it has begun. Its 16-byte slices of the state are requested first; then
// each thread computes the convolution of one or two of the HB P + 2 N channels
// that the heads need, into LDS. All W slots of the ring are loaded, and matched
// with their weights once pos has arrived, so the prologue costs one memory
// round trip, not two. The slot pos % W is written by the head itself for its x
// channels and by the first heads of a group for B and C; nobody reads that
// slot's value, so workgroups need no order.
//
// Measured, fp16 with 80 heads of 64 x 128: fp32 state 5.2 us at batch 1, 231 us
// at batch 256 (5.9 TB/s of 1.36 GB); 8-bit state 4.5 and 76 us (4.7 TB/s).
#include "ssd_conv.hpp"
#include "ssd_launch.hpp"

namespace ssd {
namespace {

constexpr int kStepThreads = 256;

struct StepArgs {
  ConvPtrs cv;
  const float* A;
  const float* D;
  ScalePtrs sc;
  void* state;
  void* Y;
  int H, G, hpg, Cd;
  int blocks;  // workgroups of a group of a sequence
};

// A state row's numbers after the convolution.
struct RowF {
  float decay, dx, Dx, unused;  // exp(dt A), dt x, D x
};
struct RowI8 {
  float qx, M, f, g;  // float(Q(Xs)), M_req, exp(dt A) s_C s_S, s_C s_B dt x
  float Dx;
  int qd;             // Q(Decay)
  float unused[2];
};
template <bool I8>
struct RowOf { typedef RowF T; };
template <>
struct RowOf<true> { typedef RowI8 T; };

template <bool I8, int ROWS, int NS>
struct StepLds {
  typename RowOf<I8>::T row[ROWS];
  float b[NS], c[NS];  // B, C (INT8: float(Q(B)))
  int8_t qc[NS];       // INT8: Q(C)
};

// One channel's convolution: the new input, the ring's W slots and the weights,
// loaded as they lie (no load is conditional and none is converted here, so that
// none is waited for before all of them are under way).
template <int DT>
struct ConvLane {
  typedef typename Store<DT>::T T;
  T raw, slot[4];
  float w[4], bias;
  __device__ __forceinline__ void load(const StepArgs& a, int64_t b, int c, int W) {
    raw = ((const T*)a.cv.xbc)[b * a.cv.ld_xbc + c];
    const int64_t r = b * W * (int64_t)a.Cd + c;
#pragma unroll
    for (int s = 0; s < 4; ++s) {  // W of them; the rest repeat the last
      slot[s] = ((const T*)a.cv.state)[r + (int64_t)min(s, W - 1) * a.Cd];
      w[s] = a.cv.weight[(int64_t)c * W + min(s, W - 1)];
    }
    bias = a.cv.bias ? a.cv.bias[c] : 0.f;
  }
  // cur = pos % W; slots of positions before the sequence's start count as zero.
  // (Selections are made of values: of array elements they would be of addresses,
  // and the arrays would live in scratch memory: 231 us a step instead of 271 at
  // 80 heads of 64 x 128 and batch 256.)
  __device__ __forceinline__ float value(int W, uint32_t pos, int cur) const {
    const float s0 = Store<DT>::to_f(slot[0]), s1 = Store<DT>::to_f(slot[1]);
    const float s2 = Store<DT>::to_f(slot[2]), s3 = Store<DT>::to_f(slot[3]);
    const float w0 = w[0], w1 = w[1], w2 = w[2], w3 = w[3];
    auto at = [&](int back) {
      const int s = cur >= back ? cur - back : cur - back + W;
      const float v = s == 0 ? s0 : s == 1 ? s1 : s == 2 ? s2 : s3;
      return pos >= (uint32_t)back ? v : 0.f;
    };
    float u = bias;
    if (W >= 4) u = fmaf(w0, at(3), u);
    if (W >= 3) u = fmaf(W == 4 ? w1 : w0, at(2), u);
    u = fmaf(W == 4 ? w2 : W == 3 ? w1 : w0, at(1), u);
    return silu(fmaf(W == 4 ? w3 : W == 3 ? w2 : w1, Store<DT>::to_f(raw), u));
  }
};

// Q(Decay) = min(128, RHAZ(128 exp(dt A))), decided in float64: float32 settles
// it unless it lies within 1e-3 of a border between two codes (its error is
// below 1e-4 for every decay up to 1).
__device__ __forceinline__ int quant_decay(float dt, float A) {
  const float v = 128.f * __expf(dt * A), n = floorf(v + 0.5f);
  if (fabsf(fabsf(v - n) - 0.5f) > 1e-3f && v < 128.25f) return (int)fminf(n, 128.f);
  return (int)fmin(round(exp((double)dt * (double)A) * 128.0), 128.0);
}

template <bool I8, int DT, int P, int NS, int HB>
__global__ __launch_bounds__(kStepThreads) void k_conv_decode(StepArgs a) {
  typedef typename Store<DT>::T T;
  constexpr int R = NS / (I8 ? 16 : 4);                             // 16-byte slices of a state row
  constexpr int ROWS = HB * P;                                      // state rows of the workgroup
  constexpr int SLOTS = ROWS * R;
  constexpr int ITER = (SLOTS + kStepThreads - 1) / kStepThreads;   // of a thread
  constexpr int NCH = ROWS + 2 * NS;
  constexpr int CIT = (NCH + kStepThreads - 1) / kStepThreads;
  __shared__ __attribute__((aligned(16))) StepLds<I8, ROWS, NS> L;

  const int tid = threadIdx.x;
  // (batch, group, block of heads)
  const unsigned bg = blockIdx.x / (unsigned)a.blocks, blk = blockIdx.x % (unsigned)a.blocks;
  const int64_t b = bg / (unsigned)a.G;
  const int g = (int)(bg % (unsigned)a.G);
  const int h0 = g * a.hpg + (int)blk * HB;
  const int rows = HB == 1 ? ROWS : min(HB, a.hpg - (int)blk * HB) * P;
  const int slots = HB == 1 ? SLOTS : rows * R;
  const int64_t row0 = (b * a.H + h0) * P;  // of the state and of Y
  const int x0 = h0 * P;                    // the first x channel
  v4u* const st = (v4u*)a.state + row0 * R;

  v4u hv[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    // behind the last slot: the last one's value, used by nobody (no branch)
    hv[i] = __builtin_nontemporal_load(&st[min(tid + i * kStepThreads, slots - 1)]);
  }

  // channels of B, C, then x; everything they need is requested here
  const int W = a.cv.width;
  const int dX = a.H * P, dBC = a.G * NS;
  const int nch = 2 * NS + rows;
  ConvLane<DT> cl[CIT];
  typename Store<DT>::T dtr[CIT];
  float dtb[CIT], Av[CIT], Dv[CIT], k0[CIT], k1[CIT], k2[CIT];
  int ch[CIT];
  float sC = 0.f, sB = 0.f;
  if constexpr (I8) {
    sC = a.sc.s_C[g];
    sB = a.sc.s_B[g];
  }
#pragma unroll
  for (int i = 0; i < CIT; ++i) {
    // threads behind the last channel, and those of B and C in the x part, load
    // what a neighbour does
    const int k = min(tid + i * kStepThreads, nch - 1), xr = max(k - 2 * NS, 0);
    ch[i] = k < NS ? dX + g * NS + k : k < 2 * NS ? dX + dBC + g * NS + (k - NS) : x0 + xr;
    cl[i].load(a, b, ch[i], W);
    const int h = HB == 1 ? h0 : h0 + xr / P;
    dtr[i] = ((const T*)a.cv.dt_raw)[b * a.cv.ld_dt + h];
    dtb[i] = a.cv.dt_bias ? a.cv.dt_bias[h] : 0.f;
    Av[i] = a.A[h];
    Dv[i] = a.D[h];
    if constexpr (I8) {
      k0[i] = *(k < NS ? a.sc.inv_B + g : k < 2 * NS ? a.sc.inv_C + g : a.sc.inv_X + x0 + xr);
      k1[i] = a.sc.M_req[x0 + xr];
      k2[i] = a.sc.s_S[x0 + xr];
    }
  }
  const uint32_t pos = (uint32_t)max(a.cv.pos[b], 0);
  const int cur = (int)(pos % (uint32_t)W);

#pragma unroll
  for (int i = 0; i < CIT; ++i) {
    const int k = tid + i * kStepThreads;
    if (k < nch) {
      const float v = cl[i].value(W, pos, cur);
      if (k < 2 * NS) {
        if constexpr (I8) {
          const int q = q8(__fmul_rn(v, k0[i]));
          if (k < NS) L.b[k] = (float)q;
          else L.qc[k - NS] = (int8_t)q;
        } else {
          if (k < NS) L.b[k] = v;
          else L.c[k - NS] = v;
        }
      } else {
        const float dt = softplus(Store<DT>::to_f(dtr[i]) + dtb[i]);
        const float decay = expf(dt * Av[i]);  // to a unit for any argument: the state keeps it
        if constexpr (I8)
          L.row[k - 2 * NS] = RowI8{(float)q8(__fmul_rn(__fmul_rn(dt, v), k0[i])), k1[i], decay * sC * k2[i],
                                    sC * sB * dt * v, Dv[i] * v, quant_decay(dt, Av[i]), {0.f, 0.f}};
        else
          L.row[k - 2 * NS] = RowF{decay, dt * v, Dv[i] * v, 0.f};
      }
      if (k >= 2 * NS || blk == 0) ((T*)a.cv.state)[(b * W + cur) * (int64_t)a.Cd + ch[i]] = cl[i].raw;
    }
  }
  __syncthreads();

  const int col = tid % R;  // R divides a wave: a thread keeps its columns
  if constexpr (I8) {
    // Q(B) . Q(C): every wave forms it from LDS
    int cb = 0;
#pragma unroll
    for (int n = 0; n < (NS + kWave - 1) / kWave; ++n) {
      const int k = lane_id() + n * kWave;
      if (NS % kWave == 0 || k < NS) cb += (int)L.b[k] * (int)L.qc[k];
    }
    cb = lane_sum_i<32>(cb);
    cb += __shfl_xor(cb, 32);
    float fb[16];
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const float4 v = *(const float4*)&L.b[16 * col + e];
      fb[e] = v.x; fb[e + 1] = v.y; fb[e + 2] = v.z; fb[e + 3] = v.w;
    }
    const uint4 qcv = *(const uint4*)&L.qc[16 * col];
    const uint32_t qcw[4] = {qcv.x, qcv.y, qcv.z, qcv.w};
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int s = tid + i * kStepThreads;
      const bool ok = s < slots;
      const int row = ok ? s / R : 0;
      const RowI8 rv = L.row[row];
      const v2s qd2 = {(short)rv.qd, (short)rv.qd};
      uint32_t nw[4];
      int acc = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t hw = hv[i][j];
        float c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = q8_pre(__fmul_rn(__fmul_rn(rv.qx, fb[4 * j + e]), rv.M));
        const v2s s01 = cvt_pair(c[0], c[1]), s23 = cvt_pair(c[2], c[3]);
        const v2s r01 = rsh7_pair(qd2, unpack_pair(hw, 0x010c000cu));
        const v2s r23 = rsh7_pair(qd2, unpack_pair(hw, 0x030c020cu));
        nw[j] = pack_pairs(sat127_pair(s01 + r01), sat127_pair(s23 + r23));
        acc = __builtin_amdgcn_sdot4((int)qcw[j], (int)hw, acc, false);
      }
      if (ok) __builtin_nontemporal_store((v4u){nw[0], nw[1], nw[2], nw[3]}, &st[s]);
      acc = lane_sum_i<R>(acc);
      if (ok && col == 0)
        ((T*)a.Y)[row0 + row] = to_store<DT>((float)acc * rv.f + (float)cb * rv.g + rv.Dx);
    }
  } else {
    const float4 bv = *(const float4*)&L.b[4 * col];
    const float4 cv = *(const float4*)&L.c[4 * col];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int s = tid + i * kStepThreads;
      const bool ok = s < slots;
      const int row = ok ? s / R : 0;
      const RowF rv = L.row[row];
      const v4f o = __builtin_bit_cast(v4f, hv[i]);
      v4f n;
      n[0] = fmaf(rv.decay, o[0], rv.dx * bv.x);
      n[1] = fmaf(rv.decay, o[1], rv.dx * bv.y);
      n[2] = fmaf(rv.decay, o[2], rv.dx * bv.z);
      n[3] = fmaf(rv.decay, o[3], rv.dx * bv.w);
      if (ok) __builtin_nontemporal_store(__builtin_bit_cast(v4u, n), &st[s]);
      const float acc = lane_sum_f<R>(cv.x * n[0] + cv.y * n[1] + cv.z * n[2] + cv.w * n[3]);
      if (ok && col == 0) ((T*)a.Y)[row0 + row] = to_store<DT>(acc + rv.Dx);
    }
  }
}

template <bool I8, int DT, int P, int NS, int HB>
hipError_t launch_hb(StepArgs& a, int64_t bg, hipStream_t st) {
  a.blocks = (a.hpg + HB - 1) / HB;
  hipLaunchKernelGGL((k_conv_decode<I8, DT, P, NS, HB>), dim3((unsigned)(bg * a.blocks)), dim3(kStepThreads), 0, st, a);
  return hipGetLastError();
}

// How many heads a workgroup takes: as many, up to 8 and 32 KB of state, as leave
// 4 workgroups on each CU and idle for less than a fifth; or, from 3 heads on each
// CU, as many as cost no more passes than one head does. Measured against one
// head (fp16 inputs, us): 114 heads of 16 x 32, 8-bit, batch 256 64 and 16 (8 of
// them), batch 16 6.8 and 4.1; 80 of 64 x 128, 8-bit, batch 256 87 and 76 (4), at
// batch 16 4 of them would take 12.8 instead of 9.8; 24 in 8 groups of 64 x 64,
// fp32, batch 256: 38, and 45 with 2; 108 of 32 x 32, fp32, batch 256 52 and 43.
// (A part of a head for each workgroup, where heads are fewer than CUs, gained
// nothing at 64 x 128.)
template <bool I8, int DT, int P, int NS, int HB>
hipError_t launch_n(StepArgs& a, int64_t B, hipStream_t st) {
  constexpr int kSlots = P * NS / (I8 ? 16 : 4);  // of a head
  if constexpr (HB > 1) {
    constexpr auto passes = [](int hb) {
      return (hb * kSlots + kStepThreads - 1) / kStepThreads + (hb * P + 2 * NS + kStepThreads - 1) / kStepThreads;
    };
    if constexpr (HB * kSlots <= 2048) {
      const int64_t ncu = cu_count() > 0 ? cu_count() : 256, blocks = (a.hpg + HB - 1) / HB;
      const bool full = 4 * HB * blocks <= 5 * (int64_t)a.hpg && B * a.G * blocks >= 4 * ncu;
      const bool free = passes(HB) == passes(1) && HB / 2 < a.hpg && B * a.H > 3 * ncu;
      if (full || free) return launch_hb<I8, DT, P, NS, HB>(a, B * a.G, st);
    }
    return launch_n<I8, DT, P, NS, HB / 2>(a, B, st);
  } else {
    return launch_hb<I8, DT, P, NS, 1>(a, B * a.G, st);
  }
}

template <int DT, int P>
hipError_t dispatch_n(bool int8, int N, StepArgs& a, int64_t B, hipStream_t st) {
  switch (N) {
    case 16: return int8 ? launch_n<true, DT, P, 16, 8>(a, B, st) : launch_n<false, DT, P, 16, 8>(a, B, st);
    case 32: return int8 ? launch_n<true, DT, P, 32, 8>(a, B, st) : launch_n<false, DT, P, 32, 8>(a, B, st);
    case 64: return int8 ? launch_n<true, DT, P, 64, 8>(a, B, st) : launch_n<false, DT, P, 64, 8>(a, B, st);
    case 128: return int8 ? launch_n<true, DT, P, 128, 8>(a, B, st) : launch_n<false, DT, P, 128, 8>(a, B, st);
    default: return hipErrorInvalidValue;
  }
}

template <int DT>
hipError_t dispatch_p(bool int8, int P, int N, StepArgs& a, int64_t B, hipStream_t st) {
  switch (P) {
    case 16: return dispatch_n<DT, 16>(int8, N, a, B, st);
    case 32: return dispatch_n<DT, 32>(int8, N, a, B, st);
    case 64: return dispatch_n<DT, 64>(int8, N, a, B, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_conv_decode_step(const Dims& d, int dtype, bool int8, const ConvPtrs& cv, const float* A,
                                   const float* D, const ScalePtrs& sc, void* state, void* Y,
                                   hipStream_t st) {
  StepArgs a{cv, A, D, sc, state, Y, d.H, d.G, d.hpg, d.H * d.P + 2 * d.G * d.N, 0};
  switch (dtype) {
    case DT_F32: return dispatch_p<DT_F32>(int8, d.P, d.N, a, d.B, st);
    case DT_F16: return dispatch_p<DT_F16>(int8, d.P, d.N, a, d.B, st);
    case DT_BF16: return dispatch_p<DT_BF16>(int8, d.P, d.N, a, d.B, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ssd
