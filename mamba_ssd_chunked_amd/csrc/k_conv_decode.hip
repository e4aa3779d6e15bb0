// Single-token step of the causal convolution and the SSD in one launch:
//
//   u[c] = sum_j w[c,j] (the last W inputs of channel c) + b[c],  x | B | C = silu(u)
//   dt = softplus(dt_raw + dt_bias),   then the step of k_decode.hip on x, B, C, dt
//
// with everything between the two kept in fp32. The state is read and written
// once and is by far the most of the traffic (at P = 64, N = 128 in fp32 64 KB
// a head against about 6 KB of the convolution's inputs, which the heads of a
// group share in the caches), so a large batch is bound by HBM and a small one
// by the latency of one pass.
//
// A workgroup of four waves per (batch, head). Its 16-byte slices of the state
// are requested first; then each thread computes the convolution of one or two
// of the P + 2 N channels that the head needs, into LDS. All W slots of the
// ring are loaded, and matched with their weights once pos has arrived, so the
// prologue costs one memory round trip, not two. The slot pos % W is written
// by the head itself for its x channels and by the first head of a group for
// B and C; nobody reads that slot's value, so heads need no order.
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
};

// The head's vectors after the convolution.
template <int P, int NS>
struct StepLds {
  float x[P];
  float bc[2 * NS];     // B, then C
  float4 rv[P];         // INT8, per state row: float(Q(Xs)), M_req, x, exp(dt A) s_C s_S
  float qb[NS];         // INT8: float(Q(B))
  int8_t qc[NS];        // INT8: Q(C)
  int cb[4];            // INT8: Q(B) . Q(C), a part of each wave
};

// One channel's convolution: the new input, the ring's W slots and the weights,
// loaded before any of them is used.
template <int DT>
struct ConvLane {
  float slot[4], w[4], bias, x;
  typename Store<DT>::T raw;
  __device__ __forceinline__ void load(const StepArgs& a, int64_t b, int c, int W) {
    raw = ((const typename Store<DT>::T*)a.cv.xbc)[b * a.cv.ld_xbc + c];
    const int64_t r = b * W * (int64_t)a.Cd + c;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      slot[s] = s < W ? ld_f<DT>(a.cv.state, r + (int64_t)s * a.Cd) : 0.f;
      w[s] = s < W ? a.cv.weight[(int64_t)c * W + s] : 0.f;
    }
    bias = a.cv.bias ? a.cv.bias[c] : 0.f;
    x = Store<DT>::to_f(raw);
  }
  // cur = pos % W; slots of positions before the sequence's start count as zero
  __device__ __forceinline__ float value(int W, uint32_t pos, int cur) const {
    float u = bias;
#pragma unroll
    for (int back = 3; back >= 1; --back) {
      if (back < W) {
        const int s = cur >= back ? cur - back : cur - back + W;
        const float v = s == 0 ? slot[0] : s == 1 ? slot[1] : s == 2 ? slot[2] : slot[3];
        const float wt = W == 4 ? w[3 - back] : W == 3 ? w[(2 - back) & 3] : w[(1 - back) & 3];
        if (pos >= (uint32_t)back) u = fmaf(wt, v, u);
      }
    }
    const float wt = W == 4 ? w[3] : W == 3 ? w[2] : w[1];
    return silu(fmaf(wt, x, u));
  }
};

template <bool I8, int DT, int P, int NS>
__global__ __launch_bounds__(kStepThreads) void k_conv_decode(StepArgs a) {
  typedef typename Store<DT>::T T;
  constexpr int R = NS / (I8 ? 16 : 4);                             // 16-byte slices of a state row
  constexpr int SLOTS = P * R;                                      // of the head
  constexpr int ITER = (SLOTS + kStepThreads - 1) / kStepThreads;   // of a thread
  constexpr int NCH = P + 2 * NS;
  constexpr int CIT = (NCH + kStepThreads - 1) / kStepThreads;
  __shared__ __attribute__((aligned(16))) StepLds<P, NS> L;

  const int tid = threadIdx.x;
  const int64_t unit = blockIdx.x;
  const int64_t b = unit / a.H;
  const int h = (int)(unit % a.H);
  const int g = h / a.hpg;
  v4u* const st = (v4u*)a.state + unit * (int64_t)SLOTS;

  v4u hv[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int s = tid + i * kStepThreads;
    if (SLOTS % kStepThreads == 0 || s < SLOTS) hv[i] = __builtin_nontemporal_load(&st[s]);
  }

  const int W = a.cv.width;
  const int dX = a.H * P, dBC = a.G * NS;
  ConvLane<DT> cl[CIT];
  int ch[CIT];
#pragma unroll
  for (int i = 0; i < CIT; ++i) {
    const int k = tid + i * kStepThreads;  // B, C, then x
    ch[i] = k < NS ? dX + g * NS + k : k < 2 * NS ? dX + dBC + g * NS + (k - NS) : h * P + (k - 2 * NS);
    if (k < NCH) cl[i].load(a, b, ch[i], W);
  }
  const uint32_t pos = (uint32_t)max(a.cv.pos[b], 0);
  const int cur = (int)(pos % (uint32_t)W);
  const float Ah = a.A[h], Dh = a.D[h];
  const float dtv = softplus(ld_f<DT>(a.cv.dt_raw, b * a.cv.ld_dt + h) + (a.cv.dt_bias ? a.cv.dt_bias[h] : 0.f));
  const float decay = __expf(dtv * Ah);
  float sC = 0.f;
  if constexpr (I8) sC = a.sc.s_C[g];

#pragma unroll
  for (int i = 0; i < CIT; ++i) {
    const int k = tid + i * kStepThreads;
    if (k < NCH) {
      const float v = cl[i].value(W, pos, cur);
      if (k < 2 * NS) {
        if constexpr (I8) {
          if (k < NS) L.qb[k] = (float)q8(__fmul_rn(v, a.sc.inv_B[g]));
          else L.qc[k - NS] = (int8_t)q8(__fmul_rn(v, a.sc.inv_C[g]));
        } else {
          L.bc[k] = v;
        }
      } else {
        const int p = k - 2 * NS;
        if constexpr (I8) {
          const int hp = h * P + p;
          const float qx = (float)q8(__fmul_rn(__fmul_rn(dtv, v), a.sc.inv_X[hp]));
          L.rv[p] = make_float4(qx, a.sc.M_req[hp], v, decay * sC * a.sc.s_S[hp]);
        } else {
          L.x[p] = v;
        }
      }
      if (k >= 2 * NS || h % a.hpg == 0) ((T*)a.cv.state)[(b * W + cur) * (int64_t)a.Cd + ch[i]] = cl[i].raw;
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
      if (NS % kWave == 0 || k < NS) cb += (int)L.qb[k] * (int)L.qc[k];
    }
    cb = lane_sum_i<32>(cb);
    cb += __shfl_xor(cb, 32);
    const int qd = (int)fmin(round(exp((double)dtv * (double)Ah) * 128.0), 128.0);
    float fb[16];
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const float4 v = *(const float4*)&L.qb[16 * col + e];
      fb[e] = v.x; fb[e + 1] = v.y; fb[e + 2] = v.z; fb[e + 3] = v.w;
    }
    const uint4 qcv = *(const uint4*)&L.qc[16 * col];
    const uint32_t qcw[4] = {qcv.x, qcv.y, qcv.z, qcv.w};
    const float ydiag = (float)cb * sC * a.sc.s_B[g] * dtv;
    const v2s qd2 = {(short)qd, (short)qd};
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int s = tid + i * kStepThreads;
      const bool ok = SLOTS % kStepThreads == 0 || s < SLOTS;
      const int row = ok ? s / R : 0;
      const float4 rv = L.rv[row];
      uint32_t nw[4];
      int acc = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t hw = hv[i][j];
        float c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = q8_pre(__fmul_rn(__fmul_rn(rv.x, fb[4 * j + e]), rv.y));
        const v2s s01 = cvt_pair(c[0], c[1]), s23 = cvt_pair(c[2], c[3]);
        const v2s r01 = rsh7_pair(qd2, unpack_pair(hw, 0x010c000cu));
        const v2s r23 = rsh7_pair(qd2, unpack_pair(hw, 0x030c020cu));
        nw[j] = pack_pairs(sat127_pair(s01 + r01), sat127_pair(s23 + r23));
        acc = __builtin_amdgcn_sdot4((int)qcw[j], (int)hw, acc, false);
      }
      if (ok) __builtin_nontemporal_store((v4u){nw[0], nw[1], nw[2], nw[3]}, &st[s]);
      acc = lane_sum_i<R>(acc);
      if (ok && col == 0)
        ((T*)a.Y)[unit * P + row] = to_store<DT>((float)acc * rv.w + ydiag * rv.z + Dh * rv.z);
    }
  } else {
    const float4 bv = *(const float4*)&L.bc[4 * col];
    const float4 cv = *(const float4*)&L.bc[NS + 4 * col];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int s = tid + i * kStepThreads;
      const bool ok = SLOTS % kStepThreads == 0 || s < SLOTS;
      const int row = ok ? s / R : 0;
      const float xv = L.x[row], dx = dtv * xv;
      const v4f o = __builtin_bit_cast(v4f, hv[i]);
      v4f n;
      n[0] = fmaf(decay, o[0], dx * bv.x);
      n[1] = fmaf(decay, o[1], dx * bv.y);
      n[2] = fmaf(decay, o[2], dx * bv.z);
      n[3] = fmaf(decay, o[3], dx * bv.w);
      if (ok) __builtin_nontemporal_store(__builtin_bit_cast(v4u, n), &st[s]);
      const float acc = lane_sum_f<R>(cv.x * n[0] + cv.y * n[1] + cv.z * n[2] + cv.w * n[3]);
      if (ok && col == 0) ((T*)a.Y)[unit * P + row] = to_store<DT>(acc + Dh * xv);
    }
  }
}

template <int DT, int P, int NS>
hipError_t launch_n(bool int8, const StepArgs& a, unsigned units, hipStream_t st) {
  if (int8)
    hipLaunchKernelGGL((k_conv_decode<true, DT, P, NS>), dim3(units), dim3(kStepThreads), 0, st, a);
  else
    hipLaunchKernelGGL((k_conv_decode<false, DT, P, NS>), dim3(units), dim3(kStepThreads), 0, st, a);
  return hipGetLastError();
}

template <int DT, int P>
hipError_t dispatch_n(bool int8, int N, const StepArgs& a, unsigned units, hipStream_t st) {
  switch (N) {
    case 16: return launch_n<DT, P, 16>(int8, a, units, st);
    case 32: return launch_n<DT, P, 32>(int8, a, units, st);
    case 64: return launch_n<DT, P, 64>(int8, a, units, st);
    case 128: return launch_n<DT, P, 128>(int8, a, units, st);
    default: return hipErrorInvalidValue;
  }
}

template <int DT>
hipError_t dispatch_p(bool int8, int P, int N, const StepArgs& a, unsigned units, hipStream_t st) {
  switch (P) {
    case 16: return dispatch_n<DT, 16>(int8, N, a, units, st);
    case 32: return dispatch_n<DT, 32>(int8, N, a, units, st);
    case 64: return dispatch_n<DT, 64>(int8, N, a, units, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_conv_decode_step(const Dims& d, int dtype, bool int8, const ConvPtrs& cv, const float* A,
                                   const float* D, const ScalePtrs& sc, void* state, void* Y,
                                   hipStream_t st) {
  StepArgs a{cv, A, D, sc, state, Y, d.H, d.G, d.hpg, d.H * d.P + 2 * d.G * d.N};
  const unsigned units = (unsigned)(d.B * d.H);
  switch (dtype) {
    case DT_F32: return dispatch_p<DT_F32>(int8, d.P, d.N, a, units, st);
    case DT_F16: return dispatch_p<DT_F16>(int8, d.P, d.N, a, units, st);
    case DT_BF16: return dispatch_p<DT_BF16>(int8, d.P, d.N, a, units, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ssd
