// The gated delta rule one position after the other: the step of single tokens,
// and the whole operator for the shortest sequences.
//   S' = a S + u k^T,  u = b (v - a S k),  y = scale S' q,   a = exp(dt A)
// on the state S [P, N] of each head in fp32. Both products of a position are taken
// with the state before it, y = scale (a S q + u k.q), so that the state is gone
// through once.
//
// A step is bound by the state, which is read and written once. A wave owns EL * 256
// of its elements (whole rows): lane i holds the 16 bytes i % R of row i / R of each
// of EL passes, R = N / 4, so that all accesses are whole lines, and the sums over a
// row cross R lanes. Everything is requested before anything is used, and the state goes
// past the caches. 256 sequences of 80 heads of 64 x 128, fp16: 220 us for 1348 MB, 6.1
// TB/s; one of 64 heads 4.1 us, which are a launch and two round trips to memory.
#include "ssd_delta.hpp"
#include "ssd_delta_kind.hpp"

namespace ssd {
namespace {

constexpr int kWaves = kDeltaStepWaves;

// A position's inputs, as a lane holds them.
template <int DT, int N, int EL>
struct DeltaRow {
  static constexpr int R = N / 4, RPI = kWave / R, XR = (EL + R - 1) / R;
  float4 k, q;
  float x[XR];  // of row i RPI + lane / R in the lanes i % R
  float dt, beta;
  __device__ __forceinline__ void load(const DeltaArgs& a, int64_t pos, int H, int G, int hpg, int h, int P, int row0) {
    const int lane = lane_id(), g = h / hpg;
    auto four = [&](const void* p) {
      const int64_t at = (pos * G + g) * N + (lane % R) * 4;
      if constexpr (DT == DT_F32) return *(const float4*)((const float*)p + at);
      else return make_float4(ld_f<DT>(p, at), ld_f<DT>(p, at + 1), ld_f<DT>(p, at + 2), ld_f<DT>(p, at + 3));
    };
    k = four(a.B);
    q = four(a.C);
    const int64_t head = pos * H + h;
#pragma unroll
    for (int j = 0; j < XR; ++j) {
      const int i = j * R + lane % R;  // the pass
      x[j] = i < EL ? ld_f<DT>(a.X, head * P + row0 + i * RPI + lane / R) : 0.f;
    }
    dt = ld_f<DT>(a.dt, head);
    beta = delta_beta<DT>(a, pos, h);
  }
};

__device__ __forceinline__ float dot4(float4 a, v4f b) { return a.x * b[0] + a.y * b[1] + a.z * b[2] + a.w * b[3]; }

// The factor that makes a vector of length 1 of one whose 4-vectors the lanes of a
// group hold. Where squares would leave fp32's range (fp16's cannot) the vector is
// scaled by a power of two first; small ones only where eps is as small.
template <int DT, int R>
__device__ __forceinline__ float unit_factor(float4& v, float eps) {
  auto sum = [&](float e) { return group_sum<R>(v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w) + e; };
  float s = sum(eps);
  if constexpr (DT != DT_F16) {
    if (!(s >= 0x1p-96f && s <= 0x1p120f)) {
      const float by = s > 1.f ? 0x1p-80f : 0x1p96f;
      v.x *= by; v.y *= by; v.z *= by; v.w *= by;
      s = sum(eps * by * by);
    }
  }
  return s > 0.f ? rsqrtf(s) : 0.f;  // a vector of zeros without eps stays zeros
}

template <int DT, int N, int EL>
__global__ __launch_bounds__(kWaves * kWave) void k_delta_step(DeltaArgs a, int64_t items, int64_t L, int H, int G,
                                                             int hpg, int P) {
  typedef DeltaRow<DT, N, EL> Row;
  constexpr int R = Row::R, RPI = Row::RPI, XR = Row::XR;
  const int lane = lane_id();
  const int64_t item = (int64_t)blockIdx.x * kWaves + wave_id();
  if (item >= items) return;
  const int parts = P / (EL * RPI);
  const int64_t unit = item / parts, b = unit / H;
  const int row0 = (int)(item % parts) * EL * RPI, h = (int)(unit % H);
  const int64_t at = (unit * P + row0) * (int64_t)N;

  v4f s[EL];
  if (a.init) {
    const v4f* const p = (const v4f*)(a.init + at) + lane;
#pragma unroll
    for (int i = 0; i < EL; ++i) s[i] = __builtin_nontemporal_load(p + i * kWave);
  } else {
#pragma unroll
    for (int i = 0; i < EL; ++i) s[i] = (v4f)(0.f);
  }
  const float A = a.A[h];
  Row nxt;
  if (L > 0) nxt.load(a, b * L, H, G, hpg, h, P, row0);
  for (int64_t t = 0; t < L; ++t) {
    Row r = nxt;
    if (t + 1 < L) nxt.load(a, b * L + t + 1, H, G, hpg, h, P, row0);
    if (a.unit) {
      const float fk = unit_factor<DT, R>(r.k, a.eps);
      const float fq = unit_factor<DT, R>(r.q, a.eps);
      r.k.x *= fk; r.k.y *= fk; r.k.z *= fk; r.k.w *= fk;
      r.q.x *= fq; r.q.y *= fq; r.q.z *= fq; r.q.w *= fq;
    }
    const float kq = group_sum<R>(r.k.x * r.q.x + r.k.y * r.q.y + r.k.z * r.q.z + r.k.w * r.q.w);
    const float decay = expf(r.dt * A);
    // what a key of zeros would write is nothing, whatever stands behind a sequence's end in
    // beta and the values
    const bool writes = __ballot(r.k.x != 0.f || r.k.y != 0.f || r.k.z != 0.f || r.k.w != 0.f) != 0;
    float y[XR];
#pragma unroll
    for (int j = 0; j < XR; ++j) y[j] = 0.f;
#pragma unroll
    for (int i = 0; i < EL; ++i) {
      const float sk = group_sum<R>(dot4(r.k, s[i])), sq = group_sum<R>(dot4(r.q, s[i]));
      const float x = __shfl(r.x[i / R], (lane & ~(R - 1)) + i % R);
      const float u = writes ? r.beta * fmaf(-decay, sk, x) : 0.f;
      s[i][0] = fmaf(decay, s[i][0], u * r.k.x);
      s[i][1] = fmaf(decay, s[i][1], u * r.k.y);
      s[i][2] = fmaf(decay, s[i][2], u * r.k.z);
      s[i][3] = fmaf(decay, s[i][3], u * r.k.w);
      const float v = a.scale * fmaf(decay, sq, u * kq);
      y[i / R] = lane % R == i % R ? v : y[i / R];
    }
    const int64_t head = (b * L + t) * H + h;
#pragma unroll
    for (int j = 0; j < XR; ++j) {
      const int i = j * R + lane % R;
      if (i < EL) ((typename Store<DT>::T*)a.Y)[head * P + row0 + i * RPI + lane / R] = to_store<DT>(y[j]);
    }
  }
  if (a.final_state) {
    v4f* const p = (v4f*)(a.final_state + at) + lane;
#pragma unroll
    for (int i = 0; i < EL; ++i) __builtin_nontemporal_store(s[i], p + i * kWave);
  }
}

template <int DT, int N, int EL>
hipError_t go(const Dims& d, const DeltaArgs& a, hipStream_t st) {
  const int64_t items = delta_step_items(d.B * d.H, d.P, N, EL);
  hipLaunchKernelGGL((k_delta_step<DT, N, EL>), dim3((unsigned)delta_step_wgs(items)), dim3(kWaves * kWave), 0, st, a, items,
                     d.L, d.H, d.G, d.hpg, d.P);
  return hipGetLastError();
}

template <int DT, int N>
hipError_t pick(const Dims& d, const DeltaArgs& a, hipStream_t st) {
  const int el = delta_step_passes(d.B * (int64_t)d.H, d.L, d.P, N, cu_count() > 0 ? cu_count() : 256);
  switch (el) {
    case 1: return go<DT, N, 1>(d, a, st);
    case 2: return go<DT, N, 2>(d, a, st);
    case 4: return go<DT, N, 4>(d, a, st);
    default: return go<DT, N, 8>(d, a, st);
  }
}

template <int DT>
hipError_t pick_n(const Dims& d, const DeltaArgs& a, hipStream_t st) {
  switch (d.N) {
    case 16: return pick<DT, 16>(d, a, st);
    case 32: return pick<DT, 32>(d, a, st);
    case 64: return pick<DT, 64>(d, a, st);
    case 128: return pick<DT, 128>(d, a, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_delta_steps(const Dims& d, int dtype, const DeltaArgs& a, hipStream_t st) {
  switch (dtype) {
    case DT_F32: return pick_n<DT_F32>(d, a, st);
    case DT_F16: return pick_n<DT_F16>(d, a, st);
    case DT_BF16: return pick_n<DT_BF16>(d, a, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ssd
