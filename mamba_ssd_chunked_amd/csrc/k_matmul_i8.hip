// Matrix product in 8-bit integers with a step for each row of both operands:
//   out[m,n] = a_scale[m] w_scale[n] sum_k a[m,k] w[n,k] + bias[n]
// The sums are exact int32 MFMA sums; one fp32 epilogue per element.
#include "ssd_device.hpp"
#include "ssd_launch.hpp"

namespace ssd {
namespace {

constexpr int kTileM = 64, kTileN = 64, kTileK = 64, kPad = 16;

template <int DT>
__global__ __launch_bounds__(256) void k_matmul_i8(MatmulI8Args g) {
  __shared__ __attribute__((aligned(16))) int8_t sa[kTileM][kTileK + kPad];
  __shared__ __attribute__((aligned(16))) int8_t sw[kTileN][kTileK + kPad];
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_id();
  const int64_t tiles_n = (g.N + kTileN - 1) / kTileN;
  const int64_t m0 = (blockIdx.x / tiles_n) * kTileM, n0 = (blockIdx.x % tiles_n) * kTileN;
  const int lr = tid / 4, lc = (tid % 4) * 16;
  // rows past the edge stand in with the last one; their results are not stored
  const int8_t* pa = g.a + min(m0 + lr, g.M - 1) * g.K + lc;
  const int8_t* pw = g.w + min(n0 + lr, g.N - 1) * g.K + lc;
  const int wm = (wv / 2) * 32, wn = (wv % 2) * 32;
  v4i acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = (v4i){0, 0, 0, 0};
  for (int64_t k = 0; k < g.K; k += kTileK) {
    v4i va = {0, 0, 0, 0}, vw = {0, 0, 0, 0};
    if (k + lc < g.K) {
      va = *(const v4i*)(pa + k);
      vw = *(const v4i*)(pw + k);
    }
    __syncthreads();
    *(v4i*)&sa[lr][lc] = va;
    *(v4i*)&sw[lr][lc] = vw;
    __syncthreads();
    v4i fa[2], fw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fa[i] = *(const v4i*)&sa[wm + 16 * i + lane % 16][(lane / 16) * 16];
      fw[i] = *(const v4i*)&sw[wn + 16 * i + lane % 16][(lane / 16) * 16];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mma_i8(fa[i], fw[j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t n = n0 + wn + 16 * j + lane % 16;
      if (n >= g.N) continue;
      const float s = g.w_scale[n], bias = g.bias ? g.bias[n] : 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t m = m0 + wm + 16 * i + (lane / 16) * 4 + r;
        if (m < g.M)
          ((typename Store<DT>::T*)g.out)[m * g.N + n] = to_store<DT>(fmaf((float)acc[i][j][r], g.a_scale[m] * s, bias));
      }
    }
}

}  // namespace

size_t matmul_i8_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_matmul_i8(int out_dtype, const MatmulI8Args& g, hipStream_t st) {
  const int64_t blocks = ((g.M + kTileM - 1) / kTileM) * ((g.N + kTileN - 1) / kTileN);
  if (blocks >= (int64_t)1 << 24) return hipErrorInvalidValue;
  switch (out_dtype) {
    case DT_F32: hipLaunchKernelGGL(k_matmul_i8<DT_F32>, dim3((unsigned)blocks), dim3(256), 0, st, g); break;
    case DT_F16: hipLaunchKernelGGL(k_matmul_i8<DT_F16>, dim3((unsigned)blocks), dim3(256), 0, st, g); break;
    case DT_BF16: hipLaunchKernelGGL(k_matmul_i8<DT_BF16>, dim3((unsigned)blocks), dim3(256), 0, st, g); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace ssd
