// Matrix product in 8-bit integers with a step for each row of both operands:
//   out[m,n] = a_scale[m] w_scale[n] sum_k a[m,k] w[n,k] + bias[n]
// The sums are exact int32 MFMA sums; one fp32 epilogue per element.
#include "ssd_device.hpp"
#include "ssd_launch.hpp"

namespace ssd {
namespace {

typedef int v16i __attribute__((ext_vector_type(16)));

// 16 bytes per lane from global memory straight into LDS: lane i's bytes land
// at l + 16 i (l is uniform over the wave).
__device__ __forceinline__ void copy16_to_lds(const void* g, void* l) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                   (__attribute__((address_space(3))) void*)l, 16, 0, 0);
}

// Waits for every copy into LDS this wave has issued (vmcnt 0, the other
// counters as they are), then for the workgroup.
__device__ __forceinline__ void wait_copies_and_sync() {
  __builtin_amdgcn_s_waitcnt(0x0f70);
  __syncthreads();
}

__device__ __constant__ const uint4 kZero16 = {0, 0, 0, 0};

// ---------------------------------------------------------------------------
// large tiles
// ---------------------------------------------------------------------------
constexpr int kBM = 256, kBN = 256, kBK = 128;
constexpr int kBigThreads = 512;
constexpr int kTileA = kBM * kBK, kTileBytes = (kBM + kBN) * kBK;
constexpr int kStagePitch = 64 * 4 + 16;  // one row of 64 sums in the epilogue's staging

// The rows of both operands this lane copies, and their LDS homes. A tile row
// is 128 bytes, eight 16-byte chunks; chunk c of row r sits at slot c ^ (r % 8),
// so that the fragment reads of 8 consecutive rows meet 8 different slots (all
// of a row's banks). The copy fills LDS in lane order, so the lane that owns
// slot s of row r fetches chunk s ^ (r % 8).
struct BigCopy {
  unsigned oa[4], ow[4];  // byte offsets of the lane's chunk in rows of the tile
  int chunk;              // the lane's chunk, in bytes
  const int8_t *a, *w;
  int lds;  // the wave's first 1 KB
  __device__ __forceinline__ void init(const MatmulI8Args& g, int64_t m0, int64_t n0) {
    const int lane = lane_id(), wv = wave_id();
    chunk = ((lane & 7) ^ (lane >> 3)) * 16;
    a = g.a + m0 * g.K;
    w = g.w + n0 * g.K;
    lds = wv * 4 * 1024;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // rows past the edge stand in with the last one; their results are not stored
      const int row = (wv * 4 + i) * 8 + (lane >> 3);
      oa[i] = (unsigned)min((int64_t)row, g.M - 1 - m0) * (unsigned)g.K + chunk;
      ow[i] = (unsigned)min((int64_t)row, g.N - 1 - n0) * (unsigned)g.K + chunk;
    }
  }
  __device__ __forceinline__ void issue(int k, int K, int8_t* buf) const {
    if (k + kBK <= K) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        copy16_to_lds(a + k + oa[i], buf + lds + i * 1024);
        copy16_to_lds(w + k + ow[i], buf + kTileA + lds + i * 1024);
      }
    } else {
      // the chunks behind the end of the rows are zeros
      const bool in = k + chunk < K;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        copy16_to_lds(in ? (const void*)(a + k + oa[i]) : &kZero16, buf + lds + i * 1024);
        copy16_to_lds(in ? (const void*)(w + k + ow[i]) : &kZero16, buf + kTileA + lds + i * 1024);
      }
    }
  }
};

// One 128-byte step of the wave's 128 (n) x 64 (m) block from `cur`, with the
// copies into `nxt` in flight. The two buffers are distinct objects, which
// __restrict__ tells the compiler: it then needs no wait for those copies in
// front of the reads.
__device__ __forceinline__ void big_step(const int8_t* __restrict__ cur, int8_t* __restrict__ nxt,
                                         const BigCopy& cp, int knext, int K, int wm, int wn,
                                         v16i (&acc)[4][2]) {
  if (knext < K) cp.issue(knext, K, nxt);
  const int lane = lane_id();
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    const int slot = ((ks * 2 + (lane >> 5)) ^ (lane & 7)) * 16;
    v4i fw[4], fa[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) fw[i] = *(const v4i*)(cur + kTileA + (wn + 32 * i + (lane & 31)) * kBK + slot);
#pragma unroll
    for (int j = 0; j < 2; ++j) fa[j] = *(const v4i*)(cur + (wm + 32 * j + (lane & 31)) * kBK + slot);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[i], fa[j], acc[i][j], 0, 0, 0);
  }
}

// Eight consecutive outputs of a row from their sums.
template <int DT>
__device__ __forceinline__ void store8(const MatmulI8Args& g, int64_t m, int64_t n, const int* sum, const float* ws,
                                       const float* bias, bool wide) {
  const float as = g.a_scale[m];
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = fmaf((float)sum[e], as * ws[e], bias[e]);
  typename Store<DT>::T* const o = (typename Store<DT>::T*)g.out + m * g.N + n;
  if (wide) {
    if constexpr (DT == DT_F32) {
      *(v4f*)o = (v4f){y[0], y[1], y[2], y[3]};
      *(v4f*)(o + 4) = (v4f){y[4], y[5], y[6], y[7]};
    } else {
      *(v4u*)o = (v4u){pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3]), pack2<DT>(y[4], y[5]), pack2<DT>(y[6], y[7])};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (n + e < g.N) o[e] = to_store<DT>(y[e]);
  }
}

template <int DT>
__global__ __launch_bounds__(kBigThreads) void k_matmul_i8_big(MatmulI8Args g, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) int8_t buf0[kTileBytes], buf1[kTileBytes];
  // Consecutive workgroups go to the eight XCDs in turn; each XCD takes a
  // contiguous run of tiles, and walks it in columns of four row tiles, so
  // that the tiles an XCD computes together share rows in its L2.
  const int tiles = tiles_m * tiles_n;
  int t;
  {
    const int xcd = blockIdx.x % 8, i = blockIdx.x / 8, per = tiles / 8, more = tiles % 8;
    t = xcd * per + min(xcd, more) + i;
  }
  const int group = t / (4 * tiles_n), rows = min(4, tiles_m - group * 4), in = t - group * 4 * tiles_n;
  const int64_t m0 = (int64_t)(group * 4 + in % rows) * kBM, n0 = (int64_t)(in / rows) * kBN;

  const int lane = lane_id(), wv = wave_id();
  const int wm = (wv & 3) * 64, wn = (wv >> 2) * 128;
  const int K = (int)g.K;
  BigCopy cp;
  cp.init(g, m0, n0);
  v16i acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = (v16i)(0);
  cp.issue(0, K, buf0);
  wait_copies_and_sync();
  for (int k = 0; k < K; k += 2 * kBK) {
    big_step(buf0, buf1, cp, k + kBK, K, wm, wn, acc);
    wait_copies_and_sync();
    if (k + kBK < K) {
      big_step(buf1, buf0, cp, k + 2 * kBK, K, wm, wn, acc);
      wait_copies_and_sync();
    }
  }

  // Epilogue: a wave passes 32 (m) x 64 (n) sums at a time through its own part
  // of LDS, so that each row leaves as full 16-byte pieces.
  int8_t* const st = (wv < 4 ? buf0 : buf1) + (wv & 3) * (32 * kStagePitch);
  const bool wide_n = g.N % 8 == 0;
#pragma unroll
  for (int ih = 0; ih < 2; ++ih) {
    const int64_t n = n0 + wn + 64 * ih + (lane & 7) * 8;
    float ws[8], bias[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = min(n + e, g.N - 1);
      ws[e] = g.w_scale[c];
      bias[e] = g.bias ? g.bias[c] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const v16i& s = acc[ih * 2 + i2][j];
          *(v4i*)(st + (lane & 31) * kStagePitch + (32 * i2 + 8 * q + 4 * (lane >> 5)) * 4) =
              (v4i){s[4 * q], s[4 * q + 1], s[4 * q + 2], s[4 * q + 3]};
        }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = r * 8 + (lane >> 3);
        const int64_t m = m0 + wm + 32 * j + row;
        int sum[8];
        *(v4i*)sum = *(const v4i*)(st + row * kStagePitch + (lane & 7) * 32);
        *(v4i*)(sum + 4) = *(const v4i*)(st + row * kStagePitch + (lane & 7) * 32 + 16);
        if (m < g.M && n < g.N) store8<DT>(g, m, n, sum, ws, bias, wide_n);
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
  }
}

// ---------------------------------------------------------------------------
// small tiles
// ---------------------------------------------------------------------------
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

template <int DT>
hipError_t launch(const MatmulI8Args& g, hipStream_t st) {
  const int64_t tm = (g.M + kBM - 1) / kBM, tn = (g.N + kBN - 1) / kBN;
  if (tm * tn >= 128) {
    if (tm * tn >= (int64_t)1 << 23) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_matmul_i8_big<DT>, dim3((unsigned)(tm * tn)), dim3(kBigThreads), 0, st, g, (int)tm, (int)tn);
    return hipGetLastError();
  }
  const int64_t blocks = ((g.M + kTileM - 1) / kTileM) * ((g.N + kTileN - 1) / kTileN);
  if (blocks >= (int64_t)1 << 24) return hipErrorInvalidValue;
  hipLaunchKernelGGL(k_matmul_i8<DT>, dim3((unsigned)blocks), dim3(256), 0, st, g);
  return hipGetLastError();
}

}  // namespace

size_t matmul_i8_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_matmul_i8(int out_dtype, const MatmulI8Args& g, hipStream_t st) {
  switch (out_dtype) {
    case DT_F32: return launch<DT_F32>(g, st);
    case DT_F16: return launch<DT_F16>(g, st);
    case DT_BF16: return launch<DT_BF16>(g, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ssd
