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

__device__ __constant__ const uint4 kZero16 = {0, 0, 0, 0};

// A pointer that is the same in all lanes, in scalar registers.
__device__ __forceinline__ const int8_t* uniform_ptr(const int8_t* p) {
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v), hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (const int8_t*)((uint64_t)hi << 32 | lo);
}

// ---------------------------------------------------------------------------
// large tiles
// ---------------------------------------------------------------------------
constexpr int kBM = 256, kBN = 256, kBK = 128;
constexpr int kBigThreads = 512;
constexpr int kTileA = kBM * kBK, kTileBytes = (kBM + kBN) * kBK;
constexpr int kStage = 32 * 128;  // a wave's part of the epilogue's staging: 32 rows of 128 bytes

// The rows of both operands this lane copies, and their LDS homes. A tile row
// is 128 bytes, eight 16-byte chunks; two rows cover the 64 banks. Chunk c of
// row r sits at slot c ^ (r / 2 % 8), so that the fragment reads of 16
// consecutive rows meet every bank once. The copy fills LDS in lane order, so
// the lane that owns slot s of row r fetches chunk s ^ (r / 2 % 8). TAIL: the
// rows are not a whole number of steps long; chunks behind their end are zeros.
template <bool TAIL>
struct BigCopy {
  unsigned o[4];  // byte offsets of the lane's chunks in the tile's rows of either operand
  const int8_t *a, *w;
  __device__ __forceinline__ int chunk(int i) const {
    return ((lane_id() & 7) ^ (lane_id() >> 4)) * 16 ^ ((i & 1) * 64);
  }
  __device__ __forceinline__ void init(const MatmulI8Args& g, int m0, int n0) {
    a = g.a + (int64_t)m0 * g.K;
    w = g.w + (int64_t)n0 * g.K;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = ((wave_id() * 4 + i) * 8 + (lane_id() >> 3)) * (unsigned)g.K + chunk(i);
  }
  __device__ __forceinline__ void issue(int k, int K, int8_t* buf) const {
    int8_t* const la = buf + wave_id() * 4096;
    const int8_t* const pa = uniform_ptr(a + k);
    const int8_t* const pw = uniform_ptr(w + k);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TAIL) {
        const bool in = k + chunk(i) < K;
        copy16_to_lds(in ? (const void*)(pa + o[i]) : &kZero16, la + i * 1024);
        copy16_to_lds(in ? (const void*)(pw + o[i]) : &kZero16, la + kTileA + i * 1024);
      } else {
        copy16_to_lds(pa + o[i], la + i * 1024);
        copy16_to_lds(pw + o[i], la + kTileA + i * 1024);
      }
    }
  }
};

// The operands of one 32-byte step of a wave's 128 (n) x 64 (m) block.
struct BigFrags {
  v4i w[4], a[2];
  __device__ __forceinline__ void load(const int8_t* buf, int ks, int wm, int wn) {
    const int lane = lane_id(), slot = ((ks * 2 + (lane >> 5)) ^ ((lane >> 1) & 7)) * 16;
#pragma unroll
    for (int j = 0; j < 2; ++j) a[j] = *(const v4i*)(buf + (wm + 32 * j + (lane & 31)) * kBK + slot);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *(const v4i*)(buf + kTileA + (wn + 32 * i + (lane & 31)) * kBK + slot);
  }
  __device__ __forceinline__ void multiply(v16i (&acc)[4][2]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[i], a[j], acc[i][j], 0, 0, 0);
  }
};

// One 128-byte step from `cur`, whose first operands are in f[0]. The operands
// of each 32-byte step are read while the products of the one before run. The
// last products run behind the barrier, and cover what follows it: the first
// reads of `nxt`, whose copies the barrier has seen arrive, and the copies of
// the step after it into `cur`, which nobody reads any more.
template <bool TAIL>
__device__ __forceinline__ void big_step(int8_t* cur, const int8_t* nxt, const BigCopy<TAIL>& cp, int k, int K,
                                         int wm, int wn, BigFrags (&f)[2], v16i (&acc)[4][2]) {
#pragma unroll
  for (int ks = 0; ks < 3; ++ks) {
    f[(ks + 1) & 1].load(cur, ks + 1, wm, wn);
    f[ks & 1].multiply(acc);
#pragma unroll
    for (int q = 0; q < 6; ++q) {  // a read, a product, ...
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  // vmcnt(0) lgkmcnt(0): this wave's copies into nxt have arrived, its reads of
  // cur have too. (A plain __syncthreads would do as well.)
  __builtin_amdgcn_s_waitcnt(0x0070);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  f[0].load(nxt, 0, wm, wn);
  cp.issue(k, K, cur);
  f[1].multiply(acc);
  __builtin_amdgcn_sched_barrier(0);
}

// 128 consecutive bytes of outputs of 32 rows at a time: the lane's sums are
// scaled and rounded, pass through the wave's own staging rows (16-byte chunk c
// of row r at slot c ^ (r / 2 % 8)), and leave as whole pieces of rows.
template <int DT, bool BIAS>
__device__ __forceinline__ void big_store(const MatmulI8Args& g, int m0, int n0, int wm, int wn, int8_t* st,
                                          const v16i (&acc)[4][2]) {
  typedef typename Store<DT>::T T;
  typedef const __attribute__((address_space(4))) float* scalar_ptr;
  constexpr int U = DT == DT_F32 ? 1 : 2;  // 32-column blocks of a piece
  constexpr int E = 16 / sizeof(T);        // outputs of a 16-byte chunk
  const int lane = lane_id(), hi = lane >> 5;
  const bool wide = g.N % E == 0;
  const int row = lane & 31, swz = (row >> 1) & 7;
  const unsigned lane_at = ((lane >> 3) * (unsigned)g.N + (lane & 7) * E) * sizeof(T);
  // The columns' steps come through the scalar cache (they are the same for all
  // lanes of a half wave): vector loads would queue behind the stores.
  auto columns = [&](const float* p, float (&v)[U][4][4]) {
    const scalar_ptr s = (scalar_ptr)(uint64_t)uniform_ptr((const int8_t*)p);
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float lo4 = s[32 * i + 8 * q + e], hi4 = s[32 * i + 8 * q + 4 + e];
          asm("" : "+s"(lo4), "+s"(hi4));  // both are loaded: no lane-wise address
          v[i][q][e] = hi ? hi4 : lo4;
        }
  };
  float as[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) as[j] = g.a_scale[m0 + wm + 32 * j + row];
#pragma unroll
  for (int u = 0; u < 4 / U; ++u) {
    const int nu = n0 + wn + 32 * U * u;
    float ws[U][4][4], bias[U][4][4];
    columns(g.w_scale + nu, ws);
    if constexpr (BIAS) columns(g.bias + nu, bias);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const v16i& s = acc[U * u + i][j];
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float sum = (float)s[4 * q + e], step = as[j] * ws[i][q][e];
            if constexpr (BIAS) y[e] = fmaf(sum, step, bias[i][q][e]);
            else y[e] = sum * step;
          }
          if constexpr (DT == DT_F32) {
            *(v4f*)(st + row * 128 + ((2 * q + hi) ^ swz) * 16) = (v4f){y[0], y[1], y[2], y[3]};
          } else {
            *(uint2*)(st + row * 128 + ((4 * i + q) ^ swz) * 16 + hi * 8) =
                make_uint2(pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3]));
          }
        }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int orow = r * 8 + (lane >> 3);
        const v4u v = *(const v4u*)(st + orow * 128 + ((lane & 7) ^ ((orow >> 1) & 7)) * 16);
        // the rows' address is uniform, the lane's place in them fits 32 bits
        T* const o = (T*)(const_cast<int8_t*>(uniform_ptr((const int8_t*)g.out + ((int64_t)(m0 + wm + 32 * j + 8 * r) * g.N + nu) * sizeof(T))) + lane_at);
        if (wide) {
          *(v4u*)o = v;
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if constexpr (DT == DT_F32) ((uint32_t*)o)[e] = v[e];
            else ((u16*)o)[e] = (u16)(v[e >> 1] >> (16 * (e & 1)));
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
  }
}

// One workgroup per CU walks its tiles; the copies of the next tile's first
// steps run under the epilogue of this one's.
template <int DT, bool TAIL, bool BIAS>
__global__ __launch_bounds__(kBigThreads, 2) void k_matmul_i8_big(MatmulI8Args g, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) int8_t buf0[kTileBytes], buf1[kTileBytes];
  __shared__ __attribute__((aligned(1024))) int8_t stage[8 * kStage];
  // Consecutive workgroups go to the eight XCDs in turn. Each XCD takes a
  // contiguous run of the tiles, which its workgroups walk together, in columns
  // of four row tiles: the tiles that an XCD computes at a time share rows in
  // its L2.
  const int tiles = tiles_m * tiles_n;
  const int xcd = blockIdx.x % 8, nwg = (gridDim.x - xcd + 7) / 8;
  const int lo = (int)((int64_t)tiles * xcd / 8), hi = (int)((int64_t)tiles * (xcd + 1) / 8);
  int t = lo + blockIdx.x / 8;
  if (t >= hi) return;
  auto place = [&](int t, int& m0, int& n0) {
    const int group = t / (4 * tiles_n), rows = min(4, tiles_m - group * 4), in = t - group * 4 * tiles_n;
    // the last tiles end with the matrix: what they share with the tiles before
    // is written twice, with the same bits
    m0 = min((group * 4 + in % rows) * kBM, (int)g.M - kBM);
    n0 = min((in / rows) * kBN, (int)g.N - kBN);
  };
  int m0, n0;
  place(t, m0, n0);
  const int wv = wave_id(), wm = (wv & 3) * 64, wn = (wv >> 2) * 128;
  const int K = (int)g.K;
  BigCopy<TAIL> cp;
  cp.init(g, m0, n0);
  cp.issue(0, K, buf0);
  __builtin_amdgcn_s_waitcnt(0x0f70);
  __syncthreads();
  cp.issue(kBK, K, buf1);
  BigFrags f[2];
  f[0].load(buf0, 0, wm, wn);
  for (;;) {
    const int tn = t + nwg;
    int m1 = m0, n1 = n0;
    if (tn < hi) place(tn, m1, n1);
    v16i acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = (v16i)(0);
    // pairs of steps; where the rows end inside a pair its rest is zeros (TAIL)
    for (int k = 0; k < K; k += 2 * kBK) {
      int kn = k + 2 * kBK;
      if (kn >= K) {  // the next tile's first steps (the last tile's once more: read by nobody)
        cp.init(g, m1, n1);
        kn = 0;
      }
      big_step<TAIL>(buf0, buf1, cp, kn, K, wm, wn, f, acc);
      big_step<TAIL>(buf1, buf0, cp, kn + kBK, K, wm, wn, f, acc);
    }
    big_store<DT, BIAS>(g, m0, n0, wm, wn, stage + wv * kStage, acc);
    if (tn >= hi) break;
    t = tn;
    m0 = m1;
    n0 = n1;
  }
  // no copy may still be on its way when the workgroup's LDS goes to another
  __builtin_amdgcn_s_waitcnt(0x0f70);
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
  if (g.M >= kBM && g.N >= kBN && tm * tn >= 128) {
    const int64_t ncu = cu_count() > 0 ? cu_count() : 256;
    const dim3 grid((unsigned)min(tm * tn, ncu));
#define BIG_(TAIL_, BIAS_) \
  hipLaunchKernelGGL((k_matmul_i8_big<DT, TAIL_, BIAS_>), grid, dim3(kBigThreads), 0, st, g, (int)tm, (int)tn)
    if (g.K % (2 * kBK) == 0) {
      if (g.bias) BIG_(false, true);
      else BIG_(false, false);
    } else {
      if (g.bias) BIG_(true, true);
      else BIG_(true, false);
    }
#undef BIG_
    return hipGetLastError();
  }
  const int64_t blocks = ((g.M + kTileM - 1) / kTileM) * ((g.N + kTileN - 1) / kTileN);
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
