// Matrix product with its epilogue:
//   out[m,n] = act(sum_k a[m,k] w[n,k] + bias[n]) + residual[m,n]
// in fp16, bf16 or fp32. Sums, bias, activation and residual are fp32 (the products of
// 16-bit elements are exact in it), rounded once. fp32 operands take the fp32 matrix
// instructions, an 8th of the rate for each byte.
//
// Rows that are 16-byte aligned and long take the ways of the 8-bit product
// (ssd_matmul.hpp): a 128-byte step is 64 positions of 16-bit rows, with the same matrix
// cycles, LDS reads and copies as 128 of 8-bit ones, and the same choice of kernel by
// the rows' bytes (over 90 products of 1 to 16384 rows, N 16 to 18560 and K 64 to 8192 it
// takes 2.4 % more than the best kernel in the geometric mean, 35 % at most: 5127 x 240 x 1024
// 16 us in blocks of 64, 12 in 128). Others go through registers, in pieces of 16 bytes at
// any element's address, the last of a row element by element; or, where the caller gives
// room for it, 16-bit ones are copied into aligned rows first: loads at odd multiples of 2
// bytes cost more than a pass over w does (fp32 rows, whose loads are at multiples of 4 bytes,
// lose by it: 1065 x 4099 x 2579 337 us against 231).
//
// us, and the sum's rate (a large library product: 1500 TF in fp16, 1600 in bf16; a
// copy: 5.1 TB/s):
//   8 x 2560 x 5120 bf16          6.6, bound by w: 4.0 TB/s
//   333 x 8512 x 2048 bf16        20 to 21, 570 TF; 201 blocks of 128 for 256 CUs
//   16384 x 10576 x 2560 fp16     785 to 825, 1100 TF; products, 8 waves' barriers between them
//   4096 x 4096 x 1024 fp32       243, 141 TF of 153
//   1065 x 4099 x 2579 bf16, with bias, GELU and an fp32 residual  62, of which the copies 12
#include "ssd_act.hpp"
#include "ssd_launch.hpp"
#include "ssd_matmul.hpp"
#include "ssd_matmul_kind.hpp"

namespace ssd {
namespace {

template <int DT>
struct OpFloat {
  typedef v16f Acc32;
  typedef v4f Acc16;
  static constexpr int kInstructions = DT == DT_F32 ? 4 : 1;  // of a product
  static __device__ __forceinline__ Acc32 mma32(v4i a, v4i b, Acc32 c) {
    if constexpr (DT == DT_F16) {
      return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
    } else if constexpr (DT == DT_BF16) {
      return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
    } else {
      const v4f x = __builtin_bit_cast(v4f, a), y = __builtin_bit_cast(v4f, b);
#pragma unroll
      for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[e], y[e], c, 0, 0, 0);
      return c;
    }
  }
  static __device__ __forceinline__ Acc16 mma16(v4i a, v4i b, Acc16 c) {
    if constexpr (DT == DT_F16) {
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
    } else if constexpr (DT == DT_BF16) {
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
    } else {
      const v4f x = __builtin_bit_cast(v4f, a), y = __builtin_bit_cast(v4f, b);
#pragma unroll
      for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], c, 0, 0, 0);
      return c;
    }
  }
};

// ---------------------------------------------------------------------------
// large tiles
// ---------------------------------------------------------------------------
// 128 consecutive bytes of outputs of 32 rows at a time, through the wave's own staging
// rows (16-byte chunk c of row r at slot c ^ (r / 2 % 8)): in come the residual's, whole
// pieces of rows; each lane adds its sums to the ones that it finds at its places; out
// go the results the same way.
template <int OT, int NW>
__device__ __forceinline__ void tile_store(const MatmulArgs& g, int m0, int n0, int mb, int nb, int wm, int wn,
                                           int8_t* st, const v16f (&acc)[Tile<NW>::TI][2]) {
  typedef typename Store<OT>::T T;
  typedef const __attribute__((address_space(4))) float* scalar_ptr;
  typedef __attribute__((address_space(1))) v4u_any* global_out;
  typedef const __attribute__((address_space(1))) v4u_any* global_in;
  constexpr int U = OT == DT_F32 ? 1 : 2;  // 32-column blocks of a piece
  constexpr int E = 16 / sizeof(T);        // outputs of a 16-byte chunk
  const int lane = lane_id(), hi = lane >> 5;
  const int row = lane & 31, swz = (row >> 1) & 7;
  const unsigned lane_at = ((lane >> 3) * (unsigned)g.N + (lane & 7) * E) * sizeof(T);
  auto meet = [] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  auto slot = [&](int r) { return (v4u*)(st + r * 128 + ((lane & 7) ^ ((r >> 1) & 7)) * 16); };
  // Where the residual is the output, what another tile may have written already must
  // not be written again.
  const bool once = g.residual == g.out && (mb > m0 || nb > n0);
  // whole lines go past the caches, as the 8-bit product's
  const bool lines = ((uint64_t)g.out | g.N * sizeof(T)) % 128 == 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
#pragma unroll
    for (int u = 0; u < Tile<NW>::TI / U; ++u) {
      const int nu = n0 + wn + 32 * U * u;
      auto rows = [&](const void* p, int r) {  // the rows' address is uniform, the lane's place in them fits 32 bits
        return (int8_t*)uniform_ptr((const int8_t*)p + ((int64_t)(m0 + wm + 32 * j + 8 * r) * g.N + nu) * sizeof(T)) + lane_at;
      };
      if (g.residual) {
        v4u v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = *(global_in)(uint64_t)rows(g.residual, r);
#pragma unroll
        for (int r = 0; r < 4; ++r) *slot(r * 8 + (lane >> 3)) = v[r];
        meet();
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = acc[U * u + i][j][e];
        if (g.bias) {
          const scalar_ptr s = (scalar_ptr)(uint64_t)uniform_ptr((const int8_t*)(g.bias + nu + 32 * i));
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float lo4 = s[8 * q + e], hi4 = s[8 * q + 4 + e];
              asm("" : "+s"(lo4), "+s"(hi4));  // both are loaded: no lane-wise address
              y[4 * q + e] += hi ? hi4 : lo4;
            }
        }
        if (g.act) activate(g.act, y);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (OT == DT_F32) {
            v4f* const at = (v4f*)(st + row * 128 + ((2 * q + hi) ^ swz) * 16);
            v4f v = {y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]};
            if (g.residual) v += *at;
            *at = v;
          } else {
            uint2* const at = (uint2*)(st + row * 128 + ((4 * i + q) ^ swz) * 16 + hi * 8);
            if (g.residual) {
              const uint2 r = *at;
              y[4 * q] += Store<OT>::to_f(__builtin_bit_cast(T, (u16)(r.x & 0xffff)));
              y[4 * q + 1] += Store<OT>::to_f(__builtin_bit_cast(T, (u16)(r.x >> 16)));
              y[4 * q + 2] += Store<OT>::to_f(__builtin_bit_cast(T, (u16)(r.y & 0xffff)));
              y[4 * q + 3] += Store<OT>::to_f(__builtin_bit_cast(T, (u16)(r.y >> 16)));
            }
            *at = make_uint2(pack2<OT>(y[4 * q], y[4 * q + 1]), pack2<OT>(y[4 * q + 2], y[4 * q + 3]));
          }
        }
      }
      meet();
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const v4u v = *slot(r * 8 + (lane >> 3));
        const global_out o = (global_out)(uint64_t)rows(g.out, r);
        if (once) {
          const int first = nb - (nu + (lane & 7) * E);  // of the chunk's outputs
          if (m0 + wm + 32 * j + 8 * r + (lane >> 3) < mb || first >= E) continue;
          const T* const from = (const T*)slot(r * 8 + (lane >> 3));
          for (int e = max(first, 0); e < E; ++e) ((T*)(rows(g.out, r)))[e] = from[e];
        } else if (lines) {
          asm volatile("; lines");  // without these the compiler makes one store of the two
          __builtin_nontemporal_store(v, o);
          asm volatile("; lines");
        } else {
          *o = v;
        }
      }
      meet();
    }
  }
}

template <int DT, int OT, bool TAIL, int NW, int S>
__global__ __launch_bounds__(64 * NW, (kTileWgs<NW, S> * NW / 4)) void k_matmul_tile(MatmulArgs g, int tiles_m,
                                                                                  int tiles_n) {
  constexpr int E = sizeof(typename Store<DT>::T);
  tile_walk<OpFloat<DT>, TAIL, false, NW, S>(
      g, (int)g.K * E, g.lda * E, tiles_m, tiles_n,
      [&](int m0, int n0, int mb, int nb, int wm, int wn, int8_t* stage,
          const v16f (&acc)[Tile<NW>::TI][2]) __attribute__((always_inline)) {
        tile_store<OT, NW>(g, m0, n0, mb, nb, wm, wn, stage, acc);
      });
}

// ---------------------------------------------------------------------------
// other outputs: four consecutive ones of a row in a lane
// ---------------------------------------------------------------------------
template <int OT>
__device__ __forceinline__ void finish4(const MatmulArgs& g, int m, int n, float (&y)[4]) {
  const int left = (int)g.N - n;
  const int64_t o = (int64_t)m * g.N + n;
  if (g.bias) {
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] += g.bias[min(n + e, (int)g.N - 1)];
  }
  if (g.act) activate(g.act, y);
  if (g.residual) {
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] += e < left ? ld_f<OT>(g.residual, o + e) : 0.f;
  }
  store4<OT>(g.out, o, y, left);
}

template <int DT, int OT, int MT, int NT, int NW, int D>
__global__ __launch_bounds__(64 * NW) void k_matmul_rows(MatmulArgs g, int blocks_m) {
  constexpr int E = sizeof(typename Store<DT>::T);
  few_rows<OpFloat<DT>, MT, NT, NW, D>(g, (int)g.K * E, g.lda * E, blocks_m, [&](int m, int n, v4f sum) __attribute__((always_inline)) {
    float y[4] = {sum[0], sum[1], sum[2], sum[3]};
    finish4<OT>(g, m, n, y);
  });
}

// ---------------------------------------------------------------------------
// rows at any alignment, of any length
// ---------------------------------------------------------------------------
// 16 bytes of a row from element k on; what lies behind the row's end is zero.
template <int DT>
__device__ __forceinline__ v4i load_any(const void* row, int k, int K) {
  constexpr int E = 16 / sizeof(typename Store<DT>::T);
  const typename Store<DT>::T* const p = (const typename Store<DT>::T*)row + k;
  if (k + E <= K) return __builtin_bit_cast(v4i, *(const v4u_any*)p);
  union {
    typename Store<DT>::T t[E];
    v4i v;
  } u;
  u.v = (v4i)(0);
#pragma unroll
  for (int e = 0; e < E - 1; ++e)
    if (k + e < K) u.t[e] = p[e];
  return u.v;
}

// Aligned copies of rows: a wave a row, its end filled up with zeros to Kp elements.
struct PackRows {
  const void* from;
  int64_t ld, rows;
  void* to;
};
template <int DT>
__global__ __launch_bounds__(256) void k_matmul_pack(PackRows a, PackRows w, int K, int Kp) {
  typedef typename Store<DT>::T T;
  constexpr int E = 16 / sizeof(T);
  for (int64_t r = (int64_t)blockIdx.x * 4 + wave_id(); r < a.rows + w.rows; r += (int64_t)gridDim.x * 4) {
    const bool second = r >= a.rows;
    const int64_t row = second ? r - a.rows : r;
    const T* const from = (const T*)(second ? w.from : a.from) + row * (second ? w.ld : a.ld);
    T* const to = (T*)(second ? w.to : a.to) + row * Kp;
    for (int k = lane_id() * E; k < Kp; k += kWave * E) *(v4i*)(to + k) = load_any<DT>(from, k, K);
  }
}

// A workgroup of four waves takes 64 TS rows and columns, a wave 32 TS of each. The
// operands of a step of 128 bytes pass through registers into one of two buffers in LDS
// (slots as the tiles') while the step before is multiplied.
template <int DT, int OT, int TS>
__global__ __launch_bounds__(256, 2) void k_matmul_any(MatmulArgs g, int blocks_m) {
  typedef OpFloat<DT> Op;
  typedef typename Store<DT>::T T;
  constexpr int kSide = 64 * TS, kStep = 128 / sizeof(T), kPer = 2 * TS;  // chunks of an operand a thread copies
  __shared__ __attribute__((aligned(1024))) int8_t buf[2][2 * kSide * kBK];
  const int lane = lane_id(), wv = wave_id(), tid = threadIdx.x;
  // XCDs take contiguous runs of the blocks, as in the few-rows kernels
  const int xcd = blockIdx.x % 8, per = (int)gridDim.x / 8, more = (int)gridDim.x % 8;
  const int t = xcd * per + min(xcd, more) + (int)blockIdx.x / 8;
  const int n0 = t / blocks_m * kSide, m0 = t % blocks_m * kSide;
  const int K = (int)g.K, steps = (K + kStep - 1) / kStep;
  // rows past the edge stand in with the last one; their results are not stored
  const T *ra[kPer], *rw[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = (i * 256 + tid) >> 3;
    ra[i] = (const T*)g.a + (int64_t)min(m0 + r, (int)g.M - 1) * g.lda;
    rw[i] = (const T*)g.w + (int64_t)min(n0 + r, (int)g.N - 1) * K;
  }
  v4i va[kPer], vw[kPer];
  auto load = [&](int step) {
    const int k = step * kStep + (tid & 7) * (16 / (int)sizeof(T));
    if ((step + 1) * kStep <= K) {  // the same for all threads: no piece ends early
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        va[i] = __builtin_bit_cast(v4i, *(const v4u_any*)(ra[i] + k));
        vw[i] = __builtin_bit_cast(v4i, *(const v4u_any*)(rw[i] + k));
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        va[i] = load_any<DT>(ra[i], k, K);
        vw[i] = load_any<DT>(rw[i], k, K);
      }
    }
  };
  auto put = [&](int8_t* b) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = (i * 256 + tid) >> 3, at = r * kBK + ((tid & 7) ^ ((r >> 1) & 7)) * 16;
      *(v4i*)(b + at) = va[i];
      *(v4i*)(b + kSide * kBK + at) = vw[i];
    }
  };
  v16f acc[TS][TS];
#pragma unroll
  for (int i = 0; i < TS; ++i)
#pragma unroll
    for (int j = 0; j < TS; ++j) acc[i][j] = (v16f)(0.f);
  const int wm = (wv & 1) * 32 * TS, wn = (wv >> 1) * 32 * TS;
  load(0);
  put(buf[0]);
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    const int8_t* const b = buf[s & 1];
    if (s + 1 < steps) load(s + 1);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const int slot = ((ks * 2 + (lane >> 5)) ^ ((lane >> 1) & 7)) * 16;
      v4i fa[TS], fw[TS];
#pragma unroll
      for (int j = 0; j < TS; ++j) {
        fa[j] = *(const v4i*)(b + (wm + 32 * j + (lane & 31)) * kBK + slot);
        fw[j] = *(const v4i*)(b + (kSide + wn + 32 * j + (lane & 31)) * kBK + slot);
      }
#pragma unroll
      for (int i = 0; i < TS; ++i)
#pragma unroll
        for (int j = 0; j < TS; ++j) acc[i][j] = Op::mma32(fw[i], fa[j], acc[i][j]);
    }
    if (s + 1 < steps) put(buf[(s + 1) & 1]);
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < TS; ++j) {
    const int m = m0 + wm + 32 * j + (lane & 31);
#pragma unroll
    for (int i = 0; i < TS; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + wn + 32 * i + 8 * q + 4 * (lane >> 5);
        float y[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        if (m < g.M && n < g.N) finish4<OT>(g, m, n, y);
      }
  }
}

// Few rows: 16 columns of 16 MT rows a workgroup, whose eight waves split the sum; each
// takes every 8th 64 bytes of the rows straight into registers, four at a time.
template <int DT, int OT, int MT>
__global__ __launch_bounds__(512) void k_matmul_any_rows(MatmulArgs g, int blocks_m) {
  typedef OpFloat<DT> Op;
  typedef typename Store<DT>::T T;
  constexpr int NW = 8, kPiece = 64 / sizeof(T), D = 4;
  __shared__ v4f part[NW][MT][kWave];
  const int lane = lane_id(), wv = wave_id();
  const int n0 = (int)blockIdx.x / blocks_m * 16, m0 = (int)blockIdx.x % blocks_m * 16 * MT;
  const int K = (int)g.K;
  const T* const rw = (const T*)g.w + (int64_t)min(n0 + (lane & 15), (int)g.N - 1) * K;
  const T* ra[MT];
  v4f acc[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    ra[j] = (const T*)g.a + (int64_t)min(m0 + 16 * j + (lane & 15), (int)g.M - 1) * g.lda;
    acc[j] = (v4f)(0.f);
  }
  for (int p = wv * kPiece; p < K; p += NW * kPiece * D) {
    v4i vw[D], va[D][MT];
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int k = p + d * NW * kPiece + (lane >> 4) * (16 / (int)sizeof(T));
      vw[d] = load_any<DT>(rw, k, K);
#pragma unroll
      for (int j = 0; j < MT; ++j) va[d][j] = load_any<DT>(ra[j], k, K);
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[j] = Op::mma16(vw[d], va[d][j], acc[j]);
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) part[wv][j][lane] = acc[j];
  __syncthreads();
  if (wv >= MT) return;
  v4f sum = part[0][wv][lane];
#pragma unroll
  for (int v = 1; v < NW; ++v) sum += part[v][wv][lane];
  const int m = m0 + 16 * wv + (lane & 15), n = n0 + (lane >> 4) * 4;
  float y[4] = {sum[0], sum[1], sum[2], sum[3]};
  if (m < g.M && n < g.N) finish4<OT>(g, m, n, y);
}

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------
template <int DT, int OT, int MT, int NT, int NW, int D>
hipError_t launch_rows(const MatmulArgs& g, hipStream_t st) {
  const int64_t bn = (g.N + 16 * NT - 1) / (16 * NT), bm = (g.M + 16 * MT - 1) / (16 * MT);
  hipLaunchKernelGGL((k_matmul_rows<DT, OT, MT, NT, NW, D>), dim3((unsigned)(bn * bm)), dim3(64 * NW), 0, st, g, (int)bm);
  return hipGetLastError();
}

template <int DT, int OT, int NW, int S>
hipError_t launch_tile(const MatmulArgs& g, int64_t ncu, hipStream_t st) {
  constexpr int kSide = Tile<NW>::kSide;
  const int tm = (int)((g.M + kSide - 1) / kSide), tn = (int)((g.N + kSide - 1) / kSide);
  const dim3 grid((unsigned)min((int64_t)tm * tn, ncu * kTileWgs<NW, S>)), block(64 * NW);
  if (g.K * sizeof(typename Store<DT>::T) % (S * kBK) == 0)
    hipLaunchKernelGGL((k_matmul_tile<DT, OT, false, NW, S>), grid, block, 0, st, g, tm, tn);
  else
    hipLaunchKernelGGL((k_matmul_tile<DT, OT, true, NW, S>), grid, block, 0, st, g, tm, tn);
  return hipGetLastError();
}

template <int DT, int OT, int TS>
hipError_t launch_any(const MatmulArgs& g, hipStream_t st) {
  const int64_t bm = (g.M + 64 * TS - 1) / (64 * TS), bn = (g.N + 64 * TS - 1) / (64 * TS);
  hipLaunchKernelGGL((k_matmul_any<DT, OT, TS>), dim3((unsigned)(bm * bn)), dim3(256), 0, st, g, (int)bm);
  return hipGetLastError();
}

template <int DT, int OT, int MT>
hipError_t launch_any_rows(const MatmulArgs& g, hipStream_t st) {
  const int64_t bm = (g.M + 16 * MT - 1) / (16 * MT), bn = (g.N + 15) / 16;
  hipLaunchKernelGGL((k_matmul_any_rows<DT, OT, MT>), dim3((unsigned)(bm * bn)), dim3(512), 0, st, g, (int)bm);
  return hipGetLastError();
}

// Elements of an aligned copy's rows.
int64_t packed_cols(int64_t K) { return K % 8 == 0 ? K : (K + 63) / 64 * 64; }

template <int DT, int OT>
hipError_t launch(MatmulArgs g, void* ws, hipStream_t st) {
  const int64_t ncu = cu_count() > 0 ? cu_count() : 256;
  constexpr int64_t E = sizeof(typename Store<DT>::T);
  if (!matmul_aligned(DT, g)) {
    // (us with a copy and without, bf16: 4 x 2561 x 5121 17 and 25, 32 rows 20 and 48, 64
    // rows 21 and 57; 4 x 4099 x 2579 16 and 17, 1065 rows 51 and 69; 4 x 1001 x 1003 6.3
    // and 6.0, 64 rows 6.7 and 12.)
    bool packed = false;
    if constexpr (DT != DT_F32) {
      packed = ws && g.M >= kMatmulPackRows;
      if (packed) {
        // w's rows are aligned where K allows it
        const int64_t Kp = packed_cols(g.K);
        PackRows a{g.a, g.lda, g.M, ws}, w{g.w, g.K, Kp == g.K ? 0 : g.N, (char*)ws + g.M * Kp * E};
        const int64_t wgs = (a.rows + w.rows + 3) / 4;
        hipLaunchKernelGGL((k_matmul_pack<DT>), dim3((unsigned)min(wgs, (int64_t)1 << 20)), dim3(256), 0, st, a, w, (int)g.K, (int)Kp);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        g.a = ws;
        if (w.rows) g.w = w.to;
        g.lda = g.K = Kp;
      }
    }
    if (!packed) {
      // Rows in 16s and 32s while they and the blocks of 64 are few (us at 16s, 32s and
      // blocks: 16 x 2561 x 5121 bf16 33, 37 and 48, 32 rows 63, 48 and 58, 48 rows 63, 94 and
      // 57; 32 x 10577 x 2561 bf16 94, 72 and 33; fp32, where LDS and copies weigh less: 32 x
      // 2561 x 2561 23, 19 and 61, 96 rows 45, 36 and 61; 48 x 10577 x 2561 86, 102 and 62).
      const int64_t blocks = (g.M + 63) / 64 * ((g.N + 63) / 64);
      if (g.M <= 16) return launch_any_rows<DT, OT, 1>(g, st);
      if (DT == DT_F32 ? blocks < ncu / 2 : g.M <= 32 && blocks < ncu / 4) return launch_any_rows<DT, OT, 2>(g, st);
      // Blocks of 128 where each CU has one, of 16-bit rows (us with 128 and 64: 1065 x
      // 4099 x 2579 bf16 70, 93; 300 x 4099 x 2579 55, 35; 1065 x 4099 x 2579 fp32, which
      // the matrix instructions bound, 340, 231).
      if constexpr (DT != DT_F32)
        if ((g.M + 127) / 128 * ((g.N + 127) / 128) >= ncu) return launch_any<DT, OT, 2>(g, st);
      return launch_any<DT, OT, 1>(g, st);
    }
  }
  // fp32: an 8th of the rate (us with that factor and without: 1024 x 4096 x 1024 66 and 73,
  // 333 x 8512 x 2048 122 and 132, 2048 x 2048 x 2048 127 and 136)
  switch (pick_matmul_kind(g.M, g.N, g.K * E, ncu, DT == DT_F32 ? 8.f : 1.f)) {
    case 0: return launch_rows<DT, OT, 1, 1, 8, 2>(g, st);
    case 1: return launch_rows<DT, OT, 1, 2, 4, 3>(g, st);
    case 2: return launch_rows<DT, OT, 2, 2, 4, 2>(g, st);
    case 3: return launch_rows<DT, OT, 4, 4, 4, 2>(g, st);
    case 4: return launch_tile<DT, OT, 4, 4>(g, ncu, st);
    case 5: return launch_tile<DT, OT, 4, 2>(g, ncu, st);
    default: return launch_tile<DT, OT, 8, 2>(g, ncu, st);
  }
}

}  // namespace

size_t matmul_workspace_bytes(int64_t M, int64_t N, int64_t K, int dtype) {
  if (dtype == DT_F32 || M < kMatmulPackRows) return 0;
  const int64_t Kp = packed_cols(K);
  return (size_t)(M + (Kp == K ? 0 : N)) * Kp * 2;
}

hipError_t launch_matmul(int dtype, int out_dtype, const MatmulArgs& g, void* ws, hipStream_t st) {
  const bool keep32 = out_dtype == DT_F32;
  switch (dtype) {
    case DT_F32: return launch<DT_F32, DT_F32>(g, ws, st);
    case DT_F16: return keep32 ? launch<DT_F16, DT_F32>(g, ws, st) : launch<DT_F16, DT_F16>(g, ws, st);
    case DT_BF16: return keep32 ? launch<DT_BF16, DT_F32>(g, ws, st) : launch<DT_BF16, DT_BF16>(g, ws, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ssd
