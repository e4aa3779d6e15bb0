// Matrix product in 8-bit integers with a step for each row of both operands:
//   out[m,n] = a_scale[m] w_scale[n] sum_k a[m,k] w[n,k] + bias[n]
// The sums are exact int32 MFMA sums; one fp32 epilogue per element, rounded once.
//
// Few rows are bound by the read of w, and there by latency: 8 x 2560 x 5120
// (13 MB) 4.4 us, of which 2 are a launch; 333 x 8512 x 2048 12 us. Large
// products are bound by power: 16384 x 10576 x 2560 449 to 475 us by card (2.0 Pop/s;
// with all codes zero 1.45 times as fast; of a run that begins at rest the first
// passes take 440 us, the fifth to the fifteenth 500 to 546, and from about the
// thirtieth on all 465), 16384 x 10752 x 2560 392 us,
// 8192 x 8192 x 8192 423 us (2.6 Pop/s). A step of 128 bytes of a 256 x 256 tile
// is 2048 cycles of each SIMD's matrix unit and as many of the LDS (192 KB read,
// 64 KB written); four waves of 128 x 128 blocks instead of eight of 64 x 128
// read a third less, but one wave a SIMD covers nothing: 8192 x 8192 x 8192 479 us.
#include "ssd_launch.hpp"
#include "ssd_matmul.hpp"
#include "ssd_matmul_kind.hpp"

namespace ssd {
namespace {

struct OpI8 {
  typedef v16i Acc32;
  typedef v4i Acc16;
  static constexpr int kInstructions = 1;  // of a product
  static __device__ __forceinline__ Acc32 mma32(v4i a, v4i b, Acc32 c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ Acc16 mma16(v4i a, v4i b, Acc16 c) { return mma_i8(a, b, c); }
};

// 128 consecutive bytes of outputs of 32 rows at a time: the lane's sums are
// scaled and rounded, pass through the wave's own staging rows (16-byte chunk c
// of row r at slot c ^ (r / 2 % 8)), and leave as whole pieces of rows.
template <int DT, bool BIAS, int NW>
__device__ __forceinline__ void tile_store(const MatmulI8Args& g, int m0, int n0, int wm, int wn, int8_t* st,
                                           const v16i (&acc)[Tile<NW>::TI][2]) {
  typedef typename Store<DT>::T T;
  typedef const __attribute__((address_space(4))) float* scalar_ptr;
  typedef __attribute__((address_space(1))) v4u_any* global_out;
  constexpr int U = DT == DT_F32 ? 1 : 2;  // 32-column blocks of a piece
  constexpr int E = 16 / sizeof(T);        // outputs of a 16-byte chunk
  const int lane = lane_id(), hi = lane >> 5;
  // Pieces that are whole 128-byte lines go past the caches (16384 x 10752 x 2560
  // fp16 431 -> 392 us); others would go to memory in parts (8192 x 3352 x 1024
  // fp32 46 -> 73 us; halves of lines, 96 to 103 % of the time, are left too).
  const bool lines = ((uint64_t)g.out | g.N * sizeof(T)) % 128 == 0;
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
  // the pieces of a row leave one after the other, so that they meet in the cache
  // where they share lines
#pragma unroll
  for (int j = 0; j < 2; ++j) {
#pragma unroll
    for (int u = 0; u < Tile<NW>::TI / U; ++u) {
      const int nu = n0 + wn + 32 * U * u;
      float ws[U][4][4], bias[U][4][4];
      columns(g.w_scale + nu, ws);
      if constexpr (BIAS) columns(g.bias + nu, bias);
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
        const int64_t at = (int64_t)(m0 + wm + 32 * j + 8 * r) * g.N + nu;
        const int8_t* const rows = uniform_ptr((const int8_t*)g.out + at * sizeof(T));
        const global_out o = (global_out)(uint64_t)(rows + lane_at);
        // rows that are not 16-byte aligned take the same stores
        if (lines) {
          asm volatile("; lines");  // without these the compiler makes one store of the two
          __builtin_nontemporal_store(v, o);
          asm volatile("; lines");
        } else {
          *o = v;
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
  }
}

template <int DT, bool TAIL, bool BIAS, int NW, int S>
__global__ __launch_bounds__(64 * NW, (kTileWgs<NW, S> * NW / 4)) void k_matmul_i8_tile(MatmulI8Args g,
                                                                                     int tiles_m, int tiles_n) {
  tile_walk<OpI8, TAIL, true, NW, S>(
      g, (int)g.K, g.K, tiles_m, tiles_n,
      [&](int m0, int n0, int, int, int wm, int wn, int8_t* stage, const v16i (&acc)[Tile<NW>::TI][2]) __attribute__((always_inline)) {
        tile_store<DT, BIAS, NW>(g, m0, n0, wm, wn, stage, acc);
      });
}

template <int MT, int NT, int NW, int D>
__global__ __launch_bounds__(64 * NW) void k_matmul_i8_rows(MatmulI8Args g, int dtype, int blocks_m) {
  few_rows<OpI8, MT, NT, NW, D>(g, (int)g.K, g.K, blocks_m, [&](int m, int n, v4i sum) __attribute__((always_inline)) {
    const float as = g.a_scale[m];
    float ws[4], bias[4], y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = min(n + e, (int)g.N - 1);
      ws[e] = g.w_scale[c];
      bias[e] = g.bias ? g.bias[c] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = fmaf((float)sum[e], as * ws[e], bias[e]);
    const int64_t o = (int64_t)m * g.N + n;
    const int left = (int)g.N - n;
    switch (dtype) {
      case DT_F32: store4<DT_F32>(g.out, o, y, left); break;
      case DT_F16: store4<DT_F16>(g.out, o, y, left); break;
      default: store4<DT_BF16>(g.out, o, y, left); break;
    }
  });
}

template <int MT, int NT, int NW, int D>
hipError_t launch_rows(const MatmulI8Args& g, int dtype, hipStream_t st) {
  const int64_t bn = (g.N + 16 * NT - 1) / (16 * NT), bm = (g.M + 16 * MT - 1) / (16 * MT);
  hipLaunchKernelGGL((k_matmul_i8_rows<MT, NT, NW, D>), dim3((unsigned)(bn * bm)), dim3(64 * NW), 0, st, g, dtype, (int)bm);
  return hipGetLastError();
}

template <int DT, int NW, int S>
hipError_t launch_tile(const MatmulI8Args& g, int64_t ncu, hipStream_t st) {
  constexpr int kSide = Tile<NW>::kSide;
  const int tm = (int)((g.M + kSide - 1) / kSide), tn = (int)((g.N + kSide - 1) / kSide);
  const dim3 grid((unsigned)min((int64_t)tm * tn, ncu * kTileWgs<NW, S>)), block(64 * NW);
#define TILE_(TAIL_, BIAS_) hipLaunchKernelGGL((k_matmul_i8_tile<DT, TAIL_, BIAS_, NW, S>), grid, block, 0, st, g, tm, tn)
  if (g.K % (S * kBK) == 0) {
    if (g.bias) TILE_(false, true);
    else TILE_(false, false);
  } else {
    if (g.bias) TILE_(true, true);
    else TILE_(true, false);
  }
#undef TILE_
  return hipGetLastError();
}

template <int DT>
hipError_t launch(const MatmulI8Args& g, hipStream_t st) {
  const int64_t ncu = cu_count() > 0 ? cu_count() : 256;
  switch (pick_matmul_kind(g.M, g.N, g.K, ncu)) {
    case 0: return launch_rows<1, 1, 8, 2>(g, DT, st);
    case 1: return launch_rows<1, 2, 4, 3>(g, DT, st);
    case 2: return launch_rows<2, 2, 4, 2>(g, DT, st);
    case 3: return launch_rows<4, 4, 4, 2>(g, DT, st);
    case 4: return launch_tile<DT, 4, 4>(g, ncu, st);
    case 5: return launch_tile<DT, 4, 2>(g, ncu, st);
    default: return launch_tile<DT, 8, 2>(g, ncu, st);
  }
}

}  // namespace

hipError_t launch_matmul_i8(int out_dtype, const MatmulI8Args& g, hipStream_t st) {
  switch (out_dtype) {
    case DT_F32: return launch<DT_F32>(g, st);
    case DT_F16: return launch<DT_F16>(g, st);
    case DT_BF16: return launch<DT_BF16>(g, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ssd
