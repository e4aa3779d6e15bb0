// The gated delta rule in chunks of 64 positions. With g_i the sum of dt A over a
// chunk up to position i, S [P, N] the state before the chunk and u_i the change that
// position i writes,
//   L_ij = b_i e^{g_i - g_j} k_i.k_j  (j < i),   T = (1 + L)^-1,
//   U = T diag(b) (V - diag(e^g) K S^T),
//   Y = scale (diag(e^g) Q S^T + (Q K^T . e^{g_i - g_j}, j <= i) U),
//   S' = e^{g_63} S + (diag(e^{g_63 - g}) U)^T K.
//
// Keys that are not taken to length 1 may differ in length by any factor, and b, as 1 / |k|^2,
// T and U by its square, which is more than products of 16-bit parts hold. There, with p_i
// the power of two of |k_i|, what the products are formed of is
//   p_i T_ij b_j p_j,   (V_j - e^{g_j} k_j S^T) / p_j   and   p_i U_i
// (p_i L_ij / p_j has entries of b |k|^2's size, and what position i adds to the state is
// p_i U_i times a key of length about 1), and queries' powers of two stay outside Y's weights.
//
// Three launches. For every chunk at once, k_delta_keys forms a group's keys and queries
// as matrix operands, and k_delta_prepare a head's T diag(b) and the weights of U in Y,
// none of which needs the state. k_delta_scan then goes through a head's chunks in order,
// with the state in registers: a wave owns 16 rows of S, which no other needs.
//
// The scan's products follow one another without a step through LDS: the 16 x 16
// result tiles hold, in lane i, rows 4 (i / 16) .. + 3 of column i % 16, and two of them
// are an operand of 32 rows whose order of rows the other operand takes on too (columns
// here are rows of S: S^T is [N, P]). An operand's lane i thus has, of step s, the 8
// positions 32 s + 4 (i / 16) + (0..3) and 16 more than those ("fragments" below).
//
// Precision. The state is kept and returned in fp32, so that no operand of the
// products that lead to it may be rounded to 16 bits. Each is taken as a sum of two
// fp16 numbers (22 significant bits), after a power of two has brought the largest of
// its column (or row, or tile row) to 2^8: what is below 2^-33 of that is lost. Keys and
// queries of 16-bit types are exact in one fp16 number in that way, fp32 ones in two.
// Products of two lower parts (2^-22 of the rest) are left out. The same goes for Y, which
// is rounded once at the end, but for its weights in bf16: see Parts.
//
// Times (us: keys, prepare, scan), heads of P x N:
//   1 x 2048 positions, 64 heads of 64 x 128, bf16          6, 18, 110
//   8 x 2048, 80 of 64 x 128, one group each, fp16          9, 132 to 144, 316 to 359
//   4 x 4096, 32 of 128 x 128, 16 groups each, bf16         70, 62, 270
// The scan is bound by its chain: 1010 to 1080 instructions a chunk and wave (580 to 650 of
// the vector unit, 132 products, 116 LDS reads) that follow one another, in 3.4 us where a
// wave has its SIMD to itself, of which 45 % issue nothing; two waves a SIMD issue 72 % of
// the cycles. Memory serves 2 to 3 TB/s meanwhile. prepare writes 22 to 25 KB a chunk and
// head at 3 to 4 TB/s, and waits at its four barriers; keys moves what it moves at the rate of
// a copy once groups are many (6 TB/s of read and written bytes in the last).
// Preparing a chunk within the scan's launch was no faster in total.
#include <cstddef>
#include <type_traits>

#include "ssd_delta.hpp"
#include "ssd_delta_scale.hpp"

namespace ssd {
namespace {

constexpr int kC = kDeltaChunk;

// What the operands of one type are made of.
template <int DT>
struct Parts {
  static constexpr int kKeys = DT == DT_F32 ? 2 : 1;     // fp16 numbers of a key's or query's element
  static constexpr int kWeights = DT == DT_F32 ? 2 : 1;  // of Y's weights of U in LDS: one rounds to 2^-12 of a term
  // Bytes of each weight's lower part that follow in memory: two for fp16's Y (terms to
  // 2^-23), one for bf16's, whose step is 8 times as large (to 2^-16: a 128th of its half step).
  // (Differences from the rounded exact outputs: bf16 1.0e-3 without and 2e-4 with; fp16 5e-5
  // to 7e-5 with one byte, under 4.3e-5 with two, which take 3 % more time.)
  static constexpr int kLowBytes = DT == DT_F16 ? 2 : DT == DT_BF16 ? 1 : 0;
};

// ---------------------------------------------------------------------------
// workspace and LDS
// ---------------------------------------------------------------------------
constexpr int kFrag = 1024;  // bytes: 16 for each lane

// Of each (batch, group, chunk): fragments of K and Q (4 tiles of 16 positions, KS
// steps of 32 channels) and of K^T (NT tiles of 16 channels, 2 steps of 32 positions),
// each row's factor, what undoes its scaling and makes it of length 1 (K's 64, Q's), the
// scalings' exponents (a byte for K and one for Q, of each row), and the fp32 tiles of the
// lower triangles of K K^T (rows i, columns j of tile (i, j)) and of Q K^T, transposed.
template <int DT, int N>
struct KeyPlan {
  static constexpr int KS = (N + 31) / 32, NT = N / 16, KP = Parts<DT>::kKeys;
  static constexpr int kK = 0, kQ = 4 * KS * KP, kT = 8 * KS * KP, kTurned = 2 * NT * KP;
  static constexpr int kFac = kT + kTurned, kKK = kFac + 1, kKQ = kKK + 10, kFrags = kKQ + 10;
  static constexpr int kExponents = kFac * kFrag + 2 * kC * sizeof(float);  // a byte's place
  static constexpr size_t kBytes = (size_t)kFrags * kFrag;
};
// Tile (i, j) of a lower triangle of 4 x 4, in rows.
__device__ __forceinline__ constexpr int lower_tile_at(int i, int j) { return i * (i + 1) / 2 + j; }
// Factors of a chunk of a head: for each position of K S^T in R (fac_k), of Q S^T in Y
// (fac_q) and of U in S' (fac_u, with the factor that undoes T's scaling); what undoes the
// scaling of each tile row of T and of Y's weights; the state's decay over the chunk, and
// whether a key is zeros: its fac_k is -1.
struct Factors {
  float fac_k[kC], fac_q[kC], fac_u[kC], inv_t[4], inv_a[4];  // read four at a time
  float decay, zero_keys;
};
static_assert(offsetof(Factors, inv_t) % 16 == 0 && offsetof(Factors, inv_a) % 16 == 0, "16-byte reads");
// Of each (batch, head, chunk): fragments of T diag(b) (6
// that are not zero, two parts), of Y's weights (6), the factors, and the weights' lower
// parts, 8 kLowBytes bytes for each lane of a fragment.
template <int DT>
struct HeadPlan {
  static constexpr int kT = 0, kA = 12, kFac = 12 + 6 * Parts<DT>::kWeights, kLow = kFac + 1;
  static constexpr int kLowFrag = kFrag / 2 * Parts<DT>::kLowBytes;
  static constexpr int kFrags = kLow + 6 * kLowFrag / kFrag;
  static constexpr size_t kBytes = (size_t)kFrags * kFrag;
};
static_assert(sizeof(Factors) <= kFrag, "a fragment's room");

// The fragment of tile row i and step s of a lower triangle of 4 x 4 tiles.
__device__ __forceinline__ constexpr int lower_frag(int i, int s) { return i < 2 ? i : 2 * i - 2 + s; }

// What a head's chunk is made of besides keys and queries, for each position. g: sums
// of dt A log2(e), twice fp32's bits, as their differences count; fk, fq: what K's and Q's
// factors are but for the powers of two p; beta: beta p^2; cols: the decay from the position
// to the end of its 16, times fk; first[j]: the decay to the position from the end of the
// 16 positions j; rows[j]: the same times beta, p and K's factor, rows[3] without it.
struct Gates {
  float g[kC], g_low[kC], beta[kC], cols[kC], rows[4][kC], first[3][kC], fk[kC], fq[kC];
  Factors f;
};
// L's four diagonal tiles, and then their inverses, with rows 20 floats apart and tiles
// 4 banks.
constexpr int kDiagRow = 20, kDiag = 16 * kDiagRow + 4;

// ---------------------------------------------------------------------------
// scaling and parts
// ---------------------------------------------------------------------------
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// Eight values, four times a factor each, as fp16 numbers, and what that leaves of them as eight
// more. (The empty asm keeps the compiler from forming the first ones twice, packed and
// one by one.)
__device__ __forceinline__ void split8(const float (&x)[8], float by0, float by4, v8h& hi, v8h& lo) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float by = e < 4 ? by0 : by4;
    uint32_t w = pack2<DT_F16>(x[e] * by, x[e + 1] * by);
    asm("" : "+v"(w));
    const v2h h = __builtin_bit_cast(v2h, w);
    hi[e] = h[0];
    hi[e + 1] = h[1];
    lo[e] = (_Float16)fmaf(x[e], by, -(float)h[0]);
    lo[e + 1] = (_Float16)fmaf(x[e + 1], by, -(float)h[1]);
  }
}
// The same of the scaled state's values, brought down to fp16's range: one operation for
// each number, which takes the factor along.
__device__ __forceinline__ void split8_state(const float (&x)[8], v8h& hi, v8h& lo) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    hi[e] = (_Float16)(x[e] * kStateDown);
    lo[e] = (_Float16)fmaf(x[e], kStateDown, -(float)hi[e]);
  }
}
// Rows 4 (lane / 16) .. of two result tiles, as an operand.
__device__ __forceinline__ void split_tiles(v4f a, v4f b, float by_a, float by_b, v8h& hi, v8h& lo) {
  const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  split8(x, by_a, by_b, hi, lo);
}
// The upper bytes of eight fp16 numbers, rounded, and the numbers that they stand for.
__device__ __forceinline__ uint2 upper_bytes(v8h v) {
  const v4u w = __builtin_bit_cast(v4u, v) + 0x00800080u;
  return make_uint2(__builtin_amdgcn_perm(w[1], w[0], 0x07050301), __builtin_amdgcn_perm(w[3], w[2], 0x07050301));
}
__device__ __forceinline__ v8h from_upper_bytes(uint2 b) {
  const v4u w = {__builtin_amdgcn_perm(0, b.x, 0x010c000c), __builtin_amdgcn_perm(0, b.x, 0x030c020c),
                 __builtin_amdgcn_perm(0, b.y, 0x010c000c), __builtin_amdgcn_perm(0, b.y, 0x030c020c)};
  return __builtin_bit_cast(v8h, w);
}
// What a lane holds of a fragment of lower parts: eight of so many bytes.
template <int BYTES>
struct LowPart {
  typedef v8h T;
};
template <>
struct LowPart<1> {
  typedef uint2 T;
};
// 2^x
__device__ __forceinline__ float exp2(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ v4f mma16(v8h a, v8h b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ float max4(float m, v4f v) {
  m = fmaxf(fmaxf(m, fabsf(v[0])), fabsf(v[1]));
  return fmaxf(fmaxf(m, fabsf(v[2])), fabsf(v[3]));
}
// The largest magnitude of N tiles: a chain of maxima for each row of a tile.
template <int N>
__device__ __forceinline__ float tiles_max(const v4f (&t)[N]) {
  v4f m = (v4f)(0.f);
#pragma unroll
  for (int n = 0; n + 1 < N; n += 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = fmaxf(fmaxf(m[e], fabsf(t[n][e])), fabsf(t[n + 1][e]));
  if constexpr (N % 2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], fabsf(t[N - 1][e]));
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
// The largest of a column, of which a lane has m of its 4 rows in each tile.
__device__ __forceinline__ float column_max(float m) {
  const uint32_t b = __float_as_uint(m);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const uint32_t c = __float_as_uint(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
  const auto q = __builtin_amdgcn_permlane32_swap(c, c, false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
  return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true)));
}
// The largest of a wave's values, none of them negative.
__device__ __forceinline__ float wave_most(float v) {
  return column_max(dpp_max<0x140>(dpp_max<0x141>(dpp_max<0x4E>(dpp_max<0xB1>(v)))));
}

// 16 bytes per lane from global memory straight into LDS: lane i's bytes land at l + 16 i.
__device__ __forceinline__ void copy_frag(const char* g, char* l) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) char*)g,
                                   (__attribute__((address_space(3))) void*)l, 16, 0, 0);
}
// Fragments f, f + n, ... of `count`.
template <int COUNT, int WAVES>
__device__ __forceinline__ void copy_frags(const char* g, char* l, int wave) {
  const char* const from = g + lane_id() * 16;
#pragma unroll
  for (int f = 0; f < COUNT; f += WAVES)
    if (COUNT % WAVES == 0 || f + wave < COUNT) copy_frag(from + (f + wave) * kFrag, l + (f + wave) * kFrag);
}
// This wave's memory operations are done but for the newest BEHIND (64: whatever), and
// its LDS operations; behind the barrier all waves' are, and what was read is free.
template <int BEHIND>
__device__ __forceinline__ void meet() {
  constexpr int n = BEHIND < 63 ? BEHIND : 63;
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (n & 15) | ((n >> 4) << 14));  // vmcnt, lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
// keys and queries
// ---------------------------------------------------------------------------
// A tile of K K^T (rows of tile row i, columns j) or of K Q^T (rows j, columns i), from
// fragments of K and Q.
template <int DT, int N>
__device__ __forceinline__ v4f key_tile(const char* frags, bool queries, int i, int j) {
  typedef KeyPlan<DT, N> KP_;
  constexpr int KS = KP_::KS, KP = KP_::KP;
  const char* const left = frags + ((queries ? j : i) * KS + KP_::kK) * kFrag + lane_id() * 16;
  const char* const right = frags + (queries ? i * KS + KP_::kQ : j * KS + KP_::kK) * kFrag + lane_id() * 16;
  constexpr int kLo = 4 * KS * kFrag;
  v4f acc = (v4f)(0.f);
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const v8h a = *(const v8h*)(left + s * kFrag), b = *(const v8h*)(right + s * kFrag);
    acc = mma16(a, b, acc);
    if constexpr (KP == 2) {
      acc = mma16(a, *(const v8h*)(right + s * kFrag + kLo), acc);
      acc = mma16(*(const v8h*)(left + s * kFrag + kLo), b, acc);
    }
  }
  return acc;
}

// A workgroup of four waves takes a chunk of a group, four threads a row, a step's 32
// channels each.
template <int DT, int N>
__global__ __launch_bounds__(256) void k_delta_keys(DeltaArgs a, char* ws, int64_t L, int G, int chunks, int64_t total) {
  typedef KeyPlan<DT, N> KP_;
  constexpr int KS = KP_::KS, NT = KP_::NT, KP = KP_::KP, E = N < 32 ? N : 32;
  __shared__ __attribute__((aligned(16))) char frags[8 * KS * KP * kFrag];  // K's, Q's
  const int tid = threadIdx.x, lane = lane_id(), sub = lane >> 4, col = lane & 15;
  const int row = tid >> 2, s = tid & 3;
  for (int64_t item = blockIdx.x; item < total; item += gridDim.x) {
    const int ck = (int)(item % chunks);
    const int64_t bg = item / chunks, b = bg / G, pos0 = (int64_t)ck * kC;
    const int g = (int)(bg % G);
    char* const out = ws + item * KP_::kBytes;
    const bool live = s < KS && pos0 + row < L;  // rows behind the end are zeros
    float x[2][32];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
      for (int e = 0; e < 32; ++e) x[which][e] = 0.f;
      if (live) {
        const int64_t at = ((b * L + pos0 + row) * G + g) * N + s * 32;
#pragma unroll
        for (int e = 0; e < E; e += 8) {
          float t[8];
          ld8_f<DT>(which ? a.C : a.B, at + e, t);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[which][e + i] = t[i];
        }
      }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float(&v)[32] = x[which];
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < 32; ++e) m = fmaxf(m, fabsf(v[e]));
      m = dpp_max<0x4E>(dpp_max<0xB1>(m));
      const Scale sc(m);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        v[e] *= sc.by;
        ss = fmaf(v[e], v[e], ss);
      }
      ss = group_sum<4>(ss);
      if (s == 0) {
        float f = sc.inv;
        const bool zeros = ss == 0.f;
        if (a.unit) {
          const float eps = a.eps * sc.by * sc.by;
          ss += eps;
          f = eps > 0x1p126f ? sc.inv * rsqrtf(a.eps) : rsqrtf(ss);  // next to a far larger eps the row counts for nothing
        }
        if (zeros) f = 0.f;  // and a key of zeros is known by its factor
        ((float*)(out + KP_::kFac * kFrag))[which * kC + row] = which ? f * a.scale : f;
        ((int8_t*)(out + KP_::kExponents))[2 * row + which] = (int8_t)sc.exponent();
      }
      if (s < KS) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float t[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            t[e] = v[4 * q + e];
            t[4 + e] = v[16 + 4 * q + e];
          }
          v8h hi, lo;
          split8(t, 1.f, 1.f, hi, lo);
          const int at = ((which ? KP_::kQ : KP_::kK) + (row >> 4) * KS + s) * kFrag + (q * 16 + (row & 15)) * 16;
          *(v8h*)(out + at) = hi;
          *(v8h*)(frags + at) = hi;
          if constexpr (KP == 2) {
            constexpr int kLo = 4 * KS * kFrag;
            *(v8h*)(out + at + kLo) = lo;
            *(v8h*)(frags + at + kLo) = lo;
          }
        }
      }
    }
    __syncthreads();
    for (int f = wave_id(); f < 2 * NT * KP; f += 4) {  // K^T: channel 16 nt + col, positions of step t
      const int part = f / (2 * NT), nt = f / 2 % NT, t = f & 1, n = 16 * nt + col;
      const char* const from = frags + part * 4 * KS * kFrag + (n >> 5) * kFrag + ((n & 15) >> 2) * 256 +
                               ((n & 3) + ((n >> 4) & 1) * 4) * 2;
      v8h v;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int p = 4 * sub + (e & 3);  // of tile 2 t + e / 4
        v[e] = *(const _Float16*)(from + (2 * t + (e >> 2)) * KS * kFrag + p * 16);
      }
      *(v8h*)(out + (KP_::kT + f) * kFrag + lane * 16) = v;
    }
    for (int t = wave_id(); t < 20; t += 4) {
      const int u = t % 10, i = u < 1 ? 0 : u < 3 ? 1 : u < 6 ? 2 : 3, j = u - i * (i + 1) / 2;
      *(v4f*)(out + (KP_::kKK + t) * kFrag + lane * 16) = key_tile<DT, N>(frags, t >= 10, i, j);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// what a chunk of a head needs besides the state
// ---------------------------------------------------------------------------
// A position's step size, write strength and factors, one to a lane; behind the end
// nothing decays and nothing is written.
struct GateInputs {
  float dt, beta, fk, fq;
  template <int DT>
  __device__ __forceinline__ void load(const DeltaArgs& a, const float* fac, int64_t row0, int64_t pos0, int64_t L, int H, int h) {
    const bool live = pos0 + lane_id() < L;
    const int64_t row = row0 + pos0 + lane_id();
    dt = live ? ld_f<DT>(a.dt, row * H + h) : 0.f;
    beta = live ? delta_beta<DT>(a, row, h) : 0.f;
    fk = fac[lane_id()];
    fq = fac[kC + lane_id()];
  }
};
// A lane's value of a double, the same in all lanes.
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = __builtin_amdgcn_readlane((int)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// v plus the value SHIFT lanes before in the row of 16.
template <int SHIFT>
__device__ __forceinline__ double row_add(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, 0x110 + SHIFT, 0xf, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), 0x110 + SHIFT, 0xf, 0xf, true);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ void form_gates(Gates& w, const GateInputs& in, float A, bool unit) {
  const int lane = lane_id(), sub = lane >> 4;
  double log_a = (double)in.dt * ((double)A * 1.4426950408889634);
  // 2^log_a is 0 either way, and 64 of them leave the sums 37 bits behind the point: what
  // decays after such a position keeps its effect
  log_a = log_a < -1024.0 ? -1024.0 : log_a;
  double gs = row_add<8>(row_add<4>(row_add<2>(row_add<1>(log_a))));
  double end[4];  // of each 16 positions
  end[0] = lane_value(gs, 15);
  end[1] = end[0] + lane_value(gs, 31);
  end[2] = end[1] + lane_value(gs, 47);
  end[3] = end[2] + lane_value(gs, 63);
  gs += sub == 0 ? 0.0 : sub == 1 ? end[0] : sub == 2 ? end[1] : end[2];
  const double own = sub == 0 ? end[0] : sub == 1 ? end[1] : sub == 2 ? end[2] : end[3];
  // what a key of zeros would write is nothing, whatever stands behind a sequence's end in beta
  const float beta = in.fk != 0.f ? in.beta : 0.f;
  // lengths that are not 1 are powers of two (zeros have none)
  const float p = unit ? 1.f : in.fk, fk = unit ? in.fk : in.fk != 0.f ? 1.f : 0.f;
  const float eg = exp2((float)gs), row = beta * p * in.fk;
  w.g[lane] = (float)gs;
  w.g_low[lane] = (float)(gs - (double)(float)gs);
  w.beta[lane] = beta * p * p;
  w.fk[lane] = fk;
  w.fq[lane] = unit ? in.fq : 1.f;
  w.cols[lane] = exp2((float)(own - gs)) * fk;
  w.rows[3][lane] = row;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const float first = exp2((float)(gs - end[q]));
    w.first[q][lane] = first;
    w.rows[q][lane] = row * first;
  }
  w.f.fac_k[lane] = in.fk != 0.f ? eg * in.fk : -1.f;
  w.f.fac_q[lane] = eg * in.fq;
  w.f.fac_u[lane] = exp2((float)(end[3] - gs)) * fk;
  const bool zero_keys = __ballot(in.fk == 0.f) != 0;
  if (lane == 0) {
    w.f.decay = exp2((float)end[3]);
    w.f.zero_keys = zero_keys ? 1.f : 0.f;
  }
}

// L's tile (i, j) below the diagonal, from K K^T's.
__device__ __forceinline__ v4f lower_tile(const Gates& w, v4f kk, int i, int j) {
  const int sub = lane_id() >> 4, col = lane_id() & 15;
  return *(const v4f*)&w.rows[j][16 * i + 4 * sub] * w.cols[16 * j + col] * kk;
}
// L's tile (i, i), into LDS.
__device__ __forceinline__ void diagonal_tile(const Gates& w, v4f kk, int i, float* diag) {
  const int sub = lane_id() >> 4, col = lane_id() & 15;
  const float gj = w.g[16 * i + col], gl = w.g_low[16 * i + col], c = w.fk[16 * i + col];
  const v4f gi = *(const v4f*)&w.g[16 * i + 4 * sub], gil = *(const v4f*)&w.g_low[16 * i + 4 * sub];
  const v4f r = *(const v4f*)&w.rows[3][16 * i + 4 * sub];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float gamma = exp2((gi[e] - gj) + (gil[e] - gl));
    diag[i * kDiag + (4 * sub + e) * kDiagRow + col] = col < 4 * sub + e ? r[e] * c * gamma * kk[e] : 0.f;
  }
}
// The inverses of the four diagonal blocks of 1 + L, in place: 16 lanes a block, each a
// column. Each value that is final is taken out of all those below it at once, so that
// 16 steps follow one another and not 120.
__device__ __forceinline__ void invert_diagonal(float* diag) {
  const int sub = lane_id() >> 4, col = lane_id() & 15;
  float* const d = diag + sub * kDiag;
  v4f l[16][4];
#pragma unroll
  for (int i = 1; i < 16; ++i)
#pragma unroll
    for (int q = 0; q <= (i - 1) / 4; ++q) l[i][q] = *(const v4f*)(d + i * kDiagRow + 4 * q);
  float t[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) t[i] = i == col ? 1.f : 0.f;
#pragma unroll
  for (int k = 0; k < 15; ++k)
#pragma unroll
    for (int i = k + 1; i < 16; ++i) t[i] = fmaf(-l[i][k >> 2][k & 3], t[k], t[i]);
  wave_sync();
#pragma unroll
  for (int i = 0; i < 16; ++i) d[i * kDiagRow + col] = t[i];
}

// Tiles of a row of a lower triangle, transposed (rows are positions j, columns i), as
// fragments for the products with R or U; LOW: lower parts' bytes that go to low. Returns
// what undoes their scaling.
template <int I, int PARTS, int LOW = 0>
__device__ __forceinline__ float write_row(const v4f (&x)[I + 1], char* out, char* low) {
  const Scale sc(wave_most(tiles_max(x)));
#pragma unroll
  for (int s = 0; s <= I / 2; ++s) {
    v8h hi, lo;
    split_tiles(x[2 * s], 2 * s + 1 <= I ? x[2 * s + 1 <= I ? 2 * s + 1 : 0] : (v4f)(0.f), sc.by, sc.by, hi, lo);
    *(v8h*)(out + lower_frag(I, s) * kFrag + lane_id() * 16) = hi;
    if constexpr (PARTS == 2) *(v8h*)(out + (6 + lower_frag(I, s)) * kFrag + lane_id() * 16) = lo;
    if constexpr (LOW == 2) *(v8h*)(low + lower_frag(I, s) * kFrag + lane_id() * 16) = lo;
    if constexpr (LOW == 1) *(uint2*)(low + lower_frag(I, s) * (kFrag / 2) + lane_id() * 8) = upper_bytes(lo);
  }
  return sc.inv;
}
// Tile row I of T diag(b), from T_ij = -(sum_{j<k<=i} T_ik L_kj) T_jj. lower(k, j): L's
// tiles; diag: the inverted blocks. The tiles are held transposed. Each one that is final
// goes into the sums of all those before it at once.
template <int I, class Lower>
__device__ __forceinline__ void form_t_row(const Gates& w, const float* diag, Lower lower, char* out, Factors& f) {
  const int sub = lane_id() >> 4, col = lane_id() & 15;
  v4f x[I + 1], l[I + 1][I + 1], d[I + 1], beta[I + 1];
  x[I] = *(const v4f*)(diag + I * kDiag + col * kDiagRow + 4 * sub);
#pragma unroll
  for (int k = I; k > 0; --k)
#pragma unroll
    for (int j = k - 1; j >= 0; --j) l[k][j] = lower(k, j);
#pragma unroll
  for (int j = I - 1; j >= 0; --j)
#pragma unroll
    for (int e = 0; e < 4; ++e) d[j][e] = diag[j * kDiag + (4 * sub + e) * kDiagRow + col];
#pragma unroll
  for (int j = 0; j <= I; ++j) beta[j] = *(const v4f*)&w.beta[16 * j + 4 * sub];
#pragma unroll
  for (int j = 0; j < I; ++j) x[j] = (v4f)(0.f);
#pragma unroll
  for (int k = I; k > 0; --k) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = k - 1; j >= 0; --j) x[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(l[k][j][e], x[k][e], x[j], 0, 0, 0);
    // two halves, that need not wait for each other
    v4f a = (v4f)(0.f), b = (v4f)(0.f);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      a = __builtin_amdgcn_mfma_f32_16x16x4f32(d[k - 1][e], x[k - 1][e], a, 0, 0, 0);
      b = __builtin_amdgcn_mfma_f32_16x16x4f32(d[k - 1][2 + e], x[k - 1][2 + e], b, 0, 0, 0);
    }
    x[k - 1] = -(a + b);
  }
#pragma unroll
  for (int j = 0; j <= I; ++j) x[j] *= beta[j];
  const float inv = write_row<I, 2>(x, out, nullptr);
  if (lane_id() < 16) f.fac_u[16 * I + lane_id()] *= inv;
  if (lane_id() == 0) f.inv_t[I] = inv;
}
// Tile row I of Y's weights of U.
template <int PARTS, int LOW, int I>
__device__ __forceinline__ void form_y_row(const Gates& w, const v4f (&kq)[I + 1], char* out, char* low, Factors& f) {
  const int sub = lane_id() >> 4, col = lane_id() & 15;
  const float fq = w.fq[16 * I + col];
  v4f x[I + 1];
#pragma unroll
  for (int j = 0; j <= I; ++j) {
    if (j < I) {
      x[j] = *(const v4f*)&w.cols[16 * j + 4 * sub] * (fq * w.first[j < 3 ? j : 0][16 * I + col]) * kq[j];
    } else {
      const float gi = w.g[16 * I + col], gil = w.g_low[16 * I + col];
      const v4f gj = *(const v4f*)&w.g[16 * I + 4 * sub], gl = *(const v4f*)&w.g_low[16 * I + 4 * sub];
      const v4f cv = *(const v4f*)&w.fk[16 * I + 4 * sub];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float gamma = exp2((gi - gj[e]) + (gil - gl[e]));
        x[j][e] = 4 * sub + e <= col ? fq * cv[e] * gamma * kq[j][e] : 0.f;
      }
    }
  }
  const float inv = write_row<I, PARTS, LOW>(x, out, low);
  if (lane_id() == 0) f.inv_a[I] = inv;
}

// Which of four waves does what of it. Part A: L's tiles; B: the inverse of L's
// diagonal, Y's rows; C: T's rows. What of the keys' tiles a wave needs it holds itself.
template <int DT, int N, int ROLE>
struct Prepare {
  typedef KeyPlan<DT, N> KP_;
  static constexpr int AP = Parts<DT>::kWeights, LOW = Parts<DT>::kLowBytes;
  // tiles of K K^T: the diagonal one (ROLE, ROLE) and up to two below it
  static constexpr int kBelow = ROLE == 0 || ROLE == 2 ? 2 : 1;
  static constexpr int kI[2] = {ROLE == 0 ? 1 : ROLE == 1 ? 2 : 3, ROLE == 0 ? 2 : 3};
  static constexpr int kJ[2] = {ROLE == 0 ? 0 : ROLE == 1 ? 1 : ROLE == 2 ? 0 : 2, ROLE == 0 ? 0 : 1};
  // rows of Y's weights: role 1 rows 1 and 0, role 2 row 3, role 3 row 2
  static constexpr int kRow = ROLE == 1 ? 1 : ROLE == 2 ? 3 : 2;
  v4f kk[1 + kBelow], kq[kRow + 1], kq0[1];

  __device__ __forceinline__ void load(const char* keys) {
    auto tile = [&](int f) { return *(const v4f*)(keys + f * kFrag + lane_id() * 16); };
    kk[0] = tile(KP_::kKK + lower_tile_at(ROLE, ROLE));
#pragma unroll
    for (int n = 0; n < kBelow; ++n) kk[1 + n] = tile(KP_::kKK + lower_tile_at(kI[n], kJ[n]));
    if constexpr (ROLE > 0) {
#pragma unroll
      for (int j = 0; j <= kRow; ++j) kq[j] = tile(KP_::kKQ + lower_tile_at(kRow, j));
    }
    if constexpr (ROLE == 1) kq0[0] = tile(KP_::kKQ);
  }
  __device__ __forceinline__ void part_a(const Gates& w, v4f (*lower)[kWave], float* diag) {
    diagonal_tile(w, kk[0], ROLE, diag);
#pragma unroll
    for (int n = 0; n < kBelow; ++n)
      lower[kI[n] * (kI[n] - 1) / 2 + kJ[n]][lane_id()] = lower_tile(w, kk[1 + n], kI[n], kJ[n]);
  }
  __device__ __forceinline__ void part_b(Gates& w, float* diag, char* head) {
    typedef HeadPlan<DT> HP_;
    char* const a_frags = head + HP_::kA * kFrag;
    char* const low = head + HP_::kLow * kFrag;
    if constexpr (ROLE == 0) invert_diagonal(diag);
    else form_y_row<AP, LOW, kRow>(w, kq, a_frags, low, w.f);
    if constexpr (ROLE == 1) form_y_row<AP, LOW, 0>(w, kq0, a_frags, low, w.f);
  }
  __device__ __forceinline__ void part_c(Gates& w, const v4f (*lower)[kWave], const float* diag, char* t_frags) {
    form_t_row<ROLE>(w, diag, [&](int k, int j) { return lower[k * (k - 1) / 2 + j][lane_id()]; }, t_frags, w.f);
  }
};

// ---------------------------------------------------------------------------
// the chain
// ---------------------------------------------------------------------------
// V's rows pass through LDS, W waves' columns of a row together: memory is asked for
// 32 W bytes of a row in one piece, instead of 2 bytes for each value.
template <int DT, int W>
constexpr int kRowBytes = 16 * W * sizeof(typename Store<DT>::T);
// A wave's part of the copies of n rows (of 64; behind the end of the sequence its last
// row stands in, and counts as 0 with the keys there) that are `step` bytes apart:
// sizeof(T) of them.
template <int DT, int W>
__device__ __forceinline__ void copy_values(const char* x, uint32_t step, int n, char* values, int wave) {
  constexpr int kRow = kRowBytes<DT, W>, kLanes = kRow / 16, kRows = kWave / kLanes, kCopies = kC / kRows / W;
  static_assert(kCopies == sizeof(typename Store<DT>::T), "copies of a wave");
#pragma unroll
  for (int c = 0; c < kCopies; ++c) {
    const int first = (wave * kCopies + c) * kRows, row = min(first + lane_id() / kLanes, n - 1);
    copy_frag(x + (row * step + lane_id() % kLanes * 16), values + first * kRow);
  }
}

// A wave's 16 rows of a head's state (columns of S^T), and a chunk's way through it. The
// state is held times a power of two, one for each row: 1 / inv_s.
template <int DT, int N>
struct Chain {
  typedef KeyPlan<DT, N> KP_;
  typedef typename Store<DT>::T T;
  static constexpr int KS = KP_::KS, NT = KP_::NT, KP = KP_::KP, AP = Parts<DT>::kWeights, LOW = Parts<DT>::kLowBytes;
  v4f s[NT], ks[4], qs[4], u[4];
  v8h wt[6], wl[6], wa[6 * AP];  // T's fragments, and Y's weights'
  typename LowPart<LOW>::T low[6];  // of those, the lower parts
  uint2 exponents[4];
  float inv_s, inv_r, max_s, max_u;
  int place;  // of the lane's column in a row of the workgroup's

  __device__ __forceinline__ static v8h frag(const char* p, int f) { return *(const v8h*)(p + f * kFrag + lane_id() * 16); }

  __device__ __forceinline__ void init(const DeltaArgs& a, int64_t unit, int P, int p) {
    const int sub = lane_id() >> 4;
    place = (wave_id() * 16 + (lane_id() & 15)) * sizeof(T);
#pragma unroll
    for (int n = 0; n < NT; ++n)
      s[n] = a.init ? *(const v4f*)(a.init + (unit * P + p) * (int64_t)N + 16 * n + 4 * sub) : (v4f)(0.f);
    const Scale sc(column_max(tiles_max(s)) * kStateDown, kWide);
    inv_s = sc.inv;
#pragma unroll
    for (int n = 0; n < NT; ++n) s[n] *= sc.by;
  }
  __device__ __forceinline__ void finish(const DeltaArgs& a, int64_t unit, int P, int p) {
    if (!a.final_state) return;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *(v4f*)(a.final_state + (unit * P + p) * (int64_t)N + 16 * n + 4 * (lane_id() >> 4)) = s[n] * inv_s;
  }
  // The exponents of keys and queries that are not taken to length 1.
  __device__ __forceinline__ void load_exponents(const char* keys) {
#pragma unroll
    for (int i = 0; i < 4; ++i) exponents[i] = *(const uint2*)(keys + KP_::kExponents + (16 * i + 4 * (lane_id() >> 4)) * 2);
  }
  // v divided by the power of two of a key's length (0), or times that of a query's (1), of
  // position 16 i + 4 (lane / 16) + e.
  __device__ __forceinline__ float scaled(float v, int which, int i, int e) const {
    const int word = (int)(e < 2 ? exponents[i].x : exponents[i].y);
    const int x = (int8_t)(word >> (16 * (e & 1) + 8 * which));
    return __builtin_amdgcn_ldexpf(v, which ? -x : x);
  }
  // The weights' lower parts, straight from memory; head: of the chunk.
  __device__ __forceinline__ void load_low(const char* head) {
    if constexpr (LOW > 0) {
      typedef typename LowPart<LOW>::T V;
      const V* const from = (const V*)(head + HeadPlan<DT>::kLow * kFrag) + lane_id();
#pragma unroll
      for (int n = 0; n < 6; ++n) low[n] = from[n * kWave];
    }
  }
  __device__ __forceinline__ v8h low_part(int n) const {
    if constexpr (LOW == 1) return from_upper_bytes(low[n]);
    else return low[n];
  }
  // K S^T and Q S^T. What comes out of LDS is read a step ahead of its use, here and
  // below: a wave has its SIMD to itself, or nearly.
  __device__ __forceinline__ void products(const char* keys) {
    v8h k[2][4 * KP], q[2][4 * KP];
    auto read = [&](int t) {
#pragma unroll
      for (int i = 0; i < 4 * KP; ++i) {
        k[t & 1][i] = frag(keys, KP_::kK + i * KS + t);
        q[t & 1][i] = frag(keys, KP_::kQ + i * KS + t);
      }
    };
    read(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) ks[i] = qs[i] = (v4f)(0.f);
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      if (t + 1 < KS) read(t + 1);
      v8h hi, lo;
      const v4f a = s[2 * t], b = 2 * t + 1 < NT ? s[2 * t + 1 < NT ? 2 * t + 1 : 0] : (v4f)(0.f);
      const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      split8_state(x, hi, lo);
#pragma unroll
      for (int i = 0; i < 4; ++i) ks[i] = mma16(k[t & 1][i], hi, ks[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) qs[i] = mma16(q[t & 1][i], hi, qs[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) ks[i] = mma16(k[t & 1][i], lo, ks[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) qs[i] = mma16(q[t & 1][i], lo, qs[i]);
      if constexpr (KP == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) ks[i] = mma16(k[t & 1][4 + i], hi, ks[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) qs[i] = mma16(q[t & 1][4 + i], hi, qs[i]);
      }
    }
    max_s = column_max(tiles_max(s));
  }
  // T's fragments and Y's weights', for what follows
  __device__ __forceinline__ void read_head(const char* frags) {
#pragma unroll
    for (int n = 0; n < 6; ++n) {
      wt[n] = frag(frags, HeadPlan<DT>::kT + n);
      wl[n] = frag(frags, HeadPlan<DT>::kT + 6 + n);
    }
#pragma unroll
    for (int n = 0; n < 6 * AP; ++n) wa[n] = frag(frags, HeadPlan<DT>::kA + n);
  }
  // R = V - e^g K S^T (divided by p), in the place of K S^T; values: V's rows, of W waves'
  // columns. What meets a key of zeros counts as 0, whatever stands in V behind a sequence's end.
  template <int W>
  __device__ __forceinline__ void remainders(const char* values, const Factors& f, bool unit) {
    const char* const at = values + 4 * (lane_id() >> 4) * kRowBytes<DT, W> + place;
    float v[4][4];
    v4f fk[4];
    const float inv_k = inv_s / kStateDown;
#pragma unroll
    for (int i = 0; i < 4; ++i) fk[i] = *(const v4f*)(f.fac_k + 16 * i + 4 * (lane_id() >> 4));
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] = ld_f<DT>(at + (16 * i + e) * kRowBytes<DT, W>, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) ks[i][e] = fmaf(-fk[i][e] * inv_k, ks[i][e], v[i][e]);
    if (!unit) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) ks[i][e] = scaled(ks[i][e], 0, i, e);
    }
    if (__builtin_amdgcn_readfirstlane(__float_as_int(f.zero_keys))) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) ks[i][e] = fk[i][e] < 0.f ? 0.f : ks[i][e];
    }
  }
  // U = T diag(b) R, as u times inv_r and, of tile row i, inv_t[i].
  __device__ __forceinline__ void changes(const Factors& f) {
    const Scale sc(column_max(tiles_max(ks)), kWide);
    inv_r = sc.inv;
    v8h hi[2], lo[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) split_tiles(ks[2 * t], ks[2 * t + 1], sc.by, sc.by, hi[t], lo[t]);
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = mma16(wt[lower_frag(i, 0)], hi[0], (v4f)(0.f));
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = mma16(wt[lower_frag(i, 0)], lo[0], u[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = mma16(wl[lower_frag(i, 0)], hi[0], u[i]);
#pragma unroll
    for (int i = 2; i < 4; ++i) u[i] = mma16(wt[lower_frag(i, 1)], hi[1], u[i]);
#pragma unroll
    for (int i = 2; i < 4; ++i) u[i] = mma16(wt[lower_frag(i, 1)], lo[1], u[i]);
#pragma unroll
    for (int i = 2; i < 4; ++i) u[i] = mma16(wl[lower_frag(i, 1)], hi[1], u[i]);
    const v4f inv = *(const v4f*)f.inv_t;
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = max4(0.f, u[i]) * inv[i];
    max_u = column_max(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
  }
  // Y of the chunk's `left` positions, through `stage` (32 rows of the wave's 16 columns), and
  //   S' = e^{g_63} S + (e^{g_63 - g} U)^T K,
  // the products added to the scaled state, whose scale lets both keep their bits: the largest
  // of the old state in a column is below 2^18, that of the new terms below 2^9, and one of
  // them is at least half as large. (As they are: factors' and changes' own largest values
  // may lie at different positions.)
  __device__ __forceinline__ void outputs_and_state(const char* turned, const Factors& f, T* stage, char* out,
                                                    uint32_t step, int left, bool unit, float scale) {
    const int sub = lane_id() >> 4;
    v8h k[2][NT];
    v4f fu[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) fu[i] = *(const v4f*)(f.fac_u + 16 * i + 4 * sub);
    const v4f inv_t = *(const v4f*)f.inv_t, inv_a = *(const v4f*)f.inv_a;
    const float decay = f.decay;
#pragma unroll
    for (int n = 0; n < NT; ++n) k[0][n] = frag(turned, 2 * n);
    v4f y[4];
    const Scale sy(max_u);
    {
      v8h hi[2], lo[2];
#pragma unroll
      for (int t = 0; t < 2; ++t)
        split_tiles(u[2 * t], u[2 * t + 1], inv_t[2 * t] * sy.by, inv_t[2 * t + 1] * sy.by, hi[t], lo[t]);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = mma16(wa[lower_frag(i, 0)], hi[0], (v4f)(0.f));
#pragma unroll
      for (int i = 2; i < 4; ++i) y[i] = mma16(wa[lower_frag(i, 1)], hi[1], y[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = mma16(wa[lower_frag(i, 0)], lo[0], y[i]);
#pragma unroll
      for (int i = 2; i < 4; ++i) y[i] = mma16(wa[lower_frag(i, 1)], lo[1], y[i]);
      if constexpr (LOW > 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = mma16(low_part(lower_frag(i, 0)), hi[0], y[i]);
#pragma unroll
        for (int i = 2; i < 4; ++i) y[i] = mma16(low_part(lower_frag(i, 1)), hi[1], y[i]);
      }
      if constexpr (AP == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = mma16(wa[6 + lower_frag(i, 0)], hi[0], y[i]);
#pragma unroll
        for (int i = 2; i < 4; ++i) y[i] = mma16(wa[6 + lower_frag(i, 1)], hi[1], y[i]);
      }
    }
    v4f w[4];  // diag(e^{g_63 - g}) U
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = u[i] * fu[i];
    const float was = inv_s / kStateDown, max_w = column_max(tiles_max(w));
    const Scale sc(fmaxf(max_s * inv_s * decay * kStateDown, max_w * inv_r), kWide);
    const float keep = decay * (inv_s * sc.by), by = inv_r * sc.by;
    inv_s = sc.inv;
#pragma unroll
    for (int n = 0; n < NT; ++n) s[n] *= keep;
    v8h hi[2], lo[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) split_tiles(w[2 * t], w[2 * t + 1], by, by, hi[t], lo[t]);
#pragma unroll
    for (int n = 0; n < NT; ++n) k[1][n] = frag(turned, 2 * n + 1);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n] = mma16(k[t][n], hi[t], s[n]);
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n] = mma16(k[t][n], lo[t], s[n]);
      if constexpr (KP == 2) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n] = mma16(frag(turned, 2 * NT + 2 * n + t), hi[t], s[n]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float inv = sy.inv * inv_r * inv_a[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[i][e] *= inv;
    }
    if (!unit) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[i][e] = scaled(y[i][e] * scale, 1, i, e);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const v4f fq = *(const v4f*)(f.fac_q + 16 * i + 4 * sub);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[i][e] = fmaf(fq[e] * was, qs[i][e], y[i][e]);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          stage[(16 * i + 4 * sub + e) * 16 + (lane_id() & 15)] = to_store<DT>(y[2 * half + i][e]);
      wave_sync();
      // 32 rows in pieces of 16 bytes, to rows of Y `step` bytes apart
      constexpr int kPer = 16 * sizeof(T) / 16;  // pieces of a row
#pragma unroll
      for (int n = 0; n < kPer / 2; ++n) {
        const int row = (n * kWave + lane_id()) / kPer, piece = lane_id() % kPer;
        const v4u v = *(const v4u*)((const char*)stage + row * 16 * sizeof(T) + piece * 16);
        if (32 * half + row < left) *(v4u*)(out + ((32 * half + row) * step + piece * 16)) = v;
      }
      wave_sync();
    }
  }
};

// ---------------------------------------------------------------------------
// kernels of a head
// ---------------------------------------------------------------------------
template <int DT, int N>
__global__ __launch_bounds__(256) void k_delta_prepare(DeltaArgs a, const char* ws, char* ws_heads, int64_t L, int H,
                                                     int G, int hpg, int chunks, int64_t total) {
  typedef KeyPlan<DT, N> KP_;
  typedef HeadPlan<DT> HP_;
  __shared__ __attribute__((aligned(16))) Gates w;
  __shared__ __attribute__((aligned(16))) v4f lower[6][kWave];
  __shared__ __attribute__((aligned(16))) float diag[4 * kDiag];
  auto chunk = [&](auto role, int64_t item) {
    constexpr int kRole = decltype(role)::value;
    const int ck = (int)(item % chunks);
    const int64_t unit = item / chunks, b = unit / H;
    const int h = (int)(unit % H);
    const char* const keys = ws + ((b * G + h / hpg) * (int64_t)chunks + ck) * KP_::kBytes;
    char* const out = ws_heads + item * HP_::kBytes;
    Prepare<DT, N, kRole> p;
    p.load(keys);
    if constexpr (kRole == 0) {
      GateInputs in;
      in.load<DT>(a, (const float*)(keys + KP_::kFac * kFrag), b * L, (int64_t)ck * kC, L, H, h);
      form_gates(w, in, a.A[h], a.unit);
    }
    __syncthreads();
    p.part_a(w, lower, diag);
    __syncthreads();
    p.part_b(w, diag, out);
    __syncthreads();
    p.part_c(w, lower, diag, out + HP_::kT * kFrag);
    __syncthreads();
    if (threadIdx.x < sizeof(Factors) / sizeof(float))
      ((float*)(out + HP_::kFac * kFrag))[threadIdx.x] = ((const float*)&w.f)[threadIdx.x];
    __syncthreads();  // the next chunk's gates overwrite this one's
  };
  for (int64_t item = blockIdx.x; item < total; item += gridDim.x) {
    switch (wave_id()) {
      case 0: chunk(std::integral_constant<int, 0>(), item); break;
      case 1: chunk(std::integral_constant<int, 1>(), item); break;
      case 2: chunk(std::integral_constant<int, 2>(), item); break;
      default: chunk(std::integral_constant<int, 3>(), item);
    }
  }
}

// A workgroup of W waves takes 16 W rows of a head's state, through whose chunks the
// fragments and V's rows come through LDS.
//   DEEP: two buffers of each; the next chunk's copies are on their way all the while,
//   with one barrier a chunk. One workgroup on a CU.
//   Otherwise one, in three parts, that are free and copied anew one after the other: K
//   and Q after the products with them, T, Y's weights and V once they are in registers
//   (the factors have two buffers), K^T at the chunk's end, with barriers in between. Two
//   workgroups on a CU (16-bit types), which cover one another's waits.
template <int DT, int N, int W, bool DEEP>
__global__ __launch_bounds__(64 * W, DT != DT_F32 && W == 4 && !DEEP ? 2 : 1) void k_delta_scan(
    DeltaArgs a, const char* ws, const char* ws_heads, int64_t L, int H, int G, int hpg, int P, int chunks,
    bool gather) {
  typedef KeyPlan<DT, N> KP_;
  typedef HeadPlan<DT> HP_;
  typedef typename Store<DT>::T T;
  constexpr int kFirst = KP_::kT * kFrag, kTurned = KP_::kTurned * kFrag, kHead = HP_::kFac * kFrag;
  constexpr int kValues = kC * kRowBytes<DT, W>;
  // separate objects, so that the compiler sees that a read of one need not wait for
  // the copies into another
  __shared__ __attribute__((aligned(1024))) char first0[kFirst], turned0[kTurned], head0[kHead], values0[kValues];
  __shared__ __attribute__((aligned(1024))) char first1[DEEP ? kFirst : 16], turned1[DEEP ? kTurned : 16];
  __shared__ __attribute__((aligned(1024))) char head1[DEEP ? kHead : 16], values1[DEEP ? kValues : 16];
  __shared__ __attribute__((aligned(1024))) char factors0[kFrag], factors1[kFrag];
  __shared__ __attribute__((aligned(1024))) T stage[W][kC / 2 * 16];
  constexpr int E = sizeof(T);
  const int wv = wave_id();
  // Consecutive workgroups go to the eight XCDs in turn. With `gather` each XCD takes a
  // contiguous run of the slices.
  const int slices = P / (16 * W), xcd = blockIdx.x % 8, per = (int)gridDim.x / 8, extra = (int)gridDim.x % 8;
  const int place = gather ? xcd * per + min(xcd, extra) + (int)blockIdx.x / 8 : (int)blockIdx.x;
  const int64_t unit = place / slices, b = unit / H;
  const int h = (int)(unit % H), start = place % slices * W * 16, p = start + wv * 16 + (lane_id() & 15);
  const uint32_t step = (uint32_t)H * P * E;  // between rows: 64 of them are less than 2^32 bytes
  const char* const x = (const char*)a.X + ((b * L * H + h) * P + start) * E;
  char* const y = (char*)a.Y + ((b * L * H + h) * P + start + wv * 16) * E;
  const char* const keys = ws + (b * G + h / hpg) * (int64_t)chunks * KP_::kBytes;
  const char* const heads = ws_heads + unit * (int64_t)chunks * HP_::kBytes;
  auto left = [&](int i) { return (int)min(L - (int64_t)i * kC, (int64_t)kC); };
  auto copy_first = [&](int i, char* to) { copy_frags<KP_::kT, W>(keys + i * (int64_t)KP_::kBytes, to, wv); };
  auto copy_turned = [&](int i, char* to) {
    copy_frags<KP_::kTurned, W>(keys + i * (int64_t)KP_::kBytes + KP_::kT * kFrag, to, wv);
  };
  auto copy_head = [&](int i, char* to, char* factors, char* values) {
    copy_frags<HP_::kFac, W>(heads + i * (int64_t)HP_::kBytes, to, wv);
    if (wv == W - 1) copy_frag(heads + i * (int64_t)HP_::kBytes + HP_::kFac * kFrag + lane_id() * 16, factors);
    copy_values<DT, W>(x + i * (kC * (int64_t)step), step, left(i), values, wv);
  };
  copy_first(0, first0);
  copy_turned(0, turned0);
  copy_head(0, head0, factors0, values0);
  Chain<DT, N> c;
  c.init(a, unit, P, p);
  meet<0>();
  // Chunk i, from one set of buffers; the next one's go to first, turned, head, factors
  // and vals. Where copies are, this chunk is whole, and a wave's newest memory operations
  // are the E stores of Y, after at least kHeadCopies of copy_head.
  constexpr int kHeadCopies = HP_::kFac / W + E;
  auto chunk = [&](int i, const char* kq, const char* kt, const char* frags, const char* fac, const char* values, char* first,
                   char* turned, char* head, char* factors, char* vals) __attribute__((always_inline)) {
    const bool more = i + 1 < chunks;
    const Factors& f = *(const Factors*)fac;
    if (!a.unit) c.load_exponents(keys + i * (int64_t)KP_::kBytes);
    c.load_low(heads + i * (int64_t)HP_::kBytes);  // here by the barrier after the products
    if (DEEP && more) {
      copy_first(i + 1, first);
      copy_turned(i + 1, turned);
      copy_head(i + 1, head, factors, vals);
      asm volatile("" ::: "memory");
    }
    c.products(kq);
    if constexpr (!DEEP) {
      meet<0>();
      if (more) copy_first(i + 1, first);
    }
    c.read_head(frags);
    c.template remainders<W>(values, f, a.unit);
    if constexpr (!DEEP) {
      meet<64>();
      if (more) copy_head(i + 1, head, factors, vals);
      asm volatile("" ::: "memory");
    }
    c.changes(f);
    c.outputs_and_state(kt, f, stage[wv], y + i * (kC * (int64_t)step), step, left(i), a.unit, a.scale);
    meet<DEEP ? E : kHeadCopies + E>();
    if (!DEEP && more) copy_turned(i + 1, turned);
  };
  for (int i = 0; i < chunks; i += 2) {
    if constexpr (DEEP) {
      chunk(i, first0, turned0, head0, factors0, values0, first1, turned1, head1, factors1, values1);
      if (i + 1 < chunks) chunk(i + 1, first1, turned1, head1, factors1, values1, first0, turned0, head0, factors0, values0);
    } else {
      chunk(i, first0, turned0, head0, factors0, values0, first0, turned0, head0, factors1, values0);
      if (i + 1 < chunks) chunk(i + 1, first0, turned0, head0, factors1, values0, first0, turned0, head0, factors0, values0);
    }
  }
  c.finish(a, unit, P, p);
}

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------
template <int DT, int N, int W>
hipError_t scan(const Dims& d, const DeltaArgs& a, const char* keys, const char* heads, int64_t ncu, hipStream_t st) {
  const int64_t wgs = d.B * d.H * (d.P / (16 * W));
  // Slices of a head share its fragments, and heads of a group the keys': one XCD's L2
  // serves them where that is one's own (us with and without, bf16: 4 x 4096 positions of 32
  // heads of 128 x 128 383 and 395; 8 x 2048 of 80 of 64 x 128 433 and 444), but not where all
  // XCDs read one group's keys either way (2048 of 64 heads 132 and 129).
  const bool gather = d.P > 16 * W || d.B * d.G >= 8;
  // Two buffers where a CU has one workgroup at most (us with two and one, bf16: 2048 positions
  // of 64 heads of 64 x 128 129 and 138; 300 of 64 heads of 64 x 64 30 and 32), one where it may
  // have two (8 x 2048 of 80 503 and 433; 4 x 1024 of 96 161 and 139). fp32 has no room for two.
  if constexpr (DT != DT_F32) {
    if (wgs <= ncu) {
      hipLaunchKernelGGL((k_delta_scan<DT, N, W, true>), dim3((unsigned)wgs), dim3(64 * W), 0, st, a, keys, heads, d.L, d.H,
                         d.G, d.hpg, d.P, d.c, gather);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((k_delta_scan<DT, N, W, false>), dim3((unsigned)wgs), dim3(64 * W), 0, st, a, keys, heads, d.L, d.H,
                     d.G, d.hpg, d.P, d.c, gather);
  return hipGetLastError();
}

template <int DT, int N>
hipError_t go(const Dims& d, const DeltaArgs& a, char* ws, hipStream_t st) {
  const int64_t total = d.B * d.G * (int64_t)d.c;
  hipLaunchKernelGGL((k_delta_keys<DT, N>), dim3((unsigned)min(total, (int64_t)1 << 20)), dim3(256), 0, st, a, ws, d.L, d.G,
                     d.c, total);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  char* const heads = ws + total * KeyPlan<DT, N>::kBytes;
  const int64_t units = d.B * d.H * (int64_t)d.c, ncu = cu_count() > 0 ? cu_count() : 256;
  hipLaunchKernelGGL((k_delta_prepare<DT, N>), dim3((unsigned)min(units, (int64_t)1 << 20)), dim3(256), 0, st, a, ws, heads,
                     d.L, d.H, d.G, d.hpg, d.c, units);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  // Four waves where the head has them (us at 4, 2 and 1: 8 x 2048 positions of 80 heads of
  // 64 x 128 fp16 443, 546 and 834; one sequence of 2048, 64 heads, bf16 129, 134 and 145).
  switch (d.P) {
    case 16: return scan<DT, N, 1>(d, a, ws, heads, ncu, st);
    case 32: return scan<DT, N, 2>(d, a, ws, heads, ncu, st);
    default: return scan<DT, N, 4>(d, a, ws, heads, ncu, st);
  }
}

template <int DT>
hipError_t go_n(const Dims& d, const DeltaArgs& a, char* ws, hipStream_t st) {
  switch (d.N) {
    case 16: return go<DT, 16>(d, a, ws, st);
    case 32: return go<DT, 32>(d, a, ws, st);
    case 64: return go<DT, 64>(d, a, ws, st);
    case 128: return go<DT, 128>(d, a, ws, st);
    default: return hipErrorInvalidValue;
  }
}

template <int DT>
size_t bytes_n(const Dims& d) {
  const size_t bg = (size_t)d.B * d.G * d.c, bh = (size_t)d.B * d.H * d.c;
  const size_t keys = d.N == 16 ? KeyPlan<DT, 16>::kBytes
                      : d.N == 32 ? KeyPlan<DT, 32>::kBytes
                      : d.N == 64 ? KeyPlan<DT, 64>::kBytes : KeyPlan<DT, 128>::kBytes;
  return bg * keys + bh * HeadPlan<DT>::kBytes;
}

}  // namespace

size_t delta_workspace_bytes(const Dims& d, int dtype) {
  return dtype == DT_F32 ? bytes_n<DT_F32>(d) : dtype == DT_F16 ? bytes_n<DT_F16>(d) : bytes_n<DT_BF16>(d);
}

hipError_t launch_delta_chunks(const Dims& d, int dtype, const DeltaArgs& a, void* ws, hipStream_t st) {
  switch (dtype) {
    case DT_F32: return go_n<DT_F32>(d, a, (char*)ws, st);
    case DT_F16: return go_n<DT_F16>(d, a, (char*)ws, st);
    case DT_BF16: return go_n<DT_BF16>(d, a, (char*)ws, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ssd
