// The gated delta rule in chunks of 64 positions. With g_i the sum of dt A over a
// chunk up to position i, S [P, N] the state before the chunk and u_i the change that
// position i writes,
//   L_ij = b_i e^{g_i - g_j} k_i.k_j  (j < i),   T = (1 + L)^-1,
//   U = T diag(b) (V - diag(e^g) K S^T),
//   Y = scale (diag(e^g) Q S^T + (Q K^T . e^{g_i - g_j}, j <= i) U),
//   S' = e^{g_63} S + (diag(e^{g_63 - g}) U)^T K.
//
// Two launches. k_delta_prepare forms, for every chunk at once, what does not need
// the state: keys and queries as matrix operands, T diag(b) and the weights of U in Y.
// k_delta_scan goes through a head's chunks in order with the state in registers; a
// wave owns 16 NC rows of S (columns here: S^T is [N, P]), which no other needs.
//
// The products of the scan follow one another without a step through LDS: the
// 16 x 16 result tiles hold, in lane i, rows 4 (i / 16) .. + 3 of column i % 16, and
// two of them are an operand of 32 rows whose order of rows the other operand takes
// on too. An operand's lane i thus has, of step s, the 8 positions
// 32 s + 4 (i / 16) + (0..3) and 16 more than those ("fragments" below).
//
// Precision. The state is kept and returned in fp32, so that no operand of the
// products that lead to it may be rounded to 16 bits. Each is taken as a sum of two
// fp16 numbers (22 significant bits), after a power of two has brought the largest of
// its column (or row, or matrix) to 2^8: what is below 2^-32 of that is lost. Keys and
// queries of 16-bit types are exact in one fp16 number in that way, fp32 ones in two.
// Products of two lower parts (2^-22 of the rest) are left out. For Y alone, which is
// rounded to 16 bits, fewer parts do: see kStateY, kNewY.
#include "ssd_delta.hpp"

namespace ssd {
namespace {

constexpr int kC = kDeltaChunk;

// What the operands of one type are made of.
template <int DT>
struct Parts {
  static constexpr int kKeys = DT == DT_F32 ? 2 : 1;     // fp16 numbers of a key's or query's element
  static constexpr int kWeights = DT == DT_F32 ? 2 : 1;  // of Y's weights of U: 2^-12 of an fp16 or bf16 Y's term
  static constexpr int kStateY = DT == DT_BF16 ? 1 : 2;  // of S in Y: one rounds to 2^-12, a 16th of bf16's step
  static constexpr int kNewY = DT == DT_BF16 ? 1 : 2;    // of U in Y
};

// ---------------------------------------------------------------------------
// workspace
// ---------------------------------------------------------------------------
constexpr int kFrag = 1024;  // bytes: 16 for each lane

// Of each (batch, group, chunk): fragments of K and Q (4 tiles of 16 positions, KS
// steps of 32 channels) and of K^T (NT tiles of 16 channels, 2 steps of 32 positions).
template <int DT, int N>
struct KeyPlan {
  static constexpr int KS = (N + 31) / 32, NT = N / 16, KP = Parts<DT>::kKeys;
  static constexpr int kK = 0, kQ = 4 * KS * KP, kT = 8 * KS * KP, kFrags = kT + 2 * NT * KP;
  static constexpr size_t kBytes = (size_t)kFrags * kFrag;
};
// Of each (batch, head, chunk): fragments of T diag(b) (6 that are not zero, two
// parts), of Y's weights (6), then floats: for each position the factors of K S^T in R
// (kFacK), of Q S^T in Y (kFacQ) and of U in S' (kFacU), the state's decay, the factors
// that undo the scaling of T and of the weights, and the largest of kFacU.
template <int DT>
struct HeadPlan {
  static constexpr int kT = 0, kA = 12, kFac = 12 + 6 * Parts<DT>::kWeights, kFrags = kFac + 1;
  static constexpr size_t kBytes = (size_t)kFrags * kFrag;
};
enum { kFacK = 0, kFacQ = kC, kFacU = 2 * kC, kDecay = 3 * kC, kInvT, kInvA, kMaxU };

// The fragment of tile row i and step s of a lower triangle of 4 x 4 tiles.
__device__ __forceinline__ constexpr int lower_frag(int i, int s) { return i < 2 ? i : 2 * i - 2 + s; }

// ---------------------------------------------------------------------------
// scaling and parts
// ---------------------------------------------------------------------------
// The power of two that brings m to [2^8, 2^9), and its inverse; from 2^-82 on down it
// is 2^90, so that products of two of them stay in fp32's range.
struct Scale {
  float by, inv;
  __device__ __forceinline__ explicit Scale(float m) {
    const int e = min(262 - (int)((__float_as_uint(m) >> 23) & 255), 217);
    by = __uint_as_float((uint32_t)e << 23);
    inv = __uint_as_float((uint32_t)(254 - e) << 23);
  }
};

typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// Eight values, times a power of two, as fp16 numbers, and what that leaves of them
// as eight more.
__device__ __forceinline__ void split8(const float (&x)[8], float by, v8h& hi, v8h& lo) {
#pragma unroll
  for (int e = 0; e < 8; ++e) hi[e] = (_Float16)(x[e] * by);
#pragma unroll
  for (int e = 0; e < 8; ++e) lo[e] = (_Float16)fmaf(x[e], by, -(float)hi[e]);
}
// Rows 4 (lane / 16) .. of two result tiles, as an operand.
__device__ __forceinline__ void split_tiles(v4f a, v4f b, float by, v8h& hi, v8h& lo) {
  const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  split8(x, by, hi, lo);
}
// 2^x
__device__ __forceinline__ float exp2(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ v4f mma16(v8h a, v8h b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
// 16 x 16 x 16 in fp32: a holds rows (lane % 16) of the left matrix, columns 4 (lane / 16)
// + (0..3); b a result tile.
__device__ __forceinline__ v4f mma32(v4f a, v4f b, v4f c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
  return c;
}

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ float max4(v4f v) { return fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))); }

// ---------------------------------------------------------------------------
// preparation
// ---------------------------------------------------------------------------
// A workgroup of four waves takes a chunk of a group's keys and queries, and `heads`
// of the group's heads, a wave one at a time.
struct PrepareWave {
  static constexpr int kDiagRow = 20, kDiag = 16 * kDiagRow + 4;  // floats; the blocks start 4 banks apart
  float g[kC], g_low[kC];  // sums of dt A log2(e): twice fp32's bits, as their differences count
  float beta[kC], cols[kC], rows[4][kC], first[3][kC];
  float diag[4 * kDiag];
};

template <int DT, int N>
__global__ __launch_bounds__(256) void k_delta_prepare(DeltaArgs a, char* ws_keys, char* ws_heads, int64_t L, int H,
                                                     int G, int hpg, int chunks, int blocks, int heads, int64_t total) {
  typedef KeyPlan<DT, N> KP_;
  typedef HeadPlan<DT> HP_;
  constexpr int KS = KP_::KS, NT = KP_::NT, KP = KP_::KP, AP = Parts<DT>::kWeights;
  // K's fragments, then Q's; once the tiles are made, what a wave holds of its head
  constexpr int kFragBytes = 8 * KS * KP * kFrag, kWaveBytes = 4 * sizeof(PrepareWave);
  __shared__ __attribute__((aligned(16))) char frags[kFragBytes > kWaveBytes ? kFragBytes : kWaveBytes];
  // tiles of K K^T and K Q^T: of tile row i, column j at i (i + 1) / 2 + j
  __shared__ __attribute__((aligned(16))) float4 lds_kk[10][kWave], lds_kq[10][kWave];
  __shared__ __attribute__((aligned(16))) float lds_fk[kC], lds_fq[kC];
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_id(), sub = lane >> 4, col = lane & 15;

  for (int64_t item = blockIdx.x; item < total; item += gridDim.x) {
    const int hb = (int)(item % blocks);
    const int64_t bgc = item / blocks;  // (b G + g) chunks + chunk
    const int ck = (int)(bgc % chunks);
    const int64_t bg = bgc / chunks, b = bg / G;
    const int g = (int)(bg % G);
    const int64_t pos0 = (int64_t)ck * kC;
    char* const out_keys = ws_keys + bgc * KP_::kBytes;

    // Rows of K and Q: four threads a row, a step's 32 channels each.
    {
      const int row = tid >> 2, s = tid & 3;
      const bool live = s < KS && pos0 + row < L;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const void* const src = which ? a.C : a.B;
        constexpr int E = N < 32 ? N : 32;
        float x[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = 0.f;
        if (live) {
          const int64_t at = ((b * L + pos0 + row) * G + g) * N + s * 32;
#pragma unroll
          for (int e = 0; e < E; e += 8) {
            float t[8];
            ld8_f<DT>(src, at + e, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[e + i] = t[i];
          }
        }
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) m = fmaxf(m, fabsf(x[e]));
        m = fmaxf(m, __shfl_xor(m, 1));
        m = fmaxf(m, __shfl_xor(m, 2));
        const Scale sc(m);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          x[e] *= sc.by;
          ss = fmaf(x[e], x[e], ss);
        }
        ss += __shfl_xor(ss, 1);
        ss += __shfl_xor(ss, 2);
        if (s == 0) {
          float f = sc.inv;
          if (a.unit) {
            const float eps = a.eps * sc.by * sc.by;
            ss += eps;
            // a row of zeros without eps stays zeros; next to a far larger eps the row counts for nothing
            f = eps > 0x1p126f ? sc.inv * rsqrtf(a.eps) : ss > 0.f ? rsqrtf(ss) : 0.f;
          }
          if (which) lds_fq[row] = f * a.scale;
          else lds_fk[row] = f;
        }
        if (s < KS) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float t[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              t[e] = x[4 * q + e];
              t[4 + e] = x[16 + 4 * q + e];
            }
            v8h hi, lo;
            split8(t, 1.f, hi, lo);
            const int at = ((which * KP * 4 + (row >> 4)) * KS + s) * kFrag + (q * 16 + (row & 15)) * 16;
            *(v8h*)(frags + at) = hi;
            if (hb == 0) *(v8h*)(out_keys + at) = hi;
            if constexpr (KP == 2) {
              constexpr int kLo = 4 * KS * kFrag;
              *(v8h*)(frags + at + kLo) = lo;
              if (hb == 0) *(v8h*)(out_keys + at + kLo) = lo;
            }
          }
        }
      }
    }
    __syncthreads();

    if (hb == 0) {
      for (int f = wv; f < 2 * NT * KP; f += 4) {  // K^T: channel 16 nt + col, positions of step s
        const int part = f / (2 * NT), nt = f / 2 % NT, s = f & 1, n = 16 * nt + col;
        const char* const from = frags + part * 4 * KS * kFrag + (n >> 5) * kFrag + ((n & 15) >> 2) * 256 + ((n & 3) + ((n >> 4) & 1) * 4) * 2;
        v8h v;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int p = 4 * sub + (e & 3);  // of tile 2 s + e / 4
          v[e] = *(const _Float16*)(from + (2 * s + (e >> 2)) * KS * kFrag + p * 16);
        }
        *(v8h*)(out_keys + (KP_::kT + f) * kFrag + lane * 16) = v;
      }
    }
    // tiles of K K^T (rows i, columns j) and K Q^T (rows j, columns i), j <= i
    auto frag = [&](int which, int part, int tile, int s) {
      return *(const v8h*)(frags + (((which * KP + part) * 4 + tile) * KS + s) * kFrag + lane * 16);
    };
    for (int t = wv; t < 20; t += 4) {
      const int which = t >= 10, u = which ? t - 10 : t;
      const int i = u < 1 ? 0 : u < 3 ? 1 : u < 6 ? 2 : 3, j = u - i * (i + 1) / 2;
      const int left = which ? j : i, right = which ? i : j;
      v4f acc = (v4f)(0.f);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        acc = mma16(frag(0, 0, left, s), frag(which, 0, right, s), acc);
        if constexpr (KP == 2) {
          acc = mma16(frag(0, 0, left, s), frag(which, 1, right, s), acc);
          acc = mma16(frag(0, 1, left, s), frag(which, 0, right, s), acc);
        }
      }
      (which ? lds_kq : lds_kk)[u][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    }
    __syncthreads();

    PrepareWave& w = ((PrepareWave*)frags)[wv];
    const int last = min(hpg, (hb + 1) * heads);
    for (int hi_ = hb * heads + wv; hi_ < last; hi_ += 4) {
      const int h = g * hpg + hi_;
      char* const out = ws_heads + ((b * H + h) * (int64_t)chunks + ck) * HP_::kBytes;
      float* const fac = (float*)(out + HP_::kFac * kFrag);
      // a lane for each position; behind the end nothing decays and nothing is written
      {
        const int64_t pos = b * L + pos0 + lane;
        const bool live = pos0 + lane < L;
        const float dt = live ? ld_f<DT>(a.dt, pos * H + h) : 0.f;
        const float beta = live ? delta_beta<DT>(a, pos, h) : 0.f;
        double gs = (double)dt * ((double)a.A[h] * 1.4426950408889634);
#pragma unroll
        for (int o = 1; o < kWave; o *= 2) {
          const double up = __shfl_up(gs, o);
          if (lane >= o) gs += up;
        }
        const double end = __shfl(gs, lane | 15), total_g = __shfl(gs, kC - 1);
        const float fk = lds_fk[lane], fq = lds_fq[lane], eg = exp2((float)gs);
        const float fu = exp2((float)(total_g - gs)) * fk;
        w.g[lane] = (float)gs;
        w.g_low[lane] = (float)(gs - (double)(float)gs);
        w.beta[lane] = beta;
        w.cols[lane] = exp2((float)(end - gs)) * fk;  // from the position to the end of its 16
        w.rows[3][lane] = beta * fk;
#pragma unroll
        for (int q = 0; q < 3; ++q) {  // from the end of the 16 positions q
          const float first = exp2((float)fmin(gs - __shfl(gs, 16 * q + 15), 0.0));
          w.first[q][lane] = first;
          w.rows[q][lane] = beta * fk * first;
        }
        fac[kFacK + lane] = eg * fk;
        fac[kFacQ + lane] = eg * fq;
        fac[kFacU + lane] = fu;
        float most = fu;
#pragma unroll
        for (int o = 1; o < kWave; o *= 2) most = fmaxf(most, __shfl_xor(most, o));
        if (lane == 0) {
          fac[kDecay] = exp2((float)total_g);
          fac[kMaxU] = most;
        }
      }
      wave_sync();

      // L: tiles below the diagonal stay in registers, the diagonal ones go to LDS
      v4f l[4][4], x[4][4];  // tile row, tile column
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j) {
          const float4 kk = lds_kk[i * (i + 1) / 2 + j][lane], rf = *(const float4*)&w.rows[j < i ? j : 3][16 * i + 4 * sub];
          const float kv[4] = {kk.x, kk.y, kk.z, kk.w}, rv[4] = {rf.x, rf.y, rf.z, rf.w};
          if (j < i) {
            const float c = w.cols[16 * j + col];
#pragma unroll
            for (int e = 0; e < 4; ++e) l[i][j][e] = rv[e] * c * kv[e];
          } else {
            const float gj = w.g[16 * i + col], gl = w.g_low[16 * i + col], c = lds_fk[16 * i + col];
            const v4f gi = *(const v4f*)&w.g[16 * i + 4 * sub], gil = *(const v4f*)&w.g_low[16 * i + 4 * sub];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float gamma = exp2(fminf((gi[e] - gj) + (gil[e] - gl), 0.f));
              w.diag[i * PrepareWave::kDiag + (4 * sub + e) * PrepareWave::kDiagRow + col] =
                  col < 4 * sub + e ? rv[e] * c * gamma * kv[e] : 0.f;
            }
          }
        }
      wave_sync();
      // inverses of the diagonal blocks: 16 lanes a block, each a column, from the top
      {
        const float* const d = w.diag + sub * PrepareWave::kDiag;
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float v = i == col ? 1.f : 0.f;
#pragma unroll
          for (int k = 0; k < i; ++k) v = fmaf(-d[i * PrepareWave::kDiagRow + k], t[k], v);
          t[i] = v;
        }
        wave_sync();
#pragma unroll
        for (int i = 0; i < 16; ++i) w.diag[sub * PrepareWave::kDiag + i * PrepareWave::kDiagRow + col] = t[i];
      }
      wave_sync();
      v4f dc[4];  // the blocks' own tiles
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* const d = w.diag + i * PrepareWave::kDiag;
#pragma unroll
        for (int e = 0; e < 4; ++e) dc[i][e] = d[(4 * sub + e) * PrepareWave::kDiagRow + col];
        const float4 v = *(const float4*)(d + col * PrepareWave::kDiagRow + 4 * sub);
        x[i][i] = (v4f){v.x, v.y, v.z, v.w};
      }
      // x: transposed tiles of T, from T_ij = -(sum_{j<k<=i} T_ik L_kj) T_jj
#pragma unroll
      for (int off = 1; off < 4; ++off)
#pragma unroll
        for (int j = 0; j + off < 4; ++j) {
          const int i = j + off;
          v4f acc = (v4f)(0.f);
#pragma unroll
          for (int k = j + 1; k <= i; ++k) acc = mma32(l[k][j], x[i][k], acc);
          x[i][j] = -mma32(dc[j], acc, (v4f)(0.f));
        }

      // two tiles of a row as a fragment
      auto write = [&](const v4f (&m)[4][4], float by, int first, int parts) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int s = 0; s <= i / 2; ++s) {
            v8h hi, lo;
            split_tiles(m[i][2 * s], 2 * s + 1 <= i ? m[i][2 * s + 1 <= i ? 2 * s + 1 : 0] : (v4f)(0.f), by, hi, lo);
            *(v8h*)(out + (first + lower_frag(i, s)) * kFrag + lane * 16) = hi;
            if (parts == 2) *(v8h*)(out + (first + 6 + lower_frag(i, s)) * kFrag + lane * 16) = lo;
          }
      };
      auto largest = [&](const v4f (&m)[4][4]) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j <= i; ++j) v = fmaxf(v, max4(m[i][j]));
#pragma unroll
        for (int o = 1; o < kWave; o *= 2) v = fmaxf(v, __shfl_xor(v, o));
        return v;
      };
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j) {
          const float4 v = *(const float4*)&w.beta[16 * j + 4 * sub];
          x[i][j] *= (v4f){v.x, v.y, v.z, v.w};
        }
      const Scale st(largest(x));
      write(x, st.by, HP_::kT, 2);
      // Y's weights, transposed too: rows j, columns i
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j) {
          const float4 kq = lds_kq[i * (i + 1) / 2 + j][lane];
          const float kv[4] = {kq.x, kq.y, kq.z, kq.w}, fq = lds_fq[16 * i + col];
          if (j < i) {
            const float4 cf = *(const float4*)&w.cols[16 * j + 4 * sub];
            const float cv[4] = {cf.x, cf.y, cf.z, cf.w}, r = fq * w.first[j][16 * i + col];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][j][e] = r * cv[e] * kv[e];
          } else {
            const float gi = w.g[16 * i + col], gil = w.g_low[16 * i + col];
            const v4f gj = *(const v4f*)&w.g[16 * i + 4 * sub], gl = *(const v4f*)&w.g_low[16 * i + 4 * sub];
            const v4f cv = *(const v4f*)&lds_fk[16 * i + 4 * sub];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float gamma = exp2(fminf((gi - gj[e]) + (gil - gl[e]), 0.f));
              x[i][j][e] = 4 * sub + e <= col ? fq * cv[e] * gamma * kv[e] : 0.f;
            }
          }
        }
      const Scale sa(largest(x));
      write(x, sa.by, HP_::kA, AP);
      if (lane == 0) {
        fac[kInvT] = st.inv;
        fac[kInvA] = sa.inv;
      }
      wave_sync();  // the next head's values overwrite this one's
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// scan
// ---------------------------------------------------------------------------
// NC consecutive values of a row.
template <int DT, int NC>
__device__ __forceinline__ void load_cols(const char* p, float (&v)[NC]) {
  if constexpr (NC == 1) {
    v[0] = ld_f<DT>(p, 0);
  } else if constexpr (DT == DT_F32) {
    const float2 t = *(const float2*)p;
    v[0] = t.x; v[1] = t.y;
  } else {
    const uint32_t t = *(const uint32_t*)p;
    if constexpr (DT == DT_BF16) {
      v[0] = __uint_as_float(t << 16); v[1] = __uint_as_float(t & 0xffff0000u);
    } else {
      const v2h h = __builtin_bit_cast(v2h, t);
      v[0] = (float)h[0]; v[1] = (float)h[1];
    }
  }
}
template <int DT, int NC>
__device__ __forceinline__ void store_cols(char* p, const float (&v)[NC]) {
  if constexpr (NC == 1) *(typename Store<DT>::T*)p = to_store<DT>(v[0]);
  else if constexpr (DT == DT_F32) *(float2*)p = make_float2(v[0], v[1]);
  else *(uint32_t*)p = pack2<DT>(v[0], v[1]);
}

// The largest of a column, of which a lane has m of its 4 rows in each tile.
__device__ __forceinline__ float column_max(float m) {
  const uint32_t b = __float_as_uint(m);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const uint32_t c = __float_as_uint(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
  const auto q = __builtin_amdgcn_permlane32_swap(c, c, false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// 16 bytes per lane from global memory straight into LDS: lane i's bytes land at l + 16 i.
__device__ __forceinline__ void copy_frag(const char* g, char* l) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) char*)g,
                                   (__attribute__((address_space(3))) void*)l, 16, 0, 0);
}

// A workgroup of W waves takes W * 16 NC rows of a head's state. The chunk's fragments
// come through LDS in two halves, K and Q (phase 1), and the rest (phase 2): the copies
// of the next chunk's half are on their way while the other half is used, with one
// barrier in between.
template <int DT, int N, int NC, int W>
__global__ __launch_bounds__(64 * W) void k_delta_scan(DeltaArgs a, const char* ws_keys, const char* ws_heads, int64_t L,
                                                     int H, int G, int hpg, int P, int chunks) {
  typedef KeyPlan<DT, N> KP_;
  typedef HeadPlan<DT> HP_;
  constexpr int KS = KP_::KS, NT = KP_::NT, KP = KP_::KP, AP = Parts<DT>::kWeights;
  constexpr int SY = Parts<DT>::kStateY, UY = Parts<DT>::kNewY;
  constexpr int kFirst = KP_::kT, kTurned = KP_::kFrags - KP_::kT;  // K and Q; K^T
  __shared__ __attribute__((aligned(1024))) char buf1[kFirst * kFrag];
  __shared__ __attribute__((aligned(1024))) char buf2[(kTurned + HP_::kFrags) * kFrag];
  const int lane = lane_id(), wv = wave_id(), sub = lane >> 4, col = lane & 15;
  const int slices = P / (16 * NC * W);
  const int64_t unit = blockIdx.x / slices, b = unit / H;
  const int h = (int)(unit % H), g = h / hpg;
  const int p0 = ((int)(blockIdx.x % slices) * W + wv) * 16 * NC + NC * col;  // the lane's columns: p0 .. p0 + NC - 1
  const char* keys = ws_keys + (b * G + g) * (int64_t)chunks * KP_::kBytes + lane * 16;
  const char* head = ws_heads + unit * (int64_t)chunks * HP_::kBytes + lane * 16;

  auto copy1 = [&](const char* k) {
#pragma unroll
    for (int f = 0; f < kFirst; f += W)
      if (kFirst % W == 0 || f + wv < kFirst) copy_frag(k + (f + wv) * kFrag, buf1 + (f + wv) * kFrag);
  };
  auto copy2 = [&](const char* k, const char* hd) {
#pragma unroll
    for (int f = 0; f < kTurned; f += W)
      if (kTurned % W == 0 || f + wv < kTurned) copy_frag(k + (kFirst + f + wv) * kFrag, buf2 + (f + wv) * kFrag);
#pragma unroll
    for (int f = 0; f < HP_::kFrags; f += W)
      if (HP_::kFrags % W == 0 || f + wv < HP_::kFrags)
        copy_frag(hd + (f + wv) * kFrag, buf2 + (kTurned + f + wv) * kFrag);
  };
  // this wave's copies have arrived; behind the barrier all have, and what was read before it is free
  auto meet = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  auto key = [&](int f) { return *(const v8h*)(buf1 + f * kFrag + lane * 16); };
  auto turned = [&](int f) { return *(const v8h*)(buf2 + f * kFrag + lane * 16); };
  auto weight = [&](int f) { return *(const v8h*)(buf2 + (kTurned + f) * kFrag + lane * 16); };
  const float* const fac = (const float*)(buf2 + (kTurned + HP_::kFac) * kFrag);

  copy1(keys);
  copy2(keys, head);
  // Rows of X and Y: a uniform address for each of a chunk's, and the lane's place in
  // it (64 rows are less than 2^32 bytes). Behind the end of the sequence the last row
  // stands in: what it meets in T is zero.
  constexpr int kE = sizeof(typename Store<DT>::T);
  const uint32_t step = (uint32_t)H * P * kE, place = 4 * sub * step + p0 * kE;
  const char* x_at = (const char*)a.X + (b * L * H + h) * P * kE;
  char* y_at = (char*)a.Y + (b * L * H + h) * P * kE;
  float v[4][4][NC];
  auto load_values = [&](int n) {
    if (n >= kC) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) load_cols<DT, NC>(x_at + (uint64_t)(16 * i + e) * step + place, v[i][e]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          load_cols<DT, NC>(x_at + (min(16 * i + 4 * sub + e, n - 1) * step + p0 * kE), v[i][e]);
    }
    x_at += (uint64_t)kC * step;
  };
  load_values((int)min(L, (int64_t)kC));
  v4f s[NC][NT];
  // The state is held times a power of two, one for each of its rows: 1 / inv_s.
  float inv_s[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float m = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      s[c][n] = a.init ? *(const v4f*)(a.init + (unit * P + p0 + c) * (int64_t)N + 16 * n + 4 * sub) : (v4f)(0.f);
      m = fmaxf(m, max4(s[c][n]));
    }
    const Scale sc(column_max(m));
    inv_s[c] = sc.inv;
#pragma unroll
    for (int n = 0; n < NT; ++n) s[c][n] *= sc.by;
  }
  meet();

  float one = 1.f;  // not known to be it: x 1 - hi, rounded to fp16, is one operation
  asm volatile("" : "+v"(one));
  for (int ck = 0; ck < chunks; ++ck) {
    const bool more = ck + 1 < chunks;
    const int left = (int)min(L - (int64_t)ck * kC, (int64_t)kC);  // positions of this chunk
    keys += KP_::kBytes;
    head += HP_::kBytes;
    // phase 1: K S^T and Q S^T
    v4f ks[NC][4], qs[NC][4];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) ks[c][i] = qs[c][i] = (v4f)(0.f);
    }
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      v8h hi[NC], lo[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c)
        split_tiles(s[c][2 * t], 2 * t + 1 < NT ? s[c][2 * t + 1 < NT ? 2 * t + 1 : 0] : (v4f)(0.f), one, hi[c], lo[c]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const v8h k = key(KP_::kK + i * KS + t), q = key(KP_::kQ + i * KS + t);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          ks[c][i] = mma16(k, hi[c], ks[c][i]);
          qs[c][i] = mma16(q, hi[c], qs[c][i]);
          ks[c][i] = mma16(k, lo[c], ks[c][i]);
          if constexpr (SY == 2) qs[c][i] = mma16(q, lo[c], qs[c][i]);
          if constexpr (KP == 2) {
            ks[c][i] = mma16(key(KP_::kK + (4 + i) * KS + t), hi[c], ks[c][i]);
            qs[c][i] = mma16(key(KP_::kQ + (4 + i) * KS + t), hi[c], qs[c][i]);
          }
        }
      }
    }
    meet();
    if (more) copy1(keys);

    // phase 2: U = T diag(b) (V - e^g K S^T), times 1 / inv_u
    v4f u[NC][4];
    float inv_u[NC], max_u[NC];
    {
      float by[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const v4f f = *(const v4f*)(fac + kFacK + 16 * i + 4 * sub);
#pragma unroll
          for (int e = 0; e < 4; ++e) ks[c][i][e] = fmaf(-f[e] * inv_s[c], ks[c][i][e], v[i][e][c]);
          m = fmaxf(m, max4(ks[c][i]));
          u[c][i] = (v4f)(0.f);
        }
        const Scale sc(column_max(m));
        by[c] = sc.by;
        inv_u[c] = sc.inv * fac[kInvT];
      }
      if (more) load_values((int)min(L - (int64_t)(ck + 1) * kC, (int64_t)kC));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        v8h hi[NC], lo[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) split_tiles(ks[c][2 * t], ks[c][2 * t + 1], by[c], hi[c], lo[c]);
#pragma unroll
        for (int i = 2 * t; i < 4; ++i) {
          const v8h w = weight(HP_::kT + lower_frag(i, t)), wl = weight(HP_::kT + 6 + lower_frag(i, t));
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            u[c][i] = mma16(w, hi[c], u[c][i]);
            u[c][i] = mma16(w, lo[c], u[c][i]);
            u[c][i] = mma16(wl, hi[c], u[c][i]);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaxf(m, max4(u[c][i]));
        max_u[c] = column_max(m);
      }
    }
    // Y
    {
      v4f yd[NC][4];
      float by[NC], inv[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) yd[c][i] = (v4f)(0.f);
        const Scale sc(max_u[c]);
        by[c] = sc.by;
        inv[c] = sc.inv * inv_u[c] * fac[kInvA];
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        v8h hi[NC], lo[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) split_tiles(u[c][2 * t], u[c][2 * t + 1], by[c], hi[c], lo[c]);
#pragma unroll
        for (int i = 2 * t; i < 4; ++i) {
          const v8h w = weight(HP_::kA + lower_frag(i, t));
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            yd[c][i] = mma16(w, hi[c], yd[c][i]);
            if constexpr (UY == 2) yd[c][i] = mma16(w, lo[c], yd[c][i]);
            if constexpr (AP == 2) yd[c][i] = mma16(weight(HP_::kA + 6 + lower_frag(i, t)), hi[c], yd[c][i]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const v4f f = *(const v4f*)(fac + kFacQ + 16 * i + 4 * sub);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) yd[c][i][e] = fmaf(f[e] * inv_s[c], qs[c][i][e], yd[c][i][e] * inv[c]);
      }
      auto store = [&](int i, int e) {
        float y[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) y[c] = yd[c][i][e];
        store_cols<DT, NC>(y_at + (uint64_t)(16 * i + e) * step + place, y);
      };
      if (left >= kC) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) store(i, e);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * i + 4 * sub + e < left) store(i, e);
      }
      y_at += (uint64_t)kC * step;
    }
    // S' = e^{g_63} S + (e^{g_63 - g} U)^T K, the products added to the scaled state: its
    // largest value is brought to 2^8 and U's part to 2 at most, so that the sums (64
    // terms, keys up to 2^8) stay below 2^16 as fp16's range asks.
    {
      const float decay = fac[kDecay], most = fac[kMaxU] * 256.f;
      float by[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float m = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) m = fmaxf(m, max4(s[c][n]));
        const Scale sc(fmaxf(column_max(m) * inv_s[c] * decay, max_u[c] * inv_u[c] * most));
        const float keep = decay * (inv_s[c] * sc.by);
        by[c] = inv_u[c] * sc.by;
        inv_s[c] = sc.inv;
#pragma unroll
        for (int n = 0; n < NT; ++n) s[c][n] *= keep;
#pragma unroll
        for (int i = 0; i < 4; ++i) u[c][i] *= *(const v4f*)(fac + kFacU + 16 * i + 4 * sub);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        v8h hi[NC], lo[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) split_tiles(u[c][2 * t], u[c][2 * t + 1], by[c], hi[c], lo[c]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const v8h k = turned(2 * n + t);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            s[c][n] = mma16(k, hi[c], s[c][n]);
            s[c][n] = mma16(k, lo[c], s[c][n]);
            if constexpr (KP == 2) s[c][n] = mma16(turned(2 * NT + 2 * n + t), hi[c], s[c][n]);
          }
        }
      }
    }
    meet();
    if (more) copy2(keys, head);
  }
  if (a.final_state) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        *(v4f*)(a.final_state + (unit * P + p0 + c) * (int64_t)N + 16 * n + 4 * sub) = s[c][n] * inv_s[c];
  }
}

template <int DT, int N, int NC, int W>
hipError_t scan(const Dims& d, const DeltaArgs& a, const char* keys, const char* heads, hipStream_t st) {
  const int64_t wgs = d.B * d.H * (d.P / (16 * NC * W));
  hipLaunchKernelGGL((k_delta_scan<DT, N, NC, W>), dim3((unsigned)wgs), dim3(64 * W), 0, st, a, keys, heads, d.L, d.H,
                     d.G, d.hpg, d.P, d.c);
  return hipGetLastError();
}

// Four waves of 16 rows each where the head has them (us at 4, 2 and 1 waves: 8 x 2048
// positions of 80 heads of 64 x 128, 16 bits, 594, 1403 and 2311 before later steps; one
// sequence of 2048, 64 heads, 192, 214 and 246). Waves of 32 rows read LDS half as
// often, but leave each SIMD one wave: 439 us with 16, 559 with 32.
template <int DT, int N>
hipError_t pick_scan(const Dims& d, const DeltaArgs& a, const char* keys, const char* heads, hipStream_t st) {
  switch (d.P) {
    case 16: return scan<DT, N, 1, 1>(d, a, keys, heads, st);
    case 32: return scan<DT, N, 1, 2>(d, a, keys, heads, st);
    default: return scan<DT, N, 1, 4>(d, a, keys, heads, st);
  }
}

template <int DT, int N>
hipError_t go(const Dims& d, const DeltaArgs& a, char* ws, hipStream_t st) {
  char* const heads = ws + d.B * d.G * (int64_t)d.c * KeyPlan<DT, N>::kBytes;
  const int64_t ncu = cu_count() > 0 ? cu_count() : 256;
  // heads of a group that a workgroup takes: four, or more where that leaves
  // workgroups enough
  const int64_t groups = d.B * d.c * d.G;
  int per = 4;
  while (per < d.hpg && groups * ((d.hpg + 2 * per - 1) / (2 * per)) >= 8 * ncu) per *= 2;
  const int blocks = (d.hpg + per - 1) / per;
  const int64_t total = groups * blocks;
  hipLaunchKernelGGL((k_delta_prepare<DT, N>), dim3((unsigned)min(total, (int64_t)1 << 20)), dim3(256), 0, st, a, ws,
                     heads, d.L, d.H, d.G, d.hpg, d.c, blocks, per, total);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return pick_scan<DT, N>(d, a, ws, heads, st);
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
