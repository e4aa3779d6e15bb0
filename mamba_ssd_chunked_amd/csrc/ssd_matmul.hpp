// The matrix products' way through their operands (k_matmul_i8.hip, k_matmul.hip):
//   sum_k a[m,k] w[n,k]
// for rows of bytes, whatever their elements are: all types' matrix instructions take
// 16 bytes of a row from each lane. An Op says which:
//   Acc32, mma32   32 x 32 results of 32 bytes of the rows
//   Acc16, mma16   16 x 16 results of 64 bytes of the rows
// Rows are 16-byte aligned and a multiple of 16 bytes long; what results become is the
// caller's.
#pragma once

#include <type_traits>

#include "ssd_device.hpp"

namespace ssd {
namespace {

typedef int v16i __attribute__((ext_vector_type(16)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t v4u_any __attribute__((ext_vector_type(4), aligned(2)));  // at any 16-bit element's address
typedef uint32_t v2u_any __attribute__((ext_vector_type(2), aligned(2)));
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));

// 16 bytes per lane from global memory straight into LDS: lane i's bytes land
// at l + 16 i (l is uniform over the wave).
typedef const __attribute__((address_space(1))) int8_t* global_ptr;
__device__ __forceinline__ void copy16_to_lds(global_ptr g, void* l) {
  __builtin_amdgcn_global_load_lds(g, (__attribute__((address_space(3))) void*)l, 16, 0, 0);
}

// Waits until at most N of this wave's copies (of its newest memory operations)
// are still on their way.
template <int N>
__device__ __forceinline__ void wait_copies() {
  __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
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
// A workgroup of NW waves computes a square tile of 32 NW rows and columns; a
// wave 16 NW columns (n) of 64 rows (m).
constexpr int kBK = 128;
template <int NW>
struct Tile {
  static constexpr int kSide = 32 * NW, kBytesA = kSide * kBK, kBytes = 2 * kBytesA;
  static constexpr int TI = NW / 2;  // 32 x 32 blocks of a wave in n; 2 in m
};
// S steps are in LDS at a time. Three steps ahead (S = 4) a step's copies are
// issued in quarters among products, which is 5 % faster; one step ahead the
// copies' latency is what counts, and at once is 5 % faster.
template <int S>
constexpr bool kSpread = S > 2;
constexpr int kStage = 32 * 128;  // a wave's part of the epilogue's staging: 32 rows of 128 bytes

// The rows of both operands this lane copies, and their LDS homes. A tile row
// is 128 bytes, eight 16-byte chunks; two rows cover the 64 banks. Chunk c of
// row r sits at slot c ^ (r / 2 % 8), so that the fragment reads of 16
// consecutive rows meet every bank once. The copy fills LDS in lane order, so
// the lane that owns slot s of row r fetches chunk s ^ (r / 2 % 8). TAIL: the
// rows are not a whole number of steps long; chunks behind their end are zeros.
// SAME: the rows of both operands are K bytes apart.
template <int NW, bool TAIL, bool SAME>
struct TileCopy {
  unsigned o[4], oa[SAME ? 1 : 4];  // byte offsets of the lane's chunks in the tile's rows of w (and a), of a
  __device__ __forceinline__ int chunk(int i) const {
    return ((lane_id() & 7) ^ (lane_id() >> 4)) * 16 ^ ((i & 1) * 64);
  }
  __device__ __forceinline__ void init(unsigned K, unsigned lda) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned row = (wave_id() * 4 + i) * 8 + (lane_id() >> 3);
      o[i] = row * K + chunk(i);
      if constexpr (!SAME) oa[i] = row * lda + chunk(i);
    }
  }
};

// Where a step's rows come from: byte k of the rows at a and w.
struct TileFrom {
  const int8_t *a, *w;
  int k;
};

// A quarter of a wave's copies of a step.
template <int NW, bool TAIL, bool SAME>
__device__ __forceinline__ void copy_quarter(const TileCopy<NW, TAIL, SAME>& cp, int i, const TileFrom& s, int K, int8_t* buf) {
  int8_t* const la = buf + wave_id() * 4096 + i * 1024;
  const global_ptr pa = (global_ptr)uniform_ptr(s.a + s.k);
  const global_ptr pw = (global_ptr)uniform_ptr(s.w + s.k);
  // opaque here, so that the address stays a scalar base and a 32-bit offset
  // (widened ahead of the loop it would be a 64-bit sum in every lane)
  unsigned o = cp.o[i];
  asm volatile("" : "+v"(o));
  unsigned oa = o;
  if constexpr (!SAME) {
    oa = cp.oa[i];
    asm volatile("" : "+v"(oa));
  }
  if constexpr (TAIL) {
    const bool in = s.k + cp.chunk(i) < K;
    const global_ptr zero = (global_ptr)(const int8_t*)&kZero16;
    copy16_to_lds(in ? pa + oa : zero, la);
    copy16_to_lds(in ? pw + o : zero, la + Tile<NW>::kBytesA);
  } else {
    copy16_to_lds(pa + oa, la);
    copy16_to_lds(pw + o, la + Tile<NW>::kBytesA);
  }
}
template <int NW, bool TAIL, bool SAME>
__device__ __forceinline__ void copy_step(const TileCopy<NW, TAIL, SAME>& cp, const TileFrom& s, int K, int8_t* buf) {
#pragma unroll
  for (int i = 0; i < 4; ++i) copy_quarter<NW, TAIL, SAME>(cp, i, s, K, buf);
}

// The operands of one 32-byte step of a wave's block.
template <class Op, int NW>
struct TileFrags {
  static constexpr int TI = Tile<NW>::TI;
  v4i w[TI], a[2];
  __device__ __forceinline__ void load(const int8_t* buf, int ks, int wm, int wn) {
    const int lane = lane_id(), slot = ((ks * 2 + (lane >> 5)) ^ ((lane >> 1) & 7)) * 16;
#pragma unroll
    for (int j = 0; j < 2; ++j) a[j] = *(const v4i*)(buf + (wm + 32 * j + (lane & 31)) * kBK + slot);
#pragma unroll
    for (int i = 0; i < TI; ++i) w[i] = *(const v4i*)(buf + Tile<NW>::kBytesA + (wn + 32 * i + (lane & 31)) * kBK + slot);
  }
  __device__ __forceinline__ void multiply(typename Op::Acc32 (&acc)[TI][2]) const {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = Op::mma32(w[i], a[j], acc[i][j]);
  }
};

// One 128-byte step from `cur`, whose first operands are in f[0]. The operands
// of each 32-byte step are read while the products of the one before run. The
// last products run behind the barrier, and cover what follows it: the first
// reads of `nxt`, whose copies the barrier has seen arrive. `cur` is then free,
// and takes the copies of the step `sn`: all at once, or (kSpread) a quarter at
// once and the others among the next step's products (here: the rest of `sp`'s
// into `prv`), so that no wave stands in front of a full memory pipe with
// products to issue.
template <class Op, int NW, int S, bool TAIL, bool SAME>
__device__ __forceinline__ void tile_step(int8_t* prv, const TileFrom& sp, int8_t* cur, const TileFrom& sn,
                                          const int8_t* nxt, const TileCopy<NW, TAIL, SAME>& cp, int K, int wm, int wn,
                                          TileFrags<Op, NW> (&f)[2], typename Op::Acc32 (&acc)[Tile<NW>::TI][2]) {
  constexpr int TI = Tile<NW>::TI;
#pragma unroll
  for (int ks = 0; ks < 3; ++ks) {
    f[(ks + 1) & 1].load(cur, ks + 1, wm, wn);
    if constexpr (kSpread<S>) copy_quarter<NW, TAIL, SAME>(cp, ks + 1, sp, K, prv);
    f[ks & 1].multiply(acc);
#pragma unroll
    for (int q = 0; q < TI + 2; ++q) {  // a read, a product, ...
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, Op::kInstructions, 0);
      if (kSpread<S> && (q == 1 || q == 3)) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
    if constexpr (TI > 2) __builtin_amdgcn_sched_group_barrier(0x008, Op::kInstructions * (TI - 2), 0);
  }
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  // This wave's copies into nxt have arrived (only those of the steps behind it,
  // 8 each, may still be on their way), its reads of cur have too (lgkmcnt 0).
  constexpr int kBehind = 8 * (S - 2);
  __builtin_amdgcn_s_waitcnt(0x0070 | (kBehind & 15) | ((kBehind >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  f[0].load(nxt, 0, wm, wn);
  if constexpr (kSpread<S>) copy_quarter<NW, TAIL, SAME>(cp, 0, sn, K, cur);
  else copy_step<NW, TAIL, SAME>(cp, sn, K, cur);
  f[1].multiply(acc);
  __builtin_amdgcn_sched_barrier(0);
}

// Workgroups on a CU: their LDS (S steps and the stages) fills the 160 KB.
template <int NW, int S>
constexpr int kTileWgs = (160 * 1024) / (S * Tile<NW>::kBytes + NW * kStage);

// As many workgroups as fit the chip's LDS walk the tiles; the copies of the
// next tile's first steps run under the epilogue of this one's.
// g: M, N, a, w; rows of K bytes, a's lda bytes apart. store(m0, n0, mb, nb, wm, wn, stage,
// acc) takes the results of rows m0 + wm + (0..63), columns n0 + wn + (0 .. 32 TI - 1), of
// which those before row mb or column nb are other tiles' too.
template <class Op, bool TAIL, bool SAME, int NW, int S, class Args, class Store_>
__device__ __forceinline__ void tile_walk(const Args& g, int K, int64_t lda, int tiles_m, int tiles_n, Store_ store) {
  constexpr int kSide = Tile<NW>::kSide, TI = Tile<NW>::TI;
  // separate objects, so that the compiler sees that a read of one need not
  // wait for the copies into another
  __shared__ __attribute__((aligned(1024))) int8_t buf0[Tile<NW>::kBytes], buf1[Tile<NW>::kBytes];
  __shared__ __attribute__((aligned(1024))) int8_t buf2[S > 2 ? Tile<NW>::kBytes : 16];
  __shared__ __attribute__((aligned(1024))) int8_t buf3[S > 2 ? Tile<NW>::kBytes : 16];
  __shared__ __attribute__((aligned(1024))) int8_t stage[NW * kStage];
  // Consecutive workgroups go to the eight XCDs in turn. Each XCD takes a
  // contiguous run of the tiles, which its workgroups walk together, in columns
  // of four row tiles: the tiles that an XCD computes at a time share rows in
  // its L2.
  const int tiles = tiles_m * tiles_n;
  const int xcd = blockIdx.x % 8, nwg = (gridDim.x - xcd + 7) / 8;
  const int lo = xcd * (tiles / 8) + min(xcd, tiles % 8), hi = lo + tiles / 8 + (xcd < tiles % 8);
  int t = lo + blockIdx.x / 8;
  if (t >= hi) return;
  auto place = [&](int t, int& m0, int& n0, int& mb, int& nb) {
    const int group = t / (4 * tiles_n), rows = min(4, tiles_m - group * 4), in = t - group * 4 * tiles_n;
    mb = (group * 4 + in % rows) * kSide;
    nb = (in / rows) * kSide;
    // the last tiles end with the matrix: what they share with the tiles before
    // may be written twice, with the same bits
    m0 = min(mb, (int)g.M - kSide);
    n0 = min(nb, (int)g.N - kSide);
  };
  int m0, n0, mb, nb;
  place(t, m0, n0, mb, nb);
  const int wv = wave_id(), wm = (wv % (NW / 2)) * 64, wn = (wv / (NW / 2)) * 32 * TI;
  TileCopy<NW, TAIL, SAME> cp;
  cp.init((unsigned)K, (unsigned)lda);
  auto from = [&](int m, int n, int k) { return TileFrom{(const int8_t*)g.a + (int64_t)m * lda, (const int8_t*)g.w + (int64_t)n * K, k}; };
  TileFrom here = from(m0, n0, 0), last = here;  // last: the newest step under way
  copy_step<NW, TAIL, SAME>(cp, here, K, buf0);
  __builtin_amdgcn_s_waitcnt(0x0f70);
  __syncthreads();
  last.k = (S - 1) * kBK;
  if constexpr (S > 2) {
    here.k = kBK;
    copy_step<NW, TAIL, SAME>(cp, here, K, buf1);
    here.k = 2 * kBK;
    copy_step<NW, TAIL, SAME>(cp, here, K, buf2);
    copy_quarter<NW, TAIL, SAME>(cp, 0, last, K, buf3);
  } else {
    copy_step<NW, TAIL, SAME>(cp, last, K, buf1);
  }
  TileFrags<Op, NW> f[2];
  f[0].load(buf0, 0, wm, wn);
  for (;;) {
    const int tn = t + nwg;
    int m1 = m0, n1 = n0, mb1 = mb, nb1 = nb;
    if (tn < hi) place(tn, m1, n1, mb1, nb1);
    typename Op::Acc32 acc[TI][2];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = (typename Op::Acc32)(0);
    // a round of all buffers at a time; where the rows end inside a round its
    // rest is zeros (TAIL)
    for (int k = 0; k < K; k += S * kBK) {
      TileFrom s{here.a, here.w, k + S * kBK};
      // the next tile's first steps (the last tile's once more: read by nobody)
      if (s.k >= K) s = here = from(m1, n1, 0);
      if constexpr (S > 2) {
        tile_step<Op, NW, S, TAIL, SAME>(buf3, last, buf0, s, buf1, cp, K, wm, wn, f, acc);
        const TileFrom s1{s.a, s.w, s.k + kBK}, s2{s.a, s.w, s.k + 2 * kBK};
        tile_step<Op, NW, S, TAIL, SAME>(buf0, s, buf1, s1, buf2, cp, K, wm, wn, f, acc);
        tile_step<Op, NW, S, TAIL, SAME>(buf1, s1, buf2, s2, buf3, cp, K, wm, wn, f, acc);
        last = TileFrom{s.a, s.w, s.k + 3 * kBK};
        tile_step<Op, NW, S, TAIL, SAME>(buf2, s2, buf3, last, buf0, cp, K, wm, wn, f, acc);
      } else {
        tile_step<Op, NW, S, TAIL, SAME>(buf1, last, buf0, s, buf1, cp, K, wm, wn, f, acc);
        last = TileFrom{s.a, s.w, s.k + kBK};
        tile_step<Op, NW, S, TAIL, SAME>(buf0, s, buf1, last, buf0, cp, K, wm, wn, f, acc);
      }
    }
    store(m0, n0, mb, nb, wm, wn, stage + wv * kStage, acc);
    if (tn >= hi) break;
    t = tn;
    m0 = m1;
    n0 = n1;
    mb = mb1;
    nb = nb1;
  }
  // no copy may still be on its way when the workgroup's LDS goes to another
  __builtin_amdgcn_s_waitcnt(0x0f70);
}

// Four consecutive outputs, of which n are inside the matrix.
template <int DT>
__device__ __forceinline__ void store4(void* out, int64_t at, const float (&y)[4], int n) {
  typename Store<DT>::T* const o = (typename Store<DT>::T*)out + at;
  if (n >= 4) {
    if constexpr (DT == DT_F32) *(v4f_any*)o = (v4f_any){y[0], y[1], y[2], y[3]};
    else *(v2u_any*)o = (v2u_any){pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3])};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) o[e] = to_store<DT>(y[e]);
  }
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------
// A workgroup of NW waves computes 16 NT columns (n) of 16 MT rows (m). The
// waves split the sum: each takes every NW-th 128 bytes of the rows, which it
// copies into its own part of LDS, D pieces ahead of their use and without a
// barrier, and the partial sums meet in LDS: one launch is all. The copies take
// whole 128-byte lines of eight rows at a time. (Operands loaded straight into
// registers are 64 bytes of sixteen rows in each load, at which a CU took in
// 41 GB/s instead of the copies' 107.)
//
// finish(m, n, sum) takes the sums of columns n .. n + 3 (of which the last may lie
// behind the matrix) of row m.
template <class Op, int MT, int NT, int NW, int D, class Args, class Finish>
__device__ __forceinline__ void few_rows(const Args& g, int K, int64_t lda, int blocks_m, Finish finish) {
  typedef typename Op::Acc16 Acc;
  constexpr int kPiece = (MT + NT) * 2048;  // a wave's rows of 128 bytes, W's first
  constexpr int kCopies = 2 * (MT + NT);    // instructions of a piece
  static_assert(D >= 2 && D <= 4 && NW * MT * NT * 1024 <= NW * kPiece * D, "LDS");
  // separate objects: see the tiles
  __shared__ __attribute__((aligned(1024))) int8_t buf0[NW * kPiece], buf1[NW * kPiece];
  __shared__ __attribute__((aligned(1024))) int8_t buf2[D > 2 ? NW * kPiece : 16], buf3[D > 3 ? NW * kPiece : 16];
  const int lane = lane_id(), wv = wave_id();
  // Each XCD takes a contiguous run of the blocks, the blocks of a column next to
  // each other: they read the same weights, which the XCD's L2 then fetches once.
  const int xcd = blockIdx.x % 8, per = (int)gridDim.x / 8, more = (int)gridDim.x % 8;
  const int t = xcd * per + min(xcd, more) + (int)blockIdx.x / 8;
  const int n0 = t / blocks_m * 16 * NT, m0 = t % blocks_m * 16 * MT;
  int8_t* const slot[4] = {buf0 + wv * kPiece, buf1 + wv * kPiece, D > 2 ? buf2 + wv * kPiece : nullptr,
                           D > 3 ? buf3 + wv * kPiece : nullptr};
  const global_ptr bw = (global_ptr)uniform_ptr((const int8_t*)g.w + (int64_t)n0 * K);
  const global_ptr ba = (global_ptr)uniform_ptr((const int8_t*)g.a + (int64_t)m0 * lda);
  // Rows past the edge stand in with the last one; their results are not stored.
  // Chunk c of row r sits at slot c ^ (r / 2 % 8), as in the tiles.
  const int rw = min((int)g.N - n0, 16 * NT), ra = min((int)g.M - m0, 16 * MT);
  auto chunk = [&](int i) { return ((lane & 7) ^ (lane >> 4)) * 16 ^ ((i & 1) * 64); };
  unsigned ow[2 * NT], oa[2 * MT];
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) ow[i] = (unsigned)min(8 * i + (lane >> 3), rw - 1) * (unsigned)K + chunk(i);
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) oa[i] = (unsigned)min(8 * i + (lane >> 3), ra - 1) * (unsigned)lda + chunk(i);
  const global_ptr zero = (global_ptr)(const int8_t*)&kZero16;
  auto copy = [&](int piece, int8_t* to) {
    const int k = (piece * NW + wv) * 128;
    // chunks behind the end of the rows are zeros
    const bool in0 = k + chunk(0) < K, in1 = k + chunk(1) < K;
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) copy16_to_lds(((i & 1) ? in1 : in0) ? bw + (ow[i] + k) : zero, to + i * 1024);
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i)
      copy16_to_lds(((i & 1) ? in1 : in0) ? ba + (oa[i] + k) : zero, to + (2 * NT + i) * 1024);
  };
  Acc acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = (Acc)(0);
  v4i fw[2][NT], fa[2][MT];
  auto read = [&](const int8_t* from) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int8_t* const p = from + (lane & 15) * 128 + ((s * 4 + (lane >> 4)) ^ ((lane >> 1) & 7)) * 16;
#pragma unroll
      for (int i = 0; i < NT; ++i) fw[s][i] = *(const v4i*)(p + i * 2048);
#pragma unroll
      for (int j = 0; j < MT; ++j) fa[s][j] = *(const v4i*)(p + (NT + j) * 2048);
    }
  };
  auto multiply = [&]() {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i][j] = Op::mma16(fw[s][i], fa[s][j], acc[i][j]);
  };
  // a wave's pieces; the last may lie behind the rows' end, as zeros
  const int pieces = (K + NW * 128 - 1) / (NW * 128);
  // takes a piece out of its slot, and once its reads are done the slot is free
  auto take = [&](const int8_t* from) {
    asm volatile("" ::: "memory");
    read(from);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
  };
#pragma unroll
  for (int d = 0; d < D; ++d) copy(d, slot[d]);  // behind the last piece: zeros
  int p = 0;
  for (; p + 2 * D <= pieces; p += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      wait_copies<(D - 1) * kCopies>();
      take(slot[d]);
      copy(p + D + d, slot[d]);
      multiply();
    }
  }
  // the last D to 2 D - 1 pieces: each wait allows for the copies known to be younger
  auto last = [&](auto dc) {
    constexpr int d = decltype(dc)::value;
    wait_copies<(D - 1 - d) * kCopies>();
    take(slot[d]);
    if (d < D - 1 && p + D + d < pieces) copy(p + D + d, slot[d]);
    multiply();
  };
  last(std::integral_constant<int, 0>());
  last(std::integral_constant<int, 1>());
  if constexpr (D > 2) last(std::integral_constant<int, 2>());
  if constexpr (D > 3) last(std::integral_constant<int, 3>());
#pragma unroll
  for (int d = 0; d < D - 1; ++d)
    if (p + D + d < pieces) {
      wait_copies<0>();
      take(slot[d]);
      multiply();
    }
  __syncthreads();

  Acc* const part = (Acc*)buf0;  // [wave][block][lane]
  static_assert(NW * MT * NT * 1024 <= NW * kPiece, "the partial sums fit the first buffer");
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) part[(wv * MT * NT + i * MT + j) * kWave + lane] = acc[i][j];
  __syncthreads();
  for (int b = wv; b < MT * NT; b += NW) {
    const int m = m0 + 16 * (b % MT) + (lane & 15), n = n0 + 16 * (b / MT) + (lane >> 4) * 4;
    if (m >= g.M || n >= g.N) continue;
    Acc sum = part[b * kWave + lane];
#pragma unroll
    for (int v = 1; v < NW; ++v) sum += part[(v * MT * NT + b) * kWave + lane];
    finish(m, n, sum);
  }
}

}  // namespace
}  // namespace ssd
