// Causal depthwise convolution, SiLU and softplus between In Proj and the SSD:
//
//   u_t[c] = sum_{j<W} w[c,j] xbc_{t-W+1+j}[c] + b[c],   x | B | C = u / (1 + exp(-u))
//   dt_t[h] = softplus(dt_raw_t[h] + dt_bias[h])
//
// The work is one read of x | B | C and one write: memory bound. A thread owns
// 16 bytes of channels and walks T positions down the sequence with the last
// W - 1 inputs in registers, so every input is read once but for W - 1 rows at
// the head of each tile. Those come from memory once more (the counters read 196 MB
// for 179): the tile before mostly runs on another XCD, behind another L2.
// Rows are loaded a set of kU ahead of their use (sets of 2 and 8 are slower by 6
// and 15 %, tiles of 16 positions instead of 32 by 8 %), and written past the
// caches: 3 to 20 % faster alone. With the SSD that reads them next, as much is lost
// again in the middle (us, and with ordinary stores, 80 heads of 64 x 128 fp16, the
// convolution and the float forward: 1 x 256 22.8, 22.4; 4 x 1024 102, 97; 8 x 2048
// 307, 301; INT8 246, 243). Rows behind a sequence's end are read and computed like
// the others before they are written as zeros: a ragged batch costs what a full one
// does. 8 x 2048 x 5376 channels in fp16: 79 us, 4.5 TB/s of its 358 MB; three
// waves on each SIMD hold 160 registers each (weights 40, window 24, sets 32),
// and a fourth, with 128, spills (193 us). The blocks behind those of the
// convolution compute dt.
//
// The ring of the last W inputs is written by the thread that computes its
// channels' first tile: it alone reads the history, and it reads it first.
#include "ssd_conv.hpp"
#include "ssd_launch.hpp"

namespace ssd {
namespace {

constexpr int kConvThreads = 256;
constexpr int kU = 4;  // rows of a set

struct ConvFwdArgs {
  ConvPtrs cv;
  const int32_t* lengths;
  void* X;
  void* Bo;
  void* Co;
  void* dt;
  int64_t B, L;
  int H, dX, dBC, Cd;  // heads, H*P, G*N, all channels
  int nvec;            // vectors of a row
  int T, ntiles;
  unsigned conv_blocks;
  int dt_rows;  // rows of one dt block
};

template <int DT, int W, bool AL>
__device__ __forceinline__ void conv_tile(const ConvFwdArgs& a, unsigned id) {
  constexpr int V = RawVec<DT>::V;
  const unsigned vec = id % (unsigned)a.nvec, rest = id / (unsigned)a.nvec;
  const int tile = (int)(rest % (unsigned)a.ntiles);
  const int64_t b = rest / (unsigned)a.ntiles;
  if (b >= a.B) return;
  const int c = (int)vec * V;
  const int64_t t0 = (int64_t)tile * a.T;
  const int64_t t1 = min(t0 + a.T, a.L);
  int64_t end = a.L;
  if (a.lengths) end = min(max((int64_t)a.lengths[b], (int64_t)0), a.L);
  const int64_t row0 = b * a.L;
  const int64_t ld = a.cv.ld_xbc;

  // the destination of this vector: x, B and C are multiples of 16 channels wide
  typedef typename Store<DT>::T T;
  T* dst;
  unsigned ldo;
  if (c < a.dX) {
    dst = (T*)a.X + c;
    ldo = a.dX;
  } else if (c < a.dX + a.dBC) {
    dst = (T*)a.Bo + (c - a.dX);
    ldo = a.dBC;
  } else {
    dst = (T*)a.Co + (c - a.dX - a.dBC);
    ldo = a.dBC;
  }
  // rows are counted from the tile's first: their offsets are one 32 x 32-bit product
  dst += (row0 + t0) * ldo;
  const T* const src = (const T*)a.cv.xbc + (row0 + t0) * ld + c;
  const int rows = (int)(t1 - t0), live = (int)min(max(end - t0, (int64_t)0), (int64_t)rows);

  float w[V][W], bias[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[e][j] = a.cv.weight[(int64_t)(c + e) * W + j];
    bias[e] = a.cv.bias ? a.cv.bias[c + e] : 0.f;
  }

  // the W - 1 inputs before the tile
  float win[W - 1][V];
  const uint32_t p0 = a.cv.pos ? (uint32_t)max(a.cv.pos[b], 0) : 0u;
  void* const ring = a.cv.state;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int back = W - 1 - j;
    RawVec<DT> v;
    v.zero();
    if (t0 >= back) {
      v.template load<AL>(a.cv.xbc, (row0 + t0 - back) * ld + c);
    } else if (p0 + (uint32_t)t0 >= (uint32_t)back) {  // only where pos is given: the ring is too
      const uint32_t slot = (p0 + (uint32_t)t0 - (uint32_t)back) % W;
      v.template load<true>(ring, (b * W + slot) * (int64_t)a.Cd + c);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) win[j][e] = v.get(e);
  }

  auto load_rows = [&](int r, RawVec<DT>* v) {
#pragma unroll
    for (int i = 0; i < kU; ++i)  // behind the tile: its last row again
      v[i].template load<AL>(src + (uint64_t)(unsigned)min(r + i, rows - 1) * (unsigned)ld, 0);
  };
  auto step = [&](const RawVec<DT>& v, int r) {
    float y[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float x = v.get(e);
      float u = bias[e];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) u = fmaf(w[e][j], win[j][e], u);
      u = fmaf(w[e][W - 1], x, u);
      y[e] = silu_rows<DT>(u);
#pragma unroll
      for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
      win[W - 2][e] = x;
    }
    RawVec<DT> out;
    out.set(y);
    if (r >= live) out.zero();
    out.template store_nt<true>(dst + (uint64_t)(unsigned)r * ldo, 0);
  };
  // two sets of kU rows by turns; no access of the loop is conditional, so that
  // a set's wait leaves the other's loads and the stores on their way
  RawVec<DT> va[kU], vb[kU];
  load_rows(0, va);
  int r = 0;
  for (; r + 2 * kU <= rows; r += 2 * kU) {
    load_rows(r + kU, vb);
#pragma unroll
    for (int i = 0; i < kU; ++i) step(va[i], r + i);
    load_rows(r + 2 * kU, va);
#pragma unroll
    for (int i = 0; i < kU; ++i) step(vb[i], r + kU + i);
  }
  if (r < rows) {  // rows behind the last one are skipped (2 to 5 % of a short prompt's time)
    if (r + kU < rows) load_rows(r + kU, vb);
#pragma unroll
    for (int i = 0; i < kU; ++i)
      if (r + i < rows) step(va[i], r + i);
    if (r + kU < rows) {
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if (r + kU + i < rows) step(vb[i], r + kU + i);
    }
  }

  if (tile == 0 && ring) {
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const int64_t t = end - W + j;
      if (t >= 0) {
        RawVec<DT> v;
        v.template load<AL>(a.cv.xbc, (row0 + t) * ld + c);
        v.store(ring, (b * W + (uint32_t)(p0 + (uint32_t)t) % W) * (int64_t)a.Cd + c);
      }
    }
  }
}

template <int DT, int W, bool AL>
__global__ __launch_bounds__(kConvThreads) void k_conv(ConvFwdArgs a) {
  typedef typename Store<DT>::T T;
  if (blockIdx.x < a.conv_blocks) {
    conv_tile<DT, W, AL>(a, blockIdx.x * kConvThreads + threadIdx.x);
    return;
  }
  const int64_t r0 = (int64_t)(blockIdx.x - a.conv_blocks) * a.dt_rows;
  const int n = (int)min((int64_t)a.dt_rows, a.B * a.L - r0) * a.H;
  for (int i = threadIdx.x; i < n; i += kConvThreads) {
    const int64_t row = r0 + (unsigned)i / (unsigned)a.H;
    const int h = (int)((unsigned)i % (unsigned)a.H);
    float v = softplus(ld_f<DT>(a.cv.dt_raw, row * a.cv.ld_dt + h) + (a.cv.dt_bias ? a.cv.dt_bias[h] : 0.f));
    if (a.lengths) {
      const int64_t b = row / a.L;
      if (row - b * a.L >= a.lengths[b]) v = 0.f;
    }
    ((T*)a.dt)[row * a.H + h] = to_store<DT>(v);
  }
}

template <int DT, int W>
hipError_t launch_w(const ConvFwdArgs& a, bool al, unsigned blocks, hipStream_t st) {
  if (al)
    hipLaunchKernelGGL((k_conv<DT, W, true>), dim3(blocks), dim3(kConvThreads), 0, st, a);
  else
    hipLaunchKernelGGL((k_conv<DT, W, false>), dim3(blocks), dim3(kConvThreads), 0, st, a);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const ConvFwdArgs& a, bool al, unsigned blocks, hipStream_t st) {
  switch (a.cv.width) {
    case 2: return launch_w<DT, 2>(a, al, blocks, st);
    case 3: return launch_w<DT, 3>(a, al, blocks, st);
    case 4: return launch_w<DT, 4>(a, al, blocks, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_conv_forward(const Dims& d, int dtype, const ConvPtrs& cv, const int32_t* lengths,
                               void* X, void* B, void* C, void* dt, hipStream_t st) {
  ConvFwdArgs a{};
  a.cv = cv;
  a.lengths = lengths;
  a.X = X; a.Bo = B; a.Co = C; a.dt = dt;
  a.B = d.B; a.L = d.L;
  a.H = d.H;
  a.dX = d.H * d.P;
  a.dBC = d.G * d.N;
  a.Cd = a.dX + 2 * a.dBC;
  const int esize = dtype == DT_F32 ? 4 : 2;
  a.nvec = a.Cd / (16 / esize);
  // Positions per thread: long tiles spread the weights' loads and the window's
  // head over more rows, short ones give every CU something to do. Three waves on
  // each CU are enough, as a wave has 8 rows under way (16-bit types, us at 1, 2,
  // 3, 4 and 16 waves: 4 x 791 x 1552 channels 15.8, 12.1, 12.5, 12.4, 14.1;
  // 3 x 701 x 10240 22 and, at 16, 27; 5 x 2954 x 1024, at 4 and 16, 16 and 24).
  // Never below kU, the rows of a set.
  const int64_t want = (int64_t)(cu_count() > 0 ? cu_count() : 256) * 3 * kWave;
  int64_t T = kU;
  while (T < 32 && d.B * ((d.L + 2 * T - 1) / (2 * T)) * a.nvec >= want) T *= 2;
  // 64 where that takes less time in rounds of 12 waves a CU, at T + 6 rows each
  // (us at 32 and 64: 4 x 4096 x 10240 161, 148; 1 x 9000 x 6912 60, 56; but 8 x
  // 4000 x 3328, 2 rounds of 64 with an almost empty second one, 99, 103)
  auto rounds = [&](int64_t t) { return (d.B * ((d.L + t - 1) / t) * a.nvec + 4 * want - 1) / (4 * want); };
  if (T == 32 && rounds(64) * 70 < rounds(32) * 38) T = 64;
  // thread indexes fit 31 bits
  while (d.B * ((d.L + T - 1) / T) * a.nvec >= (int64_t)1 << 31 && T < d.L) T *= 2;
  a.T = (int)T;
  a.ntiles = (int)((d.L + T - 1) / T);
  a.conv_blocks = (unsigned)((d.B * a.ntiles * (int64_t)a.nvec + kConvThreads - 1) / kConvThreads);
  const int64_t rows = d.B * d.L;
  int64_t dt_rows = max((int64_t)1, (int64_t)1024 / d.H);
  while ((rows + dt_rows - 1) / dt_rows >= (int64_t)1 << 22) dt_rows *= 2;
  a.dt_rows = (int)dt_rows;
  const unsigned blocks = a.conv_blocks + (unsigned)((rows + dt_rows - 1) / dt_rows);
  const bool al = (uintptr_t)cv.xbc % 16 == 0 && cv.ld_xbc * esize % 16 == 0;
  switch (dtype) {
    case DT_F32: return launch_dt<DT_F32>(a, al, blocks, st);
    case DT_F16: return launch_dt<DT_F16>(a, al, blocks, st);
    case DT_BF16: return launch_dt<DT_BF16>(a, al, blocks, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ssd
