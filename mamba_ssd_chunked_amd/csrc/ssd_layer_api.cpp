// C ABI of the steps around the SSD in a layer: the causal convolution, the
// decode step with it, the residual and gated norms with 8-bit rows, and the
// 8-bit matrix product. Argument validation (host only, before any launch) and
// dispatch to the HIP kernels.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/ssd.h"
#include "ssd_check.hpp"
#include "ssd_launch.hpp"

using ssd::Dims;
using namespace ssd::host;

namespace {

size_t elem_bytes(int dtype) { return dtype == SSD_DTYPE_F32 ? 4 : 2; }

bool known_dtype(int dtype) { return dtype >= SSD_DTYPE_F32 && dtype <= SSD_DTYPE_BF16; }

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// The convolution's parameters and its strided inputs.
int check_conv(const Dims& d, int dtype, const ssd_conv* cv, const void* xbc, int64_t ld_xbc,
               const void* dt_raw, int64_t ld_dt, const int32_t* pos) {
  if (!cv || !cv->weight || !xbc || !dt_raw) return SSD_E_NULL;
  if (cv->width < 2 || cv->width > 4) return SSD_E_UNSUPPORTED;
  if (!aligned16(cv->weight) || !aligned16(cv->bias) || !aligned_to(cv->dt_bias, 4)) return SSD_E_ALIGN;
  if (!aligned_to(xbc, elem_bytes(dtype)) || !aligned_to(dt_raw, elem_bytes(dtype)) || !aligned_to(pos, 4))
    return SSD_E_ALIGN;
  const int64_t cd = (int64_t)d.H * d.P + 2 * (int64_t)d.G * d.N;
  constexpr int64_t kMostLd = (int64_t)1 << 28;  // a row's bytes fit 32 bits
  if (ld_xbc < cd || ld_dt < d.H || ld_xbc >= kMostLd || ld_dt >= kMostLd) return SSD_E_SHAPE;
  int64_t t;
  if (!mul_ok(d.B, cd, &t) || t >= (int64_t)1 << 32) return SSD_E_SHAPE;
  if (!mul_ok(d.B, d.L, &t)) return SSD_E_SHAPE;
  int64_t u;
  if (!mul_ok(t, ld_xbc, &u) || !mul_ok(u, 4, &u) || !mul_ok(t, ld_dt, &u) || !mul_ok(u, 4, &u))
    return SSD_E_SHAPE;
  return SSD_OK;
}

ssd::ConvPtrs conv_ptrs(const ssd_conv* cv, const void* xbc, int64_t ld_xbc, const void* dt_raw,
                        int64_t ld_dt, const int32_t* pos, void* state) {
  return ssd::ConvPtrs{cv->weight, cv->bias, cv->dt_bias, cv->width, xbc, ld_xbc, dt_raw, ld_dt, pos, state};
}

constexpr int64_t kMaxNormCols = 16384;

// What both norms ask of their arguments.
int check_norm(int64_t rows, int64_t cols, int dtype, const void* x, int64_t ld_x, const float* weight,
               float eps, const void* out, const int8_t* q, const float* scale, bool* empty) {
  if (!known_dtype(dtype)) return SSD_E_UNSUPPORTED;
  if (rows < 0 || rows > INT32_MAX || cols <= 0 || cols > kMaxNormCols) return SSD_E_SHAPE;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return SSD_E_SHAPE;
  if (!x || !weight || (!out && !q)) return SSD_E_NULL;
  if ((q == nullptr) != (scale == nullptr)) return SSD_E_NULL;
  int64_t t;
  if (ld_x < cols || !mul_ok(rows, ld_x, &t) || !mul_ok(t, 4, &t)) return SSD_E_SHAPE;
  if (!aligned_to(x, elem_bytes(dtype)) || !aligned16(weight) || !aligned16(out) || !aligned16(q) ||
      !aligned_to(scale, 4))
    return SSD_E_ALIGN;
  *empty = rows == 0;
  return SSD_OK;
}

}  // namespace

extern "C" {

int ssd_conv_forward(const ssd_shape* shape, const ssd_conv* conv, const void* xbc, int64_t ld_xbc,
                     const void* dt_raw, int64_t ld_dt, const int32_t* lengths, const int32_t* pos,
                     void* conv_state, void* X, void* B, void* C, void* dt, void* stream) {
  Dims d;
  bool empty;
  int rc = check_shape(shape, &d, &empty, true);
  if (rc) return rc;
  if ((rc = check_conv(d, shape->dtype, conv, xbc, ld_xbc, dt_raw, ld_dt, pos))) return rc;
  if ((rc = check_ptrs({X, B, C, dt}))) return rc;
  if ((rc = check_opt({conv_state}))) return rc;
  if (!aligned_to(lengths, 4)) return SSD_E_ALIGN;
  if (pos && !conv_state) return SSD_E_NULL;
  if (empty) return SSD_OK;
  return hip_status(ssd::launch_conv_forward(
      d, shape->dtype, conv_ptrs(conv, xbc, ld_xbc, dt_raw, ld_dt, pos, conv_state), lengths, X, B, C, dt,
      (hipStream_t)stream));
}

int ssd_conv_decode_step(const ssd_shape* shape, int path, const ssd_conv* conv, const void* xbc,
                         int64_t ld_xbc, const void* dt_raw, int64_t ld_dt, const float* A, const float* D,
                         const ssd_scales* scales, void* conv_state, const int32_t* pos, void* state,
                         void* Y, void* stream) {
  Dims d;
  bool empty;
  int rc = check_shape(shape, &d, &empty);
  if (rc) return rc;
  if ((rc = check_path(path))) return rc;
  if (d.B > 0 && d.L != 1) return SSD_E_SHAPE;
  // a workgroup per (batch, head): keep the grid's thread count below 2^32
  if (d.B * (int64_t)d.H >= (int64_t)1 << 24) return SSD_E_SHAPE;
  const bool i8 = path == SSD_PATH_INT8;
  if ((rc = check_conv(d, shape->dtype, conv, xbc, ld_xbc, dt_raw, ld_dt, pos))) return rc;
  if (!pos) return SSD_E_NULL;
  if ((rc = check_ptrs({A, D, conv_state, state, Y}))) return rc;
  if (i8 && (rc = check_scales(scales))) return rc;
  if (empty) return SSD_OK;
  return hip_status(ssd::launch_conv_decode_step(
      d, shape->dtype, i8, conv_ptrs(conv, xbc, ld_xbc, dt_raw, ld_dt, pos, conv_state), A, D,
      scale_ptrs(i8 ? scales : nullptr), state, Y, (hipStream_t)stream));
}

int ssd_add_norm(int64_t rows, int64_t cols, int dtype, const void* x, int64_t ld_x, const void* residual,
                 int res_dtype, void* residual_out, const float* weight, float eps, void* out, int8_t* q,
                 float* scale, void* stream) {
  bool empty;
  const int rc = check_norm(rows, cols, dtype, x, ld_x, weight, eps, out, q, scale, &empty);
  if (rc) return rc;
  if (residual || residual_out) {
    if (!known_dtype(res_dtype) || (res_dtype != dtype && res_dtype != SSD_DTYPE_F32)) return SSD_E_UNSUPPORTED;
    if (!aligned16(residual) || !aligned16(residual_out)) return SSD_E_ALIGN;
  }
  if (empty) return SSD_OK;
  ssd::NormArgs a{rows, (int)cols, 1, x, ld_x, nullptr, 0, residual, residual_out, weight, eps, out, q, scale};
  return hip_status(ssd::launch_norm(dtype, res_dtype, a, (hipStream_t)stream));
}

int ssd_gated_norm(int64_t rows, int64_t cols, int64_t groups, int dtype, const void* y, const void* z,
                   int64_t ld_z, const float* weight, float eps, void* out, int8_t* q, float* scale,
                   void* stream) {
  bool empty;
  const int rc = check_norm(rows, cols, dtype, y, cols, weight, eps, out, q, scale, &empty);
  if (rc) return rc;
  if (!z) return SSD_E_NULL;
  if (groups <= 0 || cols % groups != 0) return SSD_E_SHAPE;
  int64_t t;
  if (ld_z < cols || !mul_ok(rows, ld_z, &t) || !mul_ok(t, 4, &t)) return SSD_E_SHAPE;
  if (!aligned16(y) || !aligned_to(z, elem_bytes(dtype))) return SSD_E_ALIGN;
  if (empty) return SSD_OK;
  ssd::NormArgs a{rows, (int)cols, (int)groups, y, cols, z, ld_z, nullptr, nullptr, weight, eps, out, q, scale};
  return hip_status(ssd::launch_norm(dtype, dtype, a, (hipStream_t)stream));
}

// M, N, K of the 8-bit product. The largest sum, K products of -128 * -128,
// fits an int32 up to K = 131056.
static int check_matmul(int64_t M, int64_t N, int64_t K) {
  constexpr int64_t kMost = (int64_t)1 << 26;  // rows: tile indexes and offsets in a tile's rows fit 32 bits
  if (M < 0 || N <= 0 || K <= 0 || M >= kMost || N >= kMost || K > 131056) return SSD_E_SHAPE;
  if (M * N >= (int64_t)1 << 40) return SSD_E_SHAPE;
  if (K % 16 != 0) return SSD_E_UNSUPPORTED;
  return SSD_OK;
}

// No kernel needs a workspace: sums that are split over waves meet in LDS.
size_t ssd_matmul_i8_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

int ssd_matmul_i8(int64_t M, int64_t N, int64_t K, const int8_t* a, const float* a_scale, const int8_t* w,
                  const float* w_scale, const float* bias, int out_dtype, void* out, void* workspace,
                  size_t, void* stream) {
  int rc = check_matmul(M, N, K);
  if (rc) return rc;
  if (!known_dtype(out_dtype)) return SSD_E_UNSUPPORTED;
  if ((rc = check_ptrs({a, w, out}))) return rc;
  if (!a_scale || !w_scale) return SSD_E_NULL;
  if (!aligned_to(a_scale, 4) || !aligned_to(w_scale, 4) || !aligned_to(bias, 4)) return SSD_E_ALIGN;
  if ((rc = check_opt({workspace}))) return rc;
  if (M == 0) return SSD_OK;
  ssd::MatmulI8Args m{M, N, K, a, a_scale, w, w_scale, bias, out};
  return hip_status(ssd::launch_matmul_i8(out_dtype, m, (hipStream_t)stream));
}

int ssd_pack_weight_i8(int64_t N, int64_t K, const float* w, int8_t* q, float* w_scale) {
  if (!w || !q || !w_scale) return SSD_E_NULL;
  int64_t n;
  if (N <= 0 || K <= 0 || !mul_ok(N, K, &n) || !mul_ok(n, 4, &n)) return SSD_E_SHAPE;
  n = N * K;
  // every weight is checked before anything is written
  for (int64_t i = 0; i < n; ++i)
    if (!std::isfinite(w[i])) return SSD_E_VALUE;
  for (int64_t r = 0; r < N; ++r) {
    const float* row = w + r * K;
    float most = 0.f;
    for (int64_t k = 0; k < K; ++k) most = std::fmax(most, std::fabs(row[k]));
    // a row whose step would round to zero holds nothing that codes can carry
    float step = (float)((double)most / 127.0);
    if (!(step > 0.f)) step = 1.f;
    w_scale[r] = step;
    for (int64_t k = 0; k < K; ++k) {
      const double v = std::round((double)row[k] / (double)step);  // half away from zero
      q[r * K + k] = (int8_t)std::fmin(std::fmax(v, -127.0), 127.0);
    }
  }
  return SSD_OK;
}

}  // extern "C"
