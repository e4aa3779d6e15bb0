// C ABI of the operators that stand beside the SSD in a layer: the gated delta
// rule, the product with an epilogue and the norms between two blocks. Argument
// validation (host only, before any launch) and dispatch to the HIP kernels.
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

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

bool known_dtype(int dtype) { return dtype >= SSD_DTYPE_F32 && dtype <= SSD_DTYPE_BF16; }

// Sequences that are taken one position after the other: one launch instead of three, but
// a time for each position. us, in steps and in chunks, bf16: 64 heads of 64 x 128, 8 positions
// 10.6 and 17.3, 16 17.7 and 17.2, 24 24.7 and 17.2; 4 x 32 heads of 128 x 128, 8 positions 13.4
// and 19.4, 16 22.8 and 19.5; 8 x 80 heads of 64 x 128, 8 positions 22 and 37, 12 30 and 37, 16
// 39 and 37; 64 x 80, 4 positions 75 and 148, 8 112 and 150, 12 156 and 151, 16 209 and 152.
bool delta_in_steps(const Dims& d) {
  return d.L <= 8 || (d.L <= 16 && d.B * (int64_t)d.H * d.P * d.N <= (int64_t)1 << 22);
}

// The shape of the gated delta rule; d->c counts its own chunks.
int delta_shape(const ssd_shape* shape, Dims* d, bool* empty) {
  const int rc = check_shape(shape, d, empty, true);
  if (rc) return rc;
  // the grids' thread counts stay below 2^32 (the scan's: 64 for 16 rows of a head; the steps': delta_step_passes)
  if (d->B * (int64_t)d->H >= (int64_t)1 << 23) return SSD_E_SHAPE;
  d->c = (int)((d->L + ssd::kDeltaChunk - 1) / ssd::kDeltaChunk);
  int64_t t, u;
  if (!mul_ok(d->B, d->c, &t) || !mul_ok(t, d->H, &u) || !mul_ok(u, 1 << 15, &u) || !mul_ok(t, d->G, &u) ||
      !mul_ok(u, 1 << 17, &u))
    return SSD_E_SHAPE;
  return SSD_OK;
}

int delta_args(const Dims& d, int dtype, int flags, const void* X, const void* dt, const float* A, const void* B,
               const void* C, const void* beta, int64_t ld_beta, float scale, float eps, const void* Y,
               ssd::DeltaArgs* a) {
  if (flags & ~(SSD_DELTA_UNIT | SSD_DELTA_LOGIT)) return SSD_E_UNSUPPORTED;
  if (!std::isfinite(scale) || !(eps >= 0.0f) || !std::isfinite(eps)) return SSD_E_SHAPE;
  int rc = check_ptrs({A});
  if (rc) return rc;
  if (d.L > 0) {
    if ((rc = check_ptrs({X, dt, B, C, Y}))) return rc;
    if (!beta) return SSD_E_NULL;
    if (!aligned_to(beta, elem_bytes(dtype))) return SSD_E_ALIGN;
    if (ld_beta < d.H || ld_beta >= (int64_t)1 << 28) return SSD_E_SHAPE;
    int64_t t;
    if (!mul_ok(d.B, d.L, &t) || !mul_ok(t, ld_beta, &t) || !mul_ok(t, 4, &t)) return SSD_E_SHAPE;
  }
  *a = ssd::DeltaArgs{X, dt, A, B, C, beta, ld_beta, scale, eps, (flags & SSD_DELTA_UNIT) != 0,
                      (flags & SSD_DELTA_LOGIT) != 0, const_cast<void*>(Y), nullptr, nullptr};
  return SSD_OK;
}

}  // namespace

extern "C" {

size_t ssd_delta_workspace_bytes(const ssd_shape* shape) {
  Dims d;
  bool empty;
  if (delta_shape(shape, &d, &empty) || empty || delta_in_steps(d)) return 0;
  return ssd::delta_workspace_bytes(d, shape->dtype);
}

int ssd_delta_forward(const ssd_shape* shape, int flags, const void* X, const void* dt, const float* A, const void* B,
                      const void* C, const void* beta, int64_t ld_beta, float scale, float eps, void* Y,
                      const float* initial_state, float* final_state, void* workspace, size_t workspace_bytes,
                      void* stream) {
  Dims d;
  bool empty;
  int rc = delta_shape(shape, &d, &empty);
  if (rc) return rc;
  ssd::DeltaArgs a;
  if ((rc = delta_args(d, shape->dtype, flags, X, dt, A, B, C, beta, ld_beta, scale, eps, Y, &a))) return rc;
  if ((rc = check_opt({initial_state, final_state, workspace}))) return rc;
  a.init = initial_state;
  a.final_state = final_state;
  if (d.B == 0 || (d.L == 0 && !final_state)) return SSD_OK;
  if (delta_in_steps(d)) return hip_status(ssd::launch_delta_steps(d, shape->dtype, a, (hipStream_t)stream));
  if (workspace_bytes < ssd::delta_workspace_bytes(d, shape->dtype)) return SSD_E_WORKSPACE;
  if (!workspace) return SSD_E_NULL;
  return hip_status(ssd::launch_delta_chunks(d, shape->dtype, a, workspace, (hipStream_t)stream));
}

int ssd_delta_step(const ssd_shape* shape, int flags, const void* X, const void* dt, const float* A, const void* B,
                   const void* C, const void* beta, int64_t ld_beta, float scale, float eps, float* state, void* Y,
                   void* stream) {
  Dims d;
  bool empty;
  int rc = delta_shape(shape, &d, &empty);
  if (rc) return rc;
  if (d.B > 0 && d.L != 1) return SSD_E_SHAPE;
  ssd::DeltaArgs a;
  if ((rc = delta_args(d, shape->dtype, flags, X, dt, A, B, C, beta, ld_beta, scale, eps, Y, &a))) return rc;
  if ((rc = check_ptrs({state}))) return rc;
  if (empty) return SSD_OK;
  a.init = a.final_state = state;
  return hip_status(ssd::launch_delta_steps(d, shape->dtype, a, (hipStream_t)stream));
}

// M, N, K of the product.
static int check_product(int64_t M, int64_t N, int64_t K, int dtype) {
  constexpr int64_t kMost = (int64_t)1 << 26;  // rows: tile indexes and offsets in a tile's rows fit 32 bits
  if (M < 0 || N <= 0 || K <= 0 || M >= kMost || N >= kMost || M * N >= (int64_t)1 << 40) return SSD_E_SHAPE;
  if (K >= (int64_t)1 << 22) return SSD_E_SHAPE;  // 256 rows are less than 2^32 bytes
  return known_dtype(dtype) ? SSD_OK : SSD_E_UNSUPPORTED;
}

size_t ssd_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K, int dtype) {
  return check_product(M, N, K, dtype) ? 0 : ssd::matmul_workspace_bytes(M, N, K, dtype);
}

int ssd_matmul(int64_t M, int64_t N, int64_t K, int dtype, const void* a, int64_t ld_a, const void* w,
               const float* bias, int act, const void* residual, int out_dtype, void* out, void* workspace,
               size_t workspace_bytes, void* stream) {
  int rc = check_product(M, N, K, dtype);
  if (rc) return rc;
  if (ld_a < K || ld_a >= (int64_t)1 << 22) return SSD_E_SHAPE;
  if (out_dtype != dtype && out_dtype != SSD_DTYPE_F32) return SSD_E_UNSUPPORTED;
  if (act < SSD_ACT_NONE || act > SSD_ACT_GELU_TANH) return SSD_E_UNSUPPORTED;
  if (!a || !w || !out) return SSD_E_NULL;
  if (!aligned_to(a, elem_bytes(dtype)) || !aligned_to(bias, 4)) return SSD_E_ALIGN;
  if ((rc = check_opt({w, residual, out, workspace}))) return rc;
  if (M == 0) return SSD_OK;
  ssd::MatmulArgs m{M, N, K, a, ld_a, w, bias, act, residual, out};
  if (workspace && !ssd::matmul_aligned(dtype, m) && workspace_bytes < ssd::matmul_workspace_bytes(M, N, K, dtype))
    return SSD_E_WORKSPACE;
  return hip_status(ssd::launch_matmul(dtype, out_dtype, m, workspace, (hipStream_t)stream));
}

int ssd_block_norm(int64_t rows, int64_t cols, int dtype, const void* x, int64_t ld_x, const float* post_weight,
                   const void* gate, int64_t ld_gate, int64_t rows_per_gate, int gate_act, const void* residual,
                   float res_scale, int res_dtype, void* residual_out, const float* weight, float eps, void* out,
                   int8_t* q, float* scale, void* stream) {
  if (!known_dtype(dtype)) return SSD_E_UNSUPPORTED;
  if (rows < 0 || rows > INT32_MAX || cols <= 0 || cols > 16384) return SSD_E_SHAPE;
  if (!(eps >= 0.0f) || !std::isfinite(eps) || !std::isfinite(res_scale)) return SSD_E_SHAPE;
  if (!x || !post_weight || (!out && !q && !residual_out)) return SSD_E_NULL;
  if ((q == nullptr) != (scale == nullptr) || ((out || q) && !weight)) return SSD_E_NULL;
  int64_t t;
  if (ld_x < cols || !mul_ok(rows, ld_x, &t) || !mul_ok(t, 4, &t)) return SSD_E_SHAPE;
  if (!aligned_to(x, elem_bytes(dtype)) || !aligned_to(scale, 4)) return SSD_E_ALIGN;
  const int rc = check_opt({post_weight, weight, out, q});
  if (rc) return rc;
  if (gate) {
    if (gate_act != SSD_ACT_NONE && gate_act != SSD_ACT_SILU && gate_act != SSD_ACT_SIGMOID) return SSD_E_UNSUPPORTED;
    if (rows_per_gate <= 0 || ld_gate < cols || !mul_ok(rows, ld_gate, &t) || !mul_ok(t, 4, &t)) return SSD_E_SHAPE;
    if (!aligned_to(gate, elem_bytes(dtype))) return SSD_E_ALIGN;
  }
  if (residual || residual_out) {
    if (!known_dtype(res_dtype) || (res_dtype != dtype && res_dtype != SSD_DTYPE_F32)) return SSD_E_UNSUPPORTED;
    if (!aligned16(residual) || !aligned16(residual_out)) return SSD_E_ALIGN;
  }
  if (rows == 0) return SSD_OK;
  // a gate of more rows than there are is one for all of them
  const int64_t per = gate ? (rows_per_gate < rows ? rows_per_gate : rows) : 1;
  ssd::BlockNormArgs a{rows, (int)cols, x, ld_x, post_weight, gate, ld_gate, per, gate_act, residual, res_scale,
                       residual_out, weight, eps, out, q, scale};
  return hip_status(ssd::launch_block_norm(dtype, residual || residual_out ? res_dtype : dtype, a, (hipStream_t)stream));
}

}  // extern "C"
