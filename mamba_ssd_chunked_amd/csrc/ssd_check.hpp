// Host-side argument checks shared by the C entry points (ssd_api.cpp and
// ssd_layer_api.cpp): nothing here touches the device.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "../../include/ssd.h"
#include "ssd_launch.hpp"

namespace ssd {
namespace host {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
  if (a < 0 || b < 0) return false;
  if (a != 0 && b > INT64_MAX / a) return false;
  *out = a * b;
  return true;
}

// Validates the shape; fills d. *empty is set for batch == 0 or seqlen == 0.
inline int check_shape(const ssd_shape* s, Dims* d, bool* empty) {
  if (!s) return SSD_E_NULL;
  if (s->schedule < SSD_SCHED_AUTO || s->schedule > SSD_SCHED_CHUNK) return SSD_E_SHAPE;
  if (s->batch < 0 || s->seqlen < 0) return SSD_E_SHAPE;
  if (s->nheads <= 0 || s->headdim <= 0 || s->dstate <= 0 || s->ngroups <= 0 || s->chunk <= 0)
    return SSD_E_SHAPE;
  if (s->nheads % s->ngroups != 0) return SSD_E_SHAPE;
  if (s->dtype < SSD_DTYPE_F32 || s->dtype > SSD_DTYPE_BF16) return SSD_E_UNSUPPORTED;
  if (s->chunk != 64 && s->chunk != 128 && s->chunk != 256) return SSD_E_UNSUPPORTED;
  if (s->headdim != 16 && s->headdim != 32 && s->headdim != 64) return SSD_E_UNSUPPORTED;
  if (s->dstate != 16 && s->dstate != 32 && s->dstate != 64 && s->dstate != 128)
    return SSD_E_UNSUPPORTED;
  // grid limits: H in x, chunks in y, batch in z
  const int64_t c = s->seqlen / s->chunk + (s->seqlen % s->chunk != 0);  // no overflow near INT64_MAX
  if (s->nheads > 65535 || s->batch > 65535 || c > 65535) return SSD_E_SHAPE;
  // every element count must fit an int64 byte offset
  int64_t t;
  if (!mul_ok(s->batch, s->seqlen, &t) || !mul_ok(t, s->nheads, &t) ||
      !mul_ok(t, s->headdim, &t) || !mul_ok(t, 16, &t))
    return SSD_E_SHAPE;
  int64_t u;
  if (!mul_ok(s->batch, c, &u) || !mul_ok(u, s->nheads, &u) || !mul_ok(u, s->headdim, &u) ||
      !mul_ok(u, s->dstate, &u) || !mul_ok(u, 16, &u))
    return SSD_E_SHAPE;
  int64_t v;
  if (!mul_ok(s->batch, c, &v) || !mul_ok(v, s->ngroups, &v) || !mul_ok(v, s->chunk, &v) ||
      !mul_ok(v, s->chunk, &v) || !mul_ok(v, 16, &v))
    return SSD_E_SHAPE;
  d->B = s->batch;
  d->L = s->seqlen;
  d->H = (int)s->nheads;
  d->P = (int)s->headdim;
  d->N = (int)s->dstate;
  d->G = (int)s->ngroups;
  d->l = (int)s->chunk;
  d->c = (int)c;
  d->hpg = d->H / d->G;
  d->sched = s->schedule;
  *empty = (s->batch == 0 || s->seqlen == 0);
  return SSD_OK;
}

// The module calls and the decode step compute the float and INT8 paths.
inline int check_path(int path) {
  return (path == SSD_PATH_FLOAT || path == SSD_PATH_INT8) ? SSD_OK : SSD_E_UNSUPPORTED;
}

// ssd_forward also runs the two Table 5 ablation rows.
inline int check_forward_path(int path) {
  return (path >= SSD_PATH_FLOAT && path <= SSD_PATH_ABL_RECON) ? SSD_OK : SSD_E_UNSUPPORTED;
}

// Each required pointer must be non-NULL and 16-byte aligned.
inline int check_ptrs(std::initializer_list<const void*> req) {
  for (const void* p : req)
    if (!p) return SSD_E_NULL;
  for (const void* p : req)
    if (!aligned16(p)) return SSD_E_ALIGN;
  return SSD_OK;
}

inline int check_opt(std::initializer_list<const void*> opt) {
  for (const void* p : opt)
    if (p && !aligned16(p)) return SSD_E_ALIGN;
  return SSD_OK;
}

// Scale arrays are read element-wise: non-NULL and 4-byte aligned. Which
// arrays a path reads: INT8 the first seven; the "Q(X) only" row s_Xq and
// inv_Xq; the "reconstruction + B,C" row the first seven and s_X.
inline int check_scales(const ssd_scales* sc, int path = SSD_PATH_INT8) {
  if (!sc) return SSD_E_NULL;
  const void* req[8];
  int n = 0;
  if (path == SSD_PATH_ABL_QX) {
    req[n++] = sc->s_Xq;
    req[n++] = sc->inv_Xq;
  } else {
    const void* base[] = {sc->s_B, sc->s_C, sc->inv_B, sc->inv_C, sc->inv_X, sc->s_S, sc->M_req};
    for (const void* p : base) req[n++] = p;
    if (path == SSD_PATH_ABL_RECON) req[n++] = sc->s_X;
  }
  for (int i = 0; i < n; ++i)
    if (!req[i]) return SSD_E_NULL;
  for (int i = 0; i < n; ++i)
    if (reinterpret_cast<uintptr_t>(req[i]) & 3u) return SSD_E_ALIGN;
  return SSD_OK;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_E_HIP; }

inline ssd::ScalePtrs scale_ptrs(const ssd_scales* sc) {
  ssd::ScalePtrs p{};
  if (sc) {
    p.s_B = sc->s_B;
    p.s_C = sc->s_C;
    p.inv_B = sc->inv_B;
    p.inv_C = sc->inv_C;
    p.inv_X = sc->inv_X;
    p.s_S = sc->s_S;
    p.M_req = sc->M_req;
    p.s_X = sc->s_X;
    p.s_Xq = sc->s_Xq;
    p.inv_Xq = sc->inv_Xq;
  }
  return p;
}

}  // namespace host
}  // namespace ssd
