// layer_checks.h -- argument checks of the operators around the attention (host code only).
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "tara_attn.h"

namespace tara {

inline int elem_size(tara_dtype t) { return t == TARA_FP32 ? 4 : 2; }
inline bool known_dtype(tara_dtype t) { return t == TARA_BF16 || t == TARA_FP16 || t == TARA_FP32; }
inline bool ptr_aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// Strides of dimensions of size 1 do not matter: they are replaced by 0.
inline tara_view normalised(const tara_view& v) {
  tara_view r = v;
  if (r.B == 1) r.stride_b = 0;
  if (r.H == 1) r.stride_h = 0;
  if (r.N == 1) r.stride_n = 0;
  return r;
}

// Pointer, type, sizes, strides and (align > 0) alignment of pointer and strides in bytes.
inline int check_view(const tara_view* v, int align) {
  if (!v || !v->ptr) return TARA_ERR_NULL;
  if (!known_dtype(v->dtype)) return TARA_ERR_DTYPE;
  if (v->B < 1 || v->H < 1 || v->N < 1 || v->D < 1) return TARA_ERR_SHAPE;
  if ((int64_t)v->H * v->D > 0x7fffffffLL || v->B > 65535) return TARA_ERR_TOO_LARGE;
  const tara_view n = normalised(*v);
  const int64_t limit = (int64_t)1 << 38;   // elements: bytes stay below 2^40
  for (int64_t s : {n.stride_b, n.stride_h, n.stride_n}) {
    if (s < 0) return TARA_ERR_PARAM;
    if (s >= limit) return TARA_ERR_TOO_LARGE;
    if (align && (s * elem_size(v->dtype)) % align != 0) return TARA_ERR_ALIGN;
  }
  if (!ptr_aligned(v->ptr, align ? align : elem_size(v->dtype))) return TARA_ERR_ALIGN;
  return TARA_OK;
}

// True when no two elements of the view share memory by the sufficient rule that each
// dimension, in order of stride, steps past everything the smaller ones reach.
inline bool steps_clear(const tara_view& v) {
  struct Dim { int64_t stride, size; } d[3] = {{v.stride_b, v.B}, {v.stride_h, v.H}, {v.stride_n, v.N}};
  std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  int64_t reach = v.D;
  for (const Dim& x : d) {
    if (x.size == 1) continue;
    if (x.stride < reach) return false;
    reach += x.stride * (x.size - 1);
  }
  return true;
}

inline int check_out_view(const tara_view* v, int align) {
  const int rc = check_view(v, align);
  if (rc != TARA_OK) return rc;
  return steps_clear(normalised(*v)) ? TARA_OK : TARA_ERR_PARAM;
}

inline bool same_layout(const tara_view& a, const tara_view& b) {
  const tara_view x = normalised(a), y = normalised(b);
  return x.ptr == y.ptr && x.B == y.B && x.H == y.H && x.N == y.N && x.D == y.D &&
         x.stride_b == y.stride_b && x.stride_h == y.stride_h && x.stride_n == y.stride_n;
}

inline bool same_shape(const tara_view& a, const tara_view& b) {
  return a.B == b.B && a.H == b.H && a.N == b.N && a.D == b.D;
}

// The norm and rotation of heads of D columns and N tokens.
inline int check_norm_rope(const tara_norm_rope* p, int D, int N, tara_dtype dt) {
  if (p->norm != 0 && p->norm != 1) return TARA_ERR_PARAM;
  if (!p->norm && !p->table) return TARA_ERR_PARAM;
  if (p->norm) {
    if (!std::isfinite(p->eps) || p->eps < 0.0f) return TARA_ERR_PARAM;
    if (p->weight_head_stride < 0 ||
        (p->weight_head_stride != 0 && p->weight_head_stride < D))
      return TARA_ERR_PARAM;
    if ((p->weight_head_stride * elem_size(dt)) % 16 != 0) return TARA_ERR_ALIGN;
    if (!ptr_aligned(p->q_weight, 16) || !ptr_aligned(p->k_weight, 16)) return TARA_ERR_ALIGN;
  }
  if (p->table) {
    if (p->pairing != TARA_ROPE_INTERLEAVED && p->pairing != TARA_ROPE_HALVES)
      return TARA_ERR_PARAM;
    const int unit = p->pairing == TARA_ROPE_HALVES ? 16 : 8;
    if (p->rot_dim < unit || p->rot_dim > D || p->rot_dim % unit != 0) return TARA_ERR_PARAM;
    if (p->table_batch_stride < 0 ||
        (p->table_batch_stride != 0 && p->table_batch_stride < (int64_t)N * p->rot_dim))
      return TARA_ERR_PARAM;
    if (!ptr_aligned(p->table, 16) || p->table_batch_stride % 4 != 0) return TARA_ERR_ALIGN;
  }
  return TARA_OK;
}

}  // namespace tara
