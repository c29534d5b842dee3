// Argument checks that the C entry points of the exact operators share: they run
// before anything is enqueued, and nothing here aborts or throws.
#pragma once

#include <cmath>
#include <cstdint>

#include "nys.h"
#include "nys_attn.h"

namespace nys {

inline int elem_size(int dtype) { return dtype == NYS_F32 ? 4 : 2; }

inline int check_attn(const nys_attn_config* c) {
  if (!c || c->heads < 1 || c->kv_heads < 1 || c->heads % c->kv_heads) return NYS_E_INVAL;
  if (c->d <= 0 || c->dv <= 0 || (c->d & 3) || (c->dv & 3)) return NYS_E_INVAL;
  if (c->dtype != NYS_F32 && c->dtype != NYS_BF16 && c->dtype != NYS_F16) return NYS_E_INVAL;
  if (!std::isfinite(c->scale) || c->scale < 0.f) return NYS_E_INVAL;
  if (c->d > kAttnMaxDim || c->dv > kAttnMaxDim ||
      c->heads / c->kv_heads > kAttnMaxGroup || c->heads > 65535)
    return NYS_E_UNSUPPORTED;
  return NYS_OK;
}

inline float scale_of(const nys_attn_config& c) {
  return c.scale != 0.f ? c.scale : 1.0f / std::sqrt((float)c.d);
}

// A rows argument of `rows` rows: present (unless there are no rows), its
// element type's alignment, strides that keep 64-bit offsets in range.
inline int check_rows(const nys_rows* r, int64_t rows, int elem) {
  if (!r) return NYS_E_INVAL;
  if (rows == 0) return NYS_OK;
  if (!r->data || r->row_stride < 0 || r->head_stride < 0) return NYS_E_INVAL;
  if (r->row_stride > (int64_t(1) << 40) || r->head_stride > (int64_t(1) << 40)) return NYS_E_INVAL;
  if (reinterpret_cast<uintptr_t>(r->data) % (uintptr_t)elem) return NYS_E_ALIGN;
  return NYS_OK;
}

inline Rows rows_of(const nys_rows* r) { return {r->data, r->row_stride, r->head_stride}; }

inline int check_pool(const nys_pool* p, int elem) {
  if (!p || p->n_pages < 0 || p->page < 1) return NYS_E_INVAL;
  if (p->n_pages > 0 && (!p->k || !p->v)) return NYS_E_INVAL;
  if (p->n_pages > INT32_MAX || p->page > (1 << 20)) return NYS_E_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(p->k) % (uintptr_t)elem ||
      reinterpret_cast<uintptr_t>(p->v) % (uintptr_t)elem)
    return NYS_E_ALIGN;
  return NYS_OK;
}

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) % to) == 0; }

struct Range {
  const void* p;
  int64_t bytes;
};
inline bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && a.bytes > 0 && b.bytes > 0 && x < y + (uintptr_t)b.bytes &&
         y < x + (uintptr_t)a.bytes;
}

}  // namespace nys
