// C entry points of norm and rotation, of appending to caches and of the 4-bit cache
// (declared in include/nys.h): argument checks, all before anything is enqueued.
#include <cmath>
#include <cstdint>

#include "nys_attn_check.h"
#include "nys_kv4.h"

using namespace nys;

namespace {

int64_t page4_bytes(const nys_attn_config& c, int32_t page) {
  return (int64_t)c.kv_heads * (page / kBlock4) * block4_bytes(groups4(c.d, c.dv));
}

// Rows that a caller may leave out.
Rows rows_or_none(const nys_rows* r) { return r ? rows_of(r) : Rows{}; }

int check_prepare(const nys_qk_prepare* p, const nys_attn_config& c, int64_t tokens,
                  const int32_t* positions) {
  if (!p || !std::isfinite(p->eps) || p->eps < 0.f) return NYS_E_INVAL;
  if (p->rot < 0 || (p->rot & 1) || p->rot > c.d || (p->interleaved & ~1)) return NYS_E_INVAL;
  if (p->rot > 0 && (!p->turns || (tokens > 0 && !positions))) return NYS_E_INVAL;
  if (!aligned(p->q_weight, 4) || !aligned(p->k_weight, 4) || !aligned(p->turns, 8) ||
      !aligned(positions, 4))
    return NYS_E_ALIGN;
  return NYS_OK;
}

// (A page's bytes fit 31 bits: kernels take them so.)
int check_pool4(const nys_pool4* p, const nys_attn_config& c) {
  if (!p || p->n_pages < 0 || p->page < kBlock4 || p->page % kBlock4) return NYS_E_INVAL;
  if (p->n_pages > 0 && !p->data) return NYS_E_INVAL;
  if (p->n_pages > INT32_MAX || p->page > (1 << 20) || page4_bytes(c, p->page) > INT32_MAX)
    return NYS_E_UNSUPPORTED;
  return aligned(p->data, 16) ? NYS_OK : NYS_E_ALIGN;
}

// The arguments that calls on rows share; `v` is null where there are no values.
int fill(QkArgs& a, const nys_attn_config* cfg, const nys_qk_prepare* prep, int64_t tokens,
         const nys_rows* q, const nys_rows* k, const nys_rows* v, const int32_t* positions,
         const nys_rows* q_out, const nys_rows* k_out) {
  int rc = check_attn(cfg);
  if (rc) return rc;
  if (tokens < 0 || tokens > INT32_MAX) return NYS_E_INVAL;
  if ((rc = check_prepare(prep, *cfg, tokens, positions))) return rc;
  if (!q != !q_out) return NYS_E_INVAL;
  const int es = elem_size(cfg->dtype);
  for (const nys_rows* r : {q, k, v, q_out, k_out})
    if (r && (rc = check_rows(r, tokens, es))) return rc;
  a.q = rows_or_none(q);
  a.k = rows_or_none(k);
  a.v = rows_or_none(v);
  a.q_out = rows_or_none(q_out);
  a.k_out = rows_or_none(k_out);
  a.q_weight = prep->q_weight;
  a.k_weight = prep->k_weight;
  a.eps = prep->eps;
  a.turns = prep->turns;
  a.half = prep->rot / 2;
  a.interleaved = prep->interleaved;
  a.shift = prep->shift;
  a.positions = positions;
  a.tokens = tokens;
  a.heads = q ? cfg->heads : 0;
  a.kv_heads = k ? cfg->kv_heads : 0;
  a.d = cfg->d;
  a.dv = v ? cfg->dv : cfg->d;
  a.dtype = cfg->dtype;
  return NYS_OK;
}

int run(const QkArgs& a, void* stream) {
  return launch_qk(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NYS_OK : NYS_E_CUDA;
}

}  // namespace

extern "C" {

int nys_qk_rows(const nys_attn_config* cfg, const nys_qk_prepare* prep, int64_t tokens,
                const nys_rows* q, const nys_rows* k, const int32_t* positions,
                const nys_rows* q_out, const nys_rows* k_out, void* stream) {
  if (!k != !k_out || (!q && !k)) return NYS_E_INVAL;
  QkArgs a{};
  const int rc = fill(a, cfg, prep, tokens, q, k, nullptr, positions, q_out, k_out);
  return rc ? rc : run(a, stream);
}

int nys_kv_append(const nys_attn_config* cfg, const nys_qk_prepare* prep, const nys_pool* pool,
                  int64_t tokens, const nys_rows* q, const nys_rows* k, const nys_rows* v,
                  const int32_t* positions, const int64_t* slots, const nys_rows* q_out,
                  const nys_rows* k_out, void* stream) {
  if (!k || !v) return NYS_E_INVAL;
  QkArgs a{};
  int rc = fill(a, cfg, prep, tokens, q, k, v, positions, q_out, k_out);
  if (rc || (rc = check_pool(pool, elem_size(cfg->dtype)))) return rc;
  if (tokens > 0 && !slots) return NYS_E_INVAL;
  if (!aligned(slots, 8)) return NYS_E_ALIGN;
  a.slots = slots;
  a.n_slots = pool->n_pages * pool->page;
  a.pool_k = pool->k;
  a.pool_v = pool->v;
  return run(a, stream);
}

int nys_kv4_append(const nys_attn_config* cfg, const nys_qk_prepare* prep, const nys_pool4* pool,
                   int64_t tokens, const nys_rows* q, const nys_rows* k, const nys_rows* v,
                   const int32_t* positions, const int64_t* slots, const nys_rows* q_out,
                   const nys_rows* k_out, void* stream) {
  if (!k || !v) return NYS_E_INVAL;
  QkArgs a{};
  int rc = fill(a, cfg, prep, tokens, q, k, v, positions, q_out, k_out);
  if (rc || (rc = check_pool4(pool, *cfg))) return rc;
  if (tokens > 0 && !slots) return NYS_E_INVAL;
  if (!aligned(slots, 8)) return NYS_E_ALIGN;
  a.slots = slots;
  a.n_slots = pool->n_pages * pool->page;
  a.blocks = static_cast<uint8_t*>(pool->data);
  a.page_blocks = pool->page / kBlock4;
  a.groups = groups4(cfg->d, cfg->dv);
  return run(a, stream);
}

int nys_kv4_write(const nys_attn_config* cfg, const nys_pool4* pool, int64_t tokens,
                  const nys_rows* k, const nys_rows* v, const int64_t* slots, void* stream) {
  const nys_qk_prepare none{};
  return nys_kv4_append(cfg, &none, pool, tokens, nullptr, k, v, nullptr, slots, nullptr, nullptr,
                        stream);
}

int nys_kv4_read(const nys_attn_config* cfg, const nys_pool4* pool, int64_t tokens,
                 const int64_t* slots, const nys_rows* k_out, const nys_rows* v_out,
                 void* stream) {
  int rc = check_attn(cfg);
  if (rc) return rc;
  if (tokens < 0 || tokens > INT32_MAX) return NYS_E_INVAL;
  const int es = elem_size(cfg->dtype);
  if ((rc = check_pool4(pool, *cfg)) || (rc = check_rows(k_out, tokens, es)) ||
      (rc = check_rows(v_out, tokens, es)))
    return rc;
  if (!aligned(slots, 8)) return NYS_E_ALIGN;
  if (tokens == 0) return NYS_OK;
  if (!slots) return NYS_E_INVAL;
  Read4Args a{};
  a.k = rows_of(k_out);
  a.v = rows_of(v_out);
  a.blocks = static_cast<const uint8_t*>(pool->data);
  a.slots = slots;
  a.tokens = tokens;
  a.n_slots = pool->n_pages * pool->page;
  a.kv_heads = cfg->kv_heads;
  a.d = cfg->d;
  a.dv = cfg->dv;
  a.dtype = cfg->dtype;
  a.page_blocks = pool->page / kBlock4;
  a.groups = groups4(cfg->d, cfg->dv);
  return launch_read4(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NYS_OK : NYS_E_CUDA;
}

int nys_kv4_page_bytes(const nys_attn_config* cfg, int32_t page, size_t* bytes) {
  const int rc = check_attn(cfg);
  if (rc) return rc;
  if (!bytes || page < kBlock4 || page % kBlock4) return NYS_E_INVAL;
  if (page > (1 << 20) || page4_bytes(*cfg, page) > INT32_MAX) return NYS_E_UNSUPPORTED;
  *bytes = (size_t)page4_bytes(*cfg, page);
  return NYS_OK;
}

int nys_attn4_workspace_bytes(const nys_attn_config* cfg, int64_t n, int64_t keys, size_t* bytes) {
  const int rc = check_attn(cfg);
  if (rc) return rc;
  if (!bytes || n < 0 || n > INT32_MAX / 64 || keys < 0 || keys > INT32_MAX) return NYS_E_INVAL;
  *bytes = attn4_workspace(*cfg, n, keys);
  return NYS_OK;
}

int nys_attn4(const nys_attn_config* cfg, int64_t n, const nys_pool4* pool, const int32_t* lens,
              const int32_t* table, int32_t width, const nys_rows* q, const nys_rows* first,
              const float* first_lse, const nys_rows* out, float* lse, void* workspace,
              size_t workspace_bytes, int32_t* status, void* stream) {
  int rc = check_attn(cfg);
  if (rc) return rc;
  if (n < 0 || n > INT32_MAX / 64 || width < 0) return NYS_E_INVAL;
  const int es = elem_size(cfg->dtype);
  if ((rc = check_pool4(pool, *cfg)) || (rc = check_rows(q, n, es)) || (rc = check_rows(out, n, es)))
    return rc;
  if (first && (rc = check_rows(first, n, es))) return rc;
  if (!first != !first_lse) return NYS_E_INVAL;
  if (!aligned(lse, 4) || !aligned(first_lse, 4) || !aligned(lens, 4) || !aligned(table, 4) ||
      !aligned(status, 4) || !aligned(workspace, 256))
    return NYS_E_ALIGN;
  if (n == 0) return NYS_OK;
  if (!lens || (width > 0 && !table)) return NYS_E_INVAL;
  if ((int64_t)width * pool->page > INT32_MAX) return NYS_E_UNSUPPORTED;
  const size_t need = attn4_workspace(*cfg, n, (int64_t)width * pool->page);
  if (need > 0 && (!workspace || workspace_bytes < need)) return NYS_E_BUF;
  Attn4Args a{};
  a.q = rows_of(q);
  a.out = rows_of(out);
  a.first = rows_or_none(first);
  a.first_lse = first_lse;
  a.lse = lse;
  a.blocks = static_cast<const uint8_t*>(pool->data);
  a.n_pages = pool->n_pages;
  a.lens = lens;
  a.table = table;
  a.width = width;
  a.page_blocks = pool->page / kBlock4;
  a.n = (int32_t)n;
  a.heads = cfg->heads;
  a.kv_heads = cfg->kv_heads;
  a.group = cfg->heads / cfg->kv_heads;
  a.d = cfg->d;
  a.dv = cfg->dv;
  a.dtype = cfg->dtype;
  a.scale = scale_of(*cfg);
  a.status = status;
  return launch_attn4(a, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NYS_OK
                                                                                      : NYS_E_CUDA;
}

}  // extern "C"
