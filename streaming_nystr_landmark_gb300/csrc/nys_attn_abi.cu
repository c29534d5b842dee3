// C entry points of the exact-attention operators (declared in include/nys.h):
// argument checks and the choice of kernel.  Every check runs before anything
// is enqueued; nothing here aborts or throws.
#include <cstdint>

#include "nys_attn_check.h"
#include "nys_attn_tc.h"
#include "nys_kv.h"

using namespace nys;

extern "C" {

int nys_attn_workspace_bytes(const nys_attn_config* cfg, int64_t n, int64_t rows, int64_t keys,
                             size_t* bytes) {
  const int rc = check_attn(cfg);
  if (rc) return rc;
  if (!bytes || n < 0 || rows < 0 || keys < 0 || n > INT32_MAX || rows > INT32_MAX ||
      keys > INT32_MAX)
    return NYS_E_INVAL;
  const size_t p = nys::prompt_workspace(*cfg, n, rows, keys);
  const size_t s = rows == n ? nys::shared_workspace(*cfg, n, keys) : 0;
  *bytes = p > s ? p : s;
  return NYS_OK;
}

int nys_attn_prompt(const nys_attn_config* cfg, int64_t n, int64_t q_rows, int64_t k_rows,
                    const int32_t* q_off, const int32_t* k_off, const nys_rows* q,
                    const nys_rows* k, const nys_rows* v, const nys_rows* out, float* lse,
                    void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  int rc = check_attn(cfg);
  if (rc) return rc;
  if (n < 0 || q_rows < 0 || k_rows < 0 || n >= INT32_MAX || q_rows > INT32_MAX ||
      k_rows > INT32_MAX)
    return NYS_E_INVAL;
  if (!k_off && k_rows != q_rows) return NYS_E_INVAL;
  const int es = elem_size(cfg->dtype);
  if ((rc = check_rows(q, q_rows, es)) || (rc = check_rows(k, k_rows, es)) ||
      (rc = check_rows(v, k_rows, es)) || (rc = check_rows(out, q_rows, es)))
    return rc;
  if (!aligned(lse, 4) || !aligned(q_off, 4) || !aligned(k_off, 4) || !aligned(status, 4) ||
      !aligned(workspace, 256))
    return NYS_E_ALIGN;
  if (n == 0 || q_rows == 0) return NYS_OK;
  if (!q_off) return NYS_E_INVAL;
  nys::PromptArgs a{};
  a.q = rows_of(q);
  a.k = rows_of(k);
  a.v = rows_of(v);
  a.out = rows_of(out);
  a.lse = lse;
  a.q_off = q_off;
  a.k_off = k_off ? k_off : q_off;
  a.q_rows = q_rows;
  a.k_rows = k_rows;
  a.n = (int32_t)n;
  a.heads = cfg->heads;
  a.kv_heads = cfg->kv_heads;
  a.group = cfg->heads / cfg->kv_heads;
  a.d = cfg->d;
  a.dv = cfg->dv;
  a.dtype = cfg->dtype;
  a.scale = scale_of(*cfg);
  a.status = status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool room = workspace && workspace_bytes >= nys::prompt_workspace(*cfg, n, q_rows, k_rows);
  const cudaError_t e = nys::prompt_tc_fits(a) && (room || cfg->dtype != NYS_F32)
                            ? nys::launch_prompt_tc(a, room ? workspace : nullptr, s)
                            : nys::launch_prompt_general(a, s);
  return e == cudaSuccess ? NYS_OK : NYS_E_CUDA;
}

int nys_attn_shared(const nys_attn_config* cfg, int64_t n, const nys_pool* pool,
                    const int32_t* prefix_pages, int32_t prefix_len, const int32_t* lens,
                    const int32_t* table, int32_t width, const nys_rows* q, const nys_rows* out,
                    float* lse, void* workspace, size_t workspace_bytes, int32_t* status,
                    void* stream) {
  int rc = check_attn(cfg);
  if (rc) return rc;
  const int es = elem_size(cfg->dtype);
  if (n < 0 || n > INT32_MAX / 64 || prefix_len < 0 || width < 0) return NYS_E_INVAL;
  if ((rc = check_pool(pool, es)) || (rc = check_rows(q, n, es)) || (rc = check_rows(out, n, es)))
    return rc;
  if (!aligned(lse, 4) || !aligned(prefix_pages, 4) || !aligned(lens, 4) || !aligned(table, 4) ||
      !aligned(status, 4) || !aligned(workspace, 256))
    return NYS_E_ALIGN;
  if (n == 0) return NYS_OK;
  if (!lens || (width > 0 && !table) || (prefix_len > 0 && !prefix_pages)) return NYS_E_INVAL;
  if ((int64_t)width * pool->page > INT32_MAX) return NYS_E_UNSUPPORTED;
  size_t need = 0;
  if ((rc = nys_attn_workspace_bytes(cfg, n, n, prefix_len, &need))) return rc;
  if (need > 0 && (!workspace || workspace_bytes < need)) return NYS_E_BUF;
  nys::SharedArgs a{};
  a.q = rows_of(q);
  a.out = rows_of(out);
  a.lse = lse;
  a.k = pool->k;
  a.v = pool->v;
  a.n_pages = pool->n_pages;
  a.page = pool->page;
  a.prefix_pages = prefix_pages;
  a.prefix_len = prefix_len;
  a.lens = lens;
  a.table = table;
  a.width = width;
  a.n = (int32_t)n;
  a.heads = cfg->heads;
  a.kv_heads = cfg->kv_heads;
  a.group = cfg->heads / cfg->kv_heads;
  a.d = cfg->d;
  a.dv = cfg->dv;
  a.dtype = cfg->dtype;
  a.scale = scale_of(*cfg);
  a.status = status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = nys::shared_tiled_fits(a) ? nys::launch_shared_tiled(a, workspace, s)
                                                  : nys::launch_shared_general(a, s);
  return e == cudaSuccess ? NYS_OK : NYS_E_CUDA;
}

int nys_debug_stall_attn_once(int32_t role) {
  if (role != nys::kStallCopies && role != nys::kStallProducts) return NYS_E_INVAL;
  nys::stall_next(role);
  return NYS_OK;
}

int nys_kv_plan(int64_t n, int32_t page, const int32_t* cached, const int32_t* fresh,
                const int32_t* free_pages, int64_t n_free, int32_t* table, int32_t width,
                int64_t total, int32_t* q_off, int32_t* lens, int64_t* slots,
                int32_t* positions, int32_t* taken, int32_t* status, void* stream) {
  if (n < 0 || n >= INT32_MAX || page < 1 || page > (1 << 20) || n_free < 0 ||
      n_free > INT32_MAX || width < 0 || total < 0 || total >= INT32_MAX)
    return NYS_E_INVAL;
  if (!q_off || !taken) return NYS_E_INVAL;
  if (n > 0 && (!cached || !fresh || !lens || (width > 0 && !table))) return NYS_E_INVAL;
  if (n_free > 0 && !free_pages) return NYS_E_INVAL;
  if (total > 0 && (!slots || !positions)) return NYS_E_INVAL;
  if (!aligned(cached, 4) || !aligned(fresh, 4) || !aligned(free_pages, 4) ||
      !aligned(table, 4) || !aligned(q_off, 4) || !aligned(lens, 4) || !aligned(slots, 8) ||
      !aligned(positions, 4) || !aligned(taken, 4) || !aligned(status, 4))
    return NYS_E_ALIGN;
  // Every CTA reads all lengths while others write: what is written overlaps nothing
  // else (lens may be cached itself).
  const Range in[] = {{cached, 4 * n}, {fresh, 4 * n}, {free_pages, 4 * n_free}};
  const Range out[] = {{lens, 4 * n},      {q_off, 4 * (n + 1)},   {table, 4 * n * width},
                       {slots, 8 * total}, {positions, 4 * total}, {taken, 4},
                       {status, 4}};
  for (const Range& o : out) {
    for (const Range& i : in)
      if (overlap(o, i) && !(i.p == cached && o.p == lens && cached == lens)) return NYS_E_INVAL;
    for (const Range& x : out)
      if (&x < &o && overlap(o, x)) return NYS_E_INVAL;
  }
  nys::PlanArgs a{cached,    fresh, free_pages, table,  q_off,  lens,
                  slots,     positions, taken,  status, total,  n_free,
                  (int32_t)n, width, page};
  return nys::launch_plan(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NYS_OK
                                                                              : NYS_E_CUDA;
}

int nys_kv_write(const nys_attn_config* cfg, const nys_pool* pool, int64_t tokens,
                 const nys_rows* k, const nys_rows* v, const int64_t* slots, void* stream) {
  int rc = check_attn(cfg);
  if (rc) return rc;
  if (tokens < 0 || tokens > INT32_MAX) return NYS_E_INVAL;
  const int es = elem_size(cfg->dtype);
  if ((rc = check_pool(pool, es)) || (rc = check_rows(k, tokens, es)) ||
      (rc = check_rows(v, tokens, es)))
    return rc;
  if (!aligned(slots, 8)) return NYS_E_ALIGN;
  if (tokens == 0 || pool->n_pages == 0) return NYS_OK;
  if (!slots) return NYS_E_INVAL;
  nys::WriteArgs a{};
  a.k = k->data;
  a.v = v->data;
  a.pool_k = pool->k;
  a.pool_v = pool->v;
  a.slots = slots;
  a.tokens = tokens;
  a.n_slots = pool->n_pages * pool->page;
  // The widest unit that every row start and row length is a multiple of.
  int64_t k_row = k->row_stride * es, k_head = k->head_stride * es;
  int64_t v_row = v->row_stride * es, v_head = v->head_stride * es;
  int64_t kd = (int64_t)cfg->d * es, vd = (int64_t)cfg->dv * es;
  uintptr_t all = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                  reinterpret_cast<uintptr_t>(a.pool_k) | reinterpret_cast<uintptr_t>(a.pool_v) |
                  (uintptr_t)(k_row | k_head | v_row | v_head | kd | vd);
  a.unit = all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : 2;
  a.k_row = k_row / a.unit;
  a.k_head = k_head / a.unit;
  a.v_row = v_row / a.unit;
  a.v_head = v_head / a.unit;
  a.k_head_units = (uint32_t)(kd / a.unit);
  a.v_head_units = (uint32_t)(vd / a.unit);
  a.k_units = a.k_head_units * cfg->kv_heads;
  a.v_units = a.v_head_units * cfg->kv_heads;
  return nys::launch_write(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NYS_OK
                                                                                : NYS_E_CUDA;
}

}  // extern "C"
