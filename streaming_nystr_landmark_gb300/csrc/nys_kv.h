// Internal declarations of the paged cache's bookkeeping (nys_kv.cu).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace nys {

struct PlanArgs {
  const int32_t *cached, *fresh;  // [n]
  const int32_t* free_pages;      // [n_free]
  int32_t* table;                 // [n][width]
  int32_t* q_off;                 // [n + 1]
  int32_t* lens;                  // [n]; may be `cached`
  int64_t* slots;                 // [total]
  int32_t* positions;             // [total]
  int32_t* taken;                 // [1]
  int32_t* status;
  int64_t total, n_free;
  int32_t n, width, page;
};

// Sizes and strides in units of `unit` bytes.
struct WriteArgs {
  const void *k, *v;
  void *pool_k, *pool_v;
  const int64_t* slots;
  int64_t tokens, n_slots;
  int64_t k_row, k_head, v_row, v_head;
  uint32_t k_units, v_units, k_head_units, v_head_units;
  int32_t unit;
};

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t stream);
cudaError_t launch_write(const WriteArgs& a, cudaStream_t stream);

}  // namespace nys
