// Internal declarations of the exact-attention operators: argument blocks that
// the C entry points fill and the kernels' launchers take.  Not part of the
// ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "nys.h"

namespace nys {

constexpr int kAttnMaxDim = 256;
constexpr int kAttnMaxGroup = 64;

// Rows of a [rows][heads][dim] tensor; strides in elements.
struct Rows {
  void* p;
  int64_t row, head;
};

// Packed sequences: sequence i's queries are rows q_off[i] .. q_off[i+1]-1,
// its keys rows k_off[i] .. k_off[i+1]-1; query r of nq sees the keys
// j <= r + nk - nq.
struct PromptArgs {
  Rows q, k, v, out;
  float* lse;  // [q_rows][heads] or null
  const int32_t *q_off, *k_off;
  int64_t q_rows, k_rows;
  int32_t n, heads, kv_heads, group, d, dv, dtype;
  float scale;
  int32_t* status;
};

// One query row a request over a shared prefix and the request's own keys,
// all in pages of one pool.
struct SharedArgs {
  Rows q, out;
  float* lse;  // [n][heads] or null
  const void *k, *v;
  int64_t n_pages;
  int32_t page;
  const int32_t* prefix_pages;
  int32_t prefix_len;
  const int32_t* lens;
  const int32_t* table;
  int32_t width;
  int32_t n, heads, kv_heads, group, d, dv, dtype;
  float scale;
  int32_t* status;
};

cudaError_t launch_prompt_general(const PromptArgs& a, cudaStream_t stream);
cudaError_t launch_shared_general(const SharedArgs& a, cudaStream_t stream);

#ifdef __CUDACC__
__device__ __forceinline__ void attn_report(int32_t* status, int32_t bit) {
  if (status) atomicOr(status, bit);
}

// Sequence i's row ranges, held inside the tensors whatever the offsets say.
__device__ __forceinline__ void seq_range(const int32_t* off, int i, int64_t rows, int& lo, int& n,
                                          bool& bad) {
  const int64_t a = off[i], b = off[i + 1];
  const int64_t l = a < 0 ? 0 : (a > rows ? rows : a);
  const int64_t h = b < l ? l : (b > rows ? rows : b);
  bad |= (l != a) | (h != b);
  lo = (int)l;
  n = (int)(h - l);
}
#endif

}  // namespace nys
