// The 4-bit paged cache and the rows that go into caches: argument blocks that the C
// entry points fill, and the layout that the kernels share.  Not part of the ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "nys_attn.h"

namespace nys {

// A row of d numbers is held as groups of 64, each with a middle and a step in bf16 and
// a code of 4 bits a number: value = middle + step * (code - 8).  Keys and values take
// the groups of the wider of the two.  A page's tokens lie in blocks of 16, one KV
// head's 16 tokens together: the unit that an attention warp copies and multiplies.
// Its 32-bit words are in the order in which a warp's lanes need them for products whose
// 16 rows are the block's tokens (keys) or 16 of a group's numbers (values), so that
// every read of shared memory is one 16-byte word a lane, without conflicts:
//   keys' codes    [group][token % 8][c][token / 8][h]   of numbers 64 group + 32 h + 8 c ..
//   values' codes  [group][r][token % 8 / 2][token / 8][token % 2]    64 group + 8 r ..
//   keys' scales, values' scales  [group][token % 8 / 2][token / 8][token % 2]
constexpr int kGroup4 = 64;
constexpr int kBlock4 = 16;  // tokens

__host__ __device__ constexpr int groups4(int d, int dv) {
  return ((d > dv ? d : dv) + kGroup4 - 1) / kGroup4;
}
// Bytes of a block of G groups, and where its parts start, in bytes.
__host__ __device__ constexpr int block4_bytes(int G) { return 1152 * G; }
__host__ __device__ constexpr int values4(int G) { return 512 * G; }
__host__ __device__ constexpr int key_scales4(int G) { return 1024 * G; }
__host__ __device__ constexpr int value_scales4(int G) { return 1088 * G; }

#ifdef __CUDACC__
// Place of token t (of 16) among a group's scales, and of the codes of 8 numbers from
// 64 g + 8 x, in 32-bit words.
__device__ __forceinline__ int place4(int t) { return (t & 7) / 2 * 4 + t / 8 * 2 + (t & 1); }
__device__ __forceinline__ int key_word4(int g, int t, int x) {
  return g * 128 + (t & 7) * 16 + (x & 3) * 4 + t / 8 * 2 + x / 4;
}
__device__ __forceinline__ int value_word4(int g, int t, int x) {
  return g * 128 + x * 16 + place4(t);
}

// Two f32 operations an instruction.  (A product and a sum that takes it may become one
// operation, rounded once, by measurement: where both roundings count, they are scalar.)
struct Two {
  uint64_t w;
  __device__ __forceinline__ Two() {}
  __device__ __forceinline__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(w) : "f"(a), "f"(b)); }
  __device__ __forceinline__ void get(float& a, float& b) const {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(w));
  }
};
__device__ __forceinline__ Two add(Two a, Two b) {
  Two c;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(c.w) : "l"(a.w), "l"(b.w));
  return c;
}
__device__ __forceinline__ Two mul(Two a, Two b) {
  Two c;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(c.w) : "l"(a.w), "l"(b.w));
  return c;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
  Two d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.w) : "l"(a.w), "l"(b.w), "l"(c.w));
  return d;
}
// The least and largest of numbers; NaN if one is NaN.
__device__ __forceinline__ float least(float a, float b) {
  float c;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
  return c;
}
__device__ __forceinline__ float largest(float a, float b) {
  float c;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
  return c;
}
__device__ __forceinline__ float least(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float largest(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
#endif

// Rows of queries, keys and values on their way to attention (nys_qk.cuh).
struct QkArgs {
  Rows q, k, v, q_out, k_out;  // p null: not there
  const float *q_weight, *k_weight;
  float eps;
  const uint64_t* turns;  // [half]: turns a position, as fractions of 2^64
  int32_t half, interleaved;
  int32_t shift;
  const int32_t* positions;
  const int64_t* slots;
  int64_t tokens, n_slots;
  int32_t heads, kv_heads;  // rows of a token; 0: none
  int32_t d, dv, dtype;
  // Where keys and values go: pages of their own type, or 4-bit blocks (page = blocks a page).
  void *pool_k, *pool_v;
  uint8_t* blocks;
  int32_t page_blocks, groups;
};

struct Read4Args {
  Rows k, v;
  const uint8_t* blocks;
  const int64_t* slots;
  int64_t tokens, n_slots;
  int32_t kv_heads, d, dv, dtype, page_blocks, groups;
};

// One query row a request over its keys in a 4-bit cache.
struct Attn4Args {
  Rows q, out, first;      // first: the result over other keys, joined in (p null: none)
  const float* first_lse;  // [n][heads]
  float* lse;              // [n][heads] or null
  const uint8_t* blocks;
  int64_t n_pages;
  const int32_t *lens, *table;
  int32_t width, page_blocks;
  int32_t n, heads, kv_heads, group, d, dv, dtype;
  float scale;
  int32_t* status;
};

cudaError_t launch_qk_f32(const QkArgs& a, cudaStream_t stream);
cudaError_t launch_qk_bf16(const QkArgs& a, cudaStream_t stream);
cudaError_t launch_qk_f16(const QkArgs& a, cudaStream_t stream);
cudaError_t launch_read4_f32(const Read4Args& a, cudaStream_t stream);
cudaError_t launch_read4_bf16(const Read4Args& a, cudaStream_t stream);
cudaError_t launch_read4_f16(const Read4Args& a, cudaStream_t stream);
cudaError_t launch_qk(const QkArgs& a, cudaStream_t stream);
cudaError_t launch_read4(const Read4Args& a, cudaStream_t stream);
cudaError_t launch_attn4_16(const Attn4Args& a, void* workspace, cudaStream_t stream);
cudaError_t launch_attn4_f32(const Attn4Args& a, void* workspace, cudaStream_t stream);
cudaError_t launch_attn4(const Attn4Args& a, void* workspace, cudaStream_t stream);
size_t attn4_workspace(const nys_attn_config& c, int64_t n, int64_t keys);

}  // namespace nys
