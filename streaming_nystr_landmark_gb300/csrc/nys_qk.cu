// Queries, keys and values on their way from a layer's projections to attention:
//
//   y = x / sqrt(mean_i x_i^2 + eps) * w          per head (queries and keys)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = (position + shift) f_i,
//
// for the pairs (i, i + half) or (2i, 2i + 1) of the first 2 half numbers, written to
// q_out and k_out, or with the values into the pages of their slots, as they are or in
// 4 bits.  f32 throughout, rounded once where a row is stored.
//
// Angles: f_i comes as turns a position, a 64-bit binary fraction F_i.  The product with
// the position modulo 2^64 is the exact fraction of a turn for any 32-bit position, off
// by position * 2^-65 turns for the rounding of F_i; its upper 32 bits go to sinpi and
// cospi.  (In f32 the angle of position 10^6 would be off by 0.06.)
//
// 4 bits: for a group of 64 numbers with least lo and largest hi
//   mid  = bf16(lo + (hi - lo) 8/15),  step = bf16 up(max((hi - mid) / 7, (mid - lo) / 8)),
//   code = round((x - mid) / step) + 8, ties to even, held in 0 .. 15,
// each operation rounded to f32, quotients correctly (for the codes by Markstein's
// correction of a product with the reciprocal: 2 FMAs instead of a division).  Every
// number is held to half a step; a group with a number that is not finite, or of a
// spread past f32, has a step of NaN.
//
// Bound by HBM: a row is read and written once.  A warp takes a token (a part of its rows
// where there are few tokens): it makes the token's sines once, turns them and the weights into two
// factors a number, y_i = (x_i A_i + x_pair B_i) / rms, and runs over the heads.  A row
// lies over 8, 16 or 32 lanes, 8 numbers a lane, so that a lane's numbers are one code
// word and a pair's other half is a lane away (or, where half is no multiple of 8, in
// shared memory).
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nys_attn_tc.h"
#include "nys_kv4.h"

namespace nys {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxHalf = kAttnMaxDim / 2;
constexpr float kLeastStep = 0x1p-100f;

template <typename T>
struct alignas(4 * sizeof(T)) Four {
  T x[4];
};

// Four numbers at p, as one word where that is aligned.
template <typename T>
__device__ __forceinline__ Four<T> load4(const T* p) {
  if (reinterpret_cast<uintptr_t>(p) % sizeof(Four<T>) == 0) return *reinterpret_cast<const Four<T>*>(p);
  return {p[0], p[1], p[2], p[3]};
}
// 8 numbers as they lie in memory.
template <typename T>
struct Eight {
  static constexpr int kWords = 2 * sizeof(T);
  uint32_t w[kWords];
};
__device__ __forceinline__ void widen8(const Eight<float>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r.w[i]);
}
__device__ __forceinline__ void widen8(const Eight<__nv_bfloat16>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(r.w[i] << 16);
    x[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen8(const Eight<__half>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
    x[2 * i] = y.x;
    x[2 * i + 1] = y.y;
  }
}
__device__ __forceinline__ void narrow8(const float (&x)[8], Eight<float>& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(x[i]);
}
__device__ __forceinline__ void narrow8(const float (&x)[8], Eight<__nv_bfloat16>& r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    r.w[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
}
__device__ __forceinline__ void narrow8(const float (&x)[8], Eight<__half>& r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 y = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    r.w[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// The first n (8, 4 or fewer: none) of 8 numbers at p; the others are 0.  wide: p and the
// rows' strides are multiples of 16 bytes.
template <typename T>
__device__ __forceinline__ void get8(Eight<T>& r, const T* p, int n, bool wide) {
#pragma unroll
  for (int i = 0; i < Eight<T>::kWords; ++i) r.w[i] = 0;
  if (n >= 8 && wide) {
#pragma unroll
    for (int i = 0; i < Eight<T>::kWords; i += 4) {
      const uint4 y = reinterpret_cast<const uint4*>(p)[i / 4];
      r.w[i] = y.x, r.w[i + 1] = y.y, r.w[i + 2] = y.z, r.w[i + 3] = y.w;
    }
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (n >= 4 * h + 4) {
      const Four<T> y = load4(p + 4 * h);
#pragma unroll
      for (int i = 0; i < Eight<T>::kWords / 2; ++i)
        r.w[h * (Eight<T>::kWords / 2) + i] = reinterpret_cast<const uint32_t*>(&y)[i];
    }
}
template <typename T>
__device__ __forceinline__ void put8(const Eight<T>& r, T* p, int n, bool wide) {
  if (n >= 8 && wide) {
#pragma unroll
    for (int i = 0; i < Eight<T>::kWords; i += 4)
      reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(r.w[i], r.w[i + 1], r.w[i + 2], r.w[i + 3]);
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (n >= 4 * h + 4) {
      Four<T> y;
#pragma unroll
      for (int i = 0; i < Eight<T>::kWords / 2; ++i)
        reinterpret_cast<uint32_t*>(&y)[i] = r.w[h * (Eight<T>::kWords / 2) + i];
      if (reinterpret_cast<uintptr_t>(p) % sizeof(Four<T>) == 0) {
        *reinterpret_cast<Four<T>*>(p + 4 * h) = y;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[4 * h + i] = y.x[i];
      }
    }
}
template <typename T>
__device__ __forceinline__ bool is_wide(const void* p, int64_t row, int64_t head) {
  return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)(row * sizeof(T)) | (uintptr_t)(head * sizeof(T))) %
             16 == 0;
}

// x / by, rounded correctly, for inv = 1 / by rounded (Markstein), of a quotient that is
// no subnormal number.
__device__ __forceinline__ float quotient(float x, float by, float inv) {
  const float q = __fmul_rn(x, inv);
  return __fmaf_rn(__fmaf_rn(-q, by, x), inv, q);
}

// A group of 64 numbers over 8 lanes, the first n of 8 a lane, to its scale word and this
// lane's 8 codes.
__device__ __forceinline__ uint32_t quantize(const float (&y)[8], int n, uint32_t& scale) {
  float lo = INFINITY, hi = -INFINITY, odd = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (n >= 4 * h + 4) {
#pragma unroll
      for (int i = 4 * h; i < 4 * h + 4; ++i) {
        lo = fminf(lo, y[i]);
        hi = fmaxf(hi, y[i]);
        odd += y[i];  // fminf and fmaxf pass over NaN, a sum does not
      }
    }
  // Bit 0: a NaN, bit 1: a number at all.  (Opposite infinities count as NaN, rightly.)
  uint32_t flags = (odd != odd ? 1u : 0u) | (n >= 4 ? 2u : 0u);
#pragma unroll
  for (int o = 4; o; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o, 8));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o, 8));
    flags |= __shfl_xor_sync(0xffffffffu, flags, o, 8);
  }
  if (flags == 0) {
    scale = 0;
    return 0x88888888u;
  }
  const float span = __fmul_rn(__fsub_rn(hi, lo), 8.f);
  const bool plain = span > 0x1p-90f && span < 0x1p125f;  // (the quotients' precondition)
  const float part = plain ? quotient(span, 15.f, 1.f / 15.f) : __fdiv_rn(span, 15.f);
  const float mid = __bfloat162float(__float2bfloat16_rn(__fadd_rn(lo, part)));
  const float up = __fsub_rn(hi, mid);
  float step = fmaxf(plain ? quotient(up, 7.f, 1.f / 7.f) : __fdiv_rn(up, 7.f),
                     __fmul_rn(__fsub_rn(mid, lo), 0.125f));
  step = __uint_as_float((__float_as_uint(step) + 0xffffu) & 0xffff0000u);
  if ((flags & 1) || !(fabsf(mid) < INFINITY) || !(step < INFINITY)) {
    scale = 0x7fc07fc0u;
    return 0x88888888u;
  }
  if (step < kLeastStep) step = 0.f;
  scale = __float_as_uint(step) | __float_as_uint(mid) >> 16;
  if (step == 0.f) return 0x88888888u;
  const float inv = __frcp_rn(step);
  // t is in -8 .. 7 but for its rounding: t + 1.5 * 2^23 + 8 rounds it to a whole number, ties to
  // even, and has the code in its last bits; the bits above them add up to a constant.
  uint32_t codes = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float x = n >= (i / 4 + 1) * 4 ? __fsub_rn(y[i], mid) : 0.f;
    codes = codes * 16 + __float_as_uint(__fadd_rn(quotient(x, step, inv), 12582920.f));
  }
  return codes - 0x3f400000u;  // 0x4b400000 * (1 + 16 + .. + 16^7), modulo 2^32
}

enum Kind { kQueries, kKeys, kValues };

// What a warp knows of its token.
struct Token {
  int64_t at;       // its row
  int64_t slot;     // < 0: none
  uint32_t* block;  // of KV head 0, 4-bit caches
  int in;           // place in the block
};

// Heads first + sub, first + sub + 32 / L, .. below end of one kind of rows.
template <typename T, int L, bool Q4, Kind K>
__device__ __forceinline__ void run_rows(const QkArgs& a, const Token& t, int first, int end,
                                         const float2* turns, float* stage) {
  constexpr int kPer = 32 / L;
  constexpr int kAhead = 2;  // loads in flight before the first is used
  const int lane = threadIdx.x & 31, l = lane & (L - 1), sub = lane / L;
  const Rows& from = K == kQueries ? a.q : K == kKeys ? a.k : a.v;
  const Rows& to = K == kQueries ? a.q_out : a.k_out;
  const int dim = K == kValues ? a.dv : a.d;
  const int n = dim - 8 * l;
  const T* src = static_cast<const T*>(from.p) + t.at * from.row + 8 * l;
  const bool wide = is_wide<T>(from.p, from.row, from.head);
  Eight<T> raw[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int h = first + i * kPer + sub;
    get8(raw[i], src + h * from.head, h < end ? n : 0, wide);
  }

  // y_i = (x_i A_i + x_pair B_i) * inv.
  float fa[8], fb[8];
  const float* weight = K == kQueries ? a.q_weight : a.k_weight;
  const int half = a.half;
  const bool near = (half & 7) == 0;  // a lane's pairs are all one lane's
  if (K != kValues) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = 8 * l + i;
      const float w = weight && c < dim ? weight[c] : 1.f;
      fa[i] = w;
      fb[i] = 0.f;
      if (c < 2 * half) {
        const bool second = a.interleaved ? (i & 1) : c >= half;
        const float2 z = turns[a.interleaved ? c / 2 : second ? c - half : c];
        const int pair = a.interleaved ? c ^ 1 : second ? c - half : c + half;
        const float wp = weight ? weight[pair] : 1.f;
        fa[i] = w * z.x;
        fb[i] = second ? wp * z.y : -(wp * z.y);
      }
    }
  }
  const float inv_d = 1.f / (float)a.d;
  const bool out_wide = to.p && is_wide<T>(to.p, to.row, to.head);
  T* dst = to.p ? static_cast<T*>(to.p) + t.at * to.row + 8 * l : nullptr;
  T* page = nullptr;
  bool page_wide = false;
  if (!Q4 && K != kQueries && t.slot >= 0) {
    void* pool = K == kValues ? a.pool_v : a.pool_k;
    page = static_cast<T*>(pool) + t.slot * a.kv_heads * dim + 8 * l;
    page_wide = is_wide<T>(pool, dim, dim);
  }

  for (int base = first; base < end; base += kAhead * kPer) {
#pragma unroll
    for (int b = 0; b < kAhead; ++b) {
      const int h0 = base + b * kPer, h = h0 + sub;
      if (h0 >= end) break;
      const bool row = h < end;
      if (K == kValues && !Q4) {
        if (row && page) put8(raw[b], page + h * dim, n, page_wide);
      } else {
        float y[8];
        widen8(raw[b], y);
        if (K != kValues) {
          float inv = 1.f;
          if (weight) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
            for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, L);
            inv = rsqrtf(fmaf(ss, inv_d, a.eps));
          }
          if (half > 0) {
            float p[8];
            if (a.interleaved) {
#pragma unroll
              for (int i = 0; i < 8; ++i) p[i] = y[i ^ 1];
            } else if (near) {
              const int other = 8 * l < half ? l + half / 8 : l - half / 8;
              Eight<T> z;
#pragma unroll
              for (int i = 0; i < Eight<T>::kWords; ++i) z.w[i] = __shfl_sync(0xffffffffu, raw[b].w[i], other, L);
              widen8(z, p);
            } else {
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; i += 4)
                *reinterpret_cast<float4*>(stage + sub * 8 * L + 8 * l + i) =
                    make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int c = 8 * l + i, pair = c < half ? c + half : c - half;
                p[i] = c < 2 * half ? stage[sub * 8 * L + pair] : 0.f;
              }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              // (Beyond 2 half there is no pair: what lies there may be infinite.)
              const float z = 8 * l + i < 2 * half ? p[i] : 0.f;
              y[i] = fmaf(y[i], fa[i], z * fb[i]) * inv;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = y[i] * fa[i] * inv;
          }
        }
        if (!Q4 || K != kValues) {
          Eight<T> z;
          narrow8(y, z);
          if (row && dst) put8(z, dst + h * to.head, n, out_wide);
          if (!Q4 && row && page) put8(z, page + h * dim, n, page_wide);
        }
        if (Q4 && K != kQueries && t.slot >= 0) {
          uint32_t scale;
          const uint32_t codes = quantize(y, n, scale);
          const int g = l / 8, x = l & 7;
          if (row && g < a.groups) {
            uint32_t* at = t.block + (int64_t)h * a.page_blocks * (block4_bytes(a.groups) / 4);
            at[K == kValues ? values4(a.groups) / 4 + value_word4(g, t.in, x) : key_word4(g, t.in, x)] = codes;
            if (x == 0)
              at[(K == kValues ? value_scales4(a.groups) : key_scales4(a.groups)) / 4 + g * 16 + place4(t.in)] =
                  scale;
          }
        }
      }
      const int next = h + kAhead * kPer;
      get8(raw[b], src + next * from.head, next < end ? n : 0, wide);
    }
  }
}

// Block of a slot's token, of KV head 0.
__device__ __forceinline__ int64_t block_of(int64_t slot, int kv_heads, int page_blocks) {
  const int64_t block = slot >> 4;
  if (block <= INT32_MAX) {
    const uint32_t page = (uint32_t)block / (uint32_t)page_blocks;
    return (int64_t)page * kv_heads * page_blocks + ((uint32_t)block - page * (uint32_t)page_blocks);
  }
  const int64_t page = block / page_blocks;
  return page * kv_heads * page_blocks + (block - page * page_blocks);
}

// A warp takes part `w % parts` of token w / parts's steps of 32 / L rows.
template <typename T, int L, bool Q4>
__global__ void __launch_bounds__(kThreads, 4) qk_kernel(QkArgs a, int parts) {
  constexpr int kPer = 32 / L;
  __shared__ float2 s_turn[kWarps][kMaxHalf];
  __shared__ __align__(16) float s_stage[kWarps][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
  Token t;
  t.at = parts == 1 ? w : w / parts;
  if (t.at >= a.tokens) return;
  const int part = (int)(w - t.at * parts);
  const int sq = (a.heads + kPer - 1) / kPer, sk = (a.kv_heads + kPer - 1) / kPer;
  const int all = sq + sk + (a.v.p ? sk : 0);
  const int s0 = (int)((int64_t)all * part / parts), s1 = (int)((int64_t)all * (part + 1) / parts);
  t.slot = a.slots ? a.slots[t.at] : -1;
  if (t.slot >= a.n_slots) t.slot = -1;
  if (Q4 && t.slot >= 0) {
    t.block = reinterpret_cast<uint32_t*>(a.blocks + block_of(t.slot, a.kv_heads, a.page_blocks) *
                                                         block4_bytes(a.groups));
    t.in = (int)(t.slot & 15);
  }
  if (a.half > 0 && s0 < sq + sk) {
    const uint64_t at = (uint64_t)((int64_t)a.positions[t.at] + a.shift);
    for (int i = lane; i < a.half; i += 32) {
      float2 z;  // cos, sin of the turn in [-1/2, 1/2)
      const float x = (float)(int32_t)(uint32_t)((at * a.turns[i]) >> 32) * 0x1p-31f;
      sincospif(x, &z.y, &z.x);
      s_turn[warp][i] = z;
    }
    __syncwarp();
  }
  if (s0 < sq)
    run_rows<T, L, Q4, kQueries>(a, t, s0 * kPer, min(a.heads, s1 * kPer), s_turn[warp], s_stage[warp]);
  if (s1 > sq && s0 < sq + sk)
    run_rows<T, L, Q4, kKeys>(a, t, max(s0 - sq, 0) * kPer, min(a.kv_heads, (s1 - sq) * kPer), s_turn[warp],
                              s_stage[warp]);
  if (s1 > sq + sk && t.slot >= 0)
    run_rows<T, L, Q4, kValues>(a, t, max(s0 - sq - sk, 0) * kPer, min(a.kv_heads, (s1 - sq - sk) * kPer),
                                s_turn[warp], s_stage[warp]);
}

// How many warps a token's `steps` go over: few tokens take as many as the SMs hold at once.
int64_t parts_of(int64_t tokens, int64_t steps) {
  const int64_t parts = 152 * 16 / tokens;
  return parts < 1 ? 1 : parts > steps ? steps : parts;
}

template <typename T, int L, bool Q4>
cudaError_t launch(const QkArgs& a, cudaStream_t stream) {
  constexpr int kPer = 32 / L;
  const int sk = (a.kv_heads + kPer - 1) / kPer;
  const int64_t steps = (a.heads + kPer - 1) / kPer + sk + (a.v.p ? sk : 0);
  const int64_t parts = parts_of(a.tokens, steps);
  const int64_t ctas = (a.tokens * parts + kWarps - 1) / kWarps;
  qk_kernel<T, L, Q4><<<(unsigned)ctas, kThreads, 0, stream>>>(a, (int)parts);
  return cudaGetLastError();
}

template <typename T, bool Q4>
cudaError_t launch_of(const QkArgs& a, cudaStream_t stream) {
  const int most = a.d > a.dv ? a.d : a.dv;
  if (most <= 64) return launch<T, 8, Q4>(a, stream);
  if (most <= 128) return launch<T, 16, Q4>(a, stream);
  return launch<T, 32, Q4>(a, stream);
}

// Rows of a 4-bit cache as the values they stand for; a slot outside it gives zeros.  Warps
// and lanes as above: a lane takes a code word.
template <typename T, int L>
__device__ __forceinline__ void read_rows(const Read4Args& a, const Token& t, bool values, int first, int end) {
  constexpr int kPer = 32 / L;
  const int lane = threadIdx.x & 31, l = lane & (L - 1), sub = lane / L;
  const Rows& to = values ? a.v : a.k;
  const int n = (values ? a.dv : a.d) - 8 * l;
  if (n <= 0) return;
  T* dst = static_cast<T*>(to.p) + t.at * to.row + 8 * l;
  const bool wide = is_wide<T>(to.p, to.row, to.head);
  const int g = l / 8, x = l & 7;
  const int word = values ? values4(a.groups) / 4 + value_word4(g, t.in, x) : key_word4(g, t.in, x);
  const int scale_at = (values ? value_scales4(a.groups) : key_scales4(a.groups)) / 4 + g * 16 + place4(t.in);
  const int64_t stride = (int64_t)a.page_blocks * (block4_bytes(a.groups) / 4);
#pragma unroll 4
  for (int h = first + sub; h < end; h += kPer) {
    uint32_t codes = 0, scale = 0;
    if (t.block) {
      codes = t.block[h * stride + word];
      scale = t.block[h * stride + scale_at];
    }
    const float step = __uint_as_float(scale & 0xffff0000u), mid = __uint_as_float(scale << 16);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)  // the product is exact: 8 + 4 bits
      y[i] = mid + step * (float)((int)(codes >> (4 * i) & 15) - 8);
    Eight<T> z;
    narrow8(y, z);
    put8(z, dst + h * to.head, n, wide);
  }
}

template <typename T, int L>
__global__ void __launch_bounds__(kThreads) read4_kernel(Read4Args a, int parts) {
  constexpr int kPer = 32 / L;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  Token t;
  t.at = parts == 1 ? w : w / parts;
  if (t.at >= a.tokens) return;
  const int part = (int)(w - t.at * parts), sk = (a.kv_heads + kPer - 1) / kPer;
  const int s0 = (int)((int64_t)2 * sk * part / parts), s1 = (int)((int64_t)2 * sk * (part + 1) / parts);
  t.slot = a.slots[t.at];
  t.block = nullptr;
  t.in = (int)(t.slot & 15);
  if (t.slot >= 0 && t.slot < a.n_slots)
    t.block = const_cast<uint32_t*>(reinterpret_cast<const uint32_t*>(
        a.blocks + block_of(t.slot, a.kv_heads, a.page_blocks) * block4_bytes(a.groups)));
  if (s0 < sk) read_rows<T, L>(a, t, false, s0 * kPer, min(a.kv_heads, s1 * kPer));
  if (s1 > sk) read_rows<T, L>(a, t, true, max(s0 - sk, 0) * kPer, min(a.kv_heads, (s1 - sk) * kPer));
}

template <typename T, int L>
cudaError_t launch_read(const Read4Args& a, cudaStream_t stream) {
  const int64_t parts = parts_of(a.tokens, 2 * ((a.kv_heads + 32 / L - 1) / (32 / L)));
  const int64_t ctas = (a.tokens * parts + kWarps - 1) / kWarps;
  read4_kernel<T, L><<<(unsigned)ctas, kThreads, 0, stream>>>(a, (int)parts);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_read_of(const Read4Args& a, cudaStream_t stream) {
  const int most = a.d > a.dv ? a.d : a.dv;
  if (most <= 64) return launch_read<T, 8>(a, stream);
  if (most <= 128) return launch_read<T, 16>(a, stream);
  return launch_read<T, 32>(a, stream);
}

}  // namespace

cudaError_t launch_qk(const QkArgs& a, cudaStream_t stream) {
  if (a.tokens == 0) return cudaSuccess;
  const bool q4 = a.blocks != nullptr;
  switch (a.dtype) {
    case NYS_F32: return q4 ? launch_of<float, true>(a, stream) : launch_of<float, false>(a, stream);
    case NYS_BF16:
      return q4 ? launch_of<__nv_bfloat16, true>(a, stream) : launch_of<__nv_bfloat16, false>(a, stream);
    default: return q4 ? launch_of<__half, true>(a, stream) : launch_of<__half, false>(a, stream);
  }
}

cudaError_t launch_read4(const Read4Args& a, cudaStream_t stream) {
  if (a.tokens == 0) return cudaSuccess;
  switch (a.dtype) {
    case NYS_F32: return launch_read_of<float>(a, stream);
    case NYS_BF16: return launch_read_of<__nv_bfloat16>(a, stream);
    default: return launch_read_of<__half>(a, stream);
  }
}

}  // namespace nys
