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
// by position * 2^-65 turns for the rounding of F_i; its upper 32 bits, rounded to f32 (2^-25 of
// half a turn), go to sinpi and cospi.  (In f32 the angle of position 10^6 would be off by 0.06.)
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
// lies over 8, 16 or 32 lanes, two chunks of 4 numbers a lane: where half is a multiple
// of 4 those are the two sides of 4 pairs, so that no number leaves its lane; for 4 bits a
// row goes through shared memory once more, to 8 numbers in a row a lane, a code word.
//
// Measured: 16,384 tokens of 16 + 8 rows of 128 in f32 68 us (403 MB, 88% of a copy's rate), with the values
// into pages 89 us (537 MB, 90%); 32,768 of 32 + 4 in bf16 107 us (604 MB, 84%; issue slots 64% busy).  A part
// of each row turned with an odd half (4,099 tokens of 18 rows of 80, 26 pairs, fp16) 16 us for 24 MB: pairs go
// through shared memory, a warp makes one token and starts late.  4 bits are bound by instructions: 16,384
// tokens of 8 + 8 rows of 128 in bf16 34 us in (86 MB; issue slots 67% busy), 18 us out (ALU pipe 68%), in f32 36 and
// 39 us (153 MB); with 16 rows of queries, norm and rotation 68 us in bf16 (220 MB), 86 in f32 (422 MB).  One
// token, or 64: 3.3 to 4.2 us, the launch and one chain of loads.
#pragma once

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
// Pairs: none; numbers i and i + half, half a multiple of 4; 2i and 2i + 1; i and i + half, any half.
enum Turn { kNone, kSides, kNext, kOdd };
// Rows: 16-byte aligned and 8 numbers for each lane; every 4 numbers an aligned word; any.
enum Form { kWhole, kWords, kAny };
constexpr float kLeastStep = 0x1p-100f;

template <typename T>
struct alignas(4 * sizeof(T)) Four {
  T x[4];
};

// Four numbers widened, and back.
__device__ __forceinline__ void widen(const Four<float>& r, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = r.x[i];
}
__device__ __forceinline__ void widen(const Four<__nv_bfloat16>& r, float* x) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen(const Four<__half>& r, float* x) {
  const __half2* w = reinterpret_cast<const __half2*>(&r);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 y = __half22float2(w[i]);
    x[2 * i] = y.x;
    x[2 * i + 1] = y.y;
  }
}
__device__ __forceinline__ Four<float> narrow(const float* x, float) { return {x[0], x[1], x[2], x[3]}; }
__device__ __forceinline__ Four<__nv_bfloat16> narrow(const float* x, __nv_bfloat16) {
  Four<__nv_bfloat16> r;
  __nv_bfloat162* w = reinterpret_cast<__nv_bfloat162*>(&r);
  w[0] = __floats2bfloat162_rn(x[0], x[1]);
  w[1] = __floats2bfloat162_rn(x[2], x[3]);
  return r;
}
__device__ __forceinline__ Four<__half> narrow(const float* x, __half) {
  Four<__half> r;
  __half2* w = reinterpret_cast<__half2*>(&r);
  w[0] = __floats2half2_rn(x[0], x[1]);
  w[1] = __floats2half2_rn(x[2], x[3]);
  return r;
}

// A lane's two chunks of 4 numbers: at p + c0 and p + c1 (in0, in1: of the row; others are 0).
template <typename T, Form F, bool InARow>
__device__ __forceinline__ void get8(Four<T> (&r)[2], const T* p, int c0, int c1, bool in0, bool in1) {
  if (F == kWhole && InARow && sizeof(T) == 2) {
    uint4 y = make_uint4(0, 0, 0, 0);
    if (in0) y = *reinterpret_cast<const uint4*>(p + c0);
    *reinterpret_cast<uint2*>(&r[0]) = make_uint2(y.x, y.y);
    *reinterpret_cast<uint2*>(&r[1]) = make_uint2(y.z, y.w);
    return;
  }
  r[0] = r[1] = Four<T>{};
  if (F != kAny) {
    if (in0) r[0] = *reinterpret_cast<const Four<T>*>(p + c0);
    if (in1) r[1] = *reinterpret_cast<const Four<T>*>(p + c1);
  } else {
    if (in0) r[0] = {p[c0], p[c0 + 1], p[c0 + 2], p[c0 + 3]};
    if (in1) r[1] = {p[c1], p[c1 + 1], p[c1 + 2], p[c1 + 3]};
  }
}
template <typename T, Form F, bool InARow>
__device__ __forceinline__ void put8(const Four<T> (&r)[2], T* p, int c0, int c1, bool in0, bool in1) {
  if (F == kWhole && InARow && sizeof(T) == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(&r[0]), y = *reinterpret_cast<const uint2*>(&r[1]);
    if (in0) *reinterpret_cast<uint4*>(p + c0) = make_uint4(x.x, x.y, y.x, y.y);
    return;
  }
  if (F != kAny) {
    if (in0) *reinterpret_cast<Four<T>*>(p + c0) = r[0];
    if (in1) *reinterpret_cast<Four<T>*>(p + c1) = r[1];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (in0) p[c0 + i] = r[0].x[i];
      if (in1) p[c1 + i] = r[1].x[i];
    }
  }
}
// The form that rows have which start at p.
template <typename T>
Form form_of(const void* p, int64_t row, int64_t head, int dim, int lanes) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(p) | (uintptr_t)(row * sizeof(T)) | (uintptr_t)(head * sizeof(T));
  return all % 16 == 0 && dim == 8 * lanes ? kWhole : all % sizeof(Four<T>) == 0 ? kWords : kAny;
}

// x / by, rounded correctly, for inv = 1 / by rounded (Markstein), of a quotient that is
// no subnormal number.
__device__ __forceinline__ float quotient(float x, float by, float inv) {
  const float q = __fmul_rn(x, inv);
  return __fmaf_rn(__fmaf_rn(-q, by, x), inv, q);
}

// A group of 64 numbers over 8 lanes, the first n of 8 a lane (All: 8), to its scale word and
// this lane's 8 codes.
template <bool All>
__device__ __forceinline__ uint32_t quantize(const float (&y)[8], int n, uint32_t& scale) {
  float lo = INFINITY, hi = -INFINITY;
  if (All || n >= 8) {
    lo = least(least(y[0], y[1], y[2]), least(y[3], y[4], y[5]), least(y[6], y[7]));
    hi = largest(largest(y[0], y[1], y[2]), largest(y[3], y[4], y[5]), largest(y[6], y[7]));
  } else if (n >= 4) {
    lo = least(least(y[0], y[1]), y[2], y[3]);
    hi = largest(largest(y[0], y[1]), y[2], y[3]);
  }
#pragma unroll
  for (int o = 4; o; o >>= 1) {
    lo = least(lo, __shfl_xor_sync(0xffffffffu, lo, o, 8));
    hi = largest(hi, __shfl_xor_sync(0xffffffffu, hi, o, 8));
  }
  scale = 0;
  if (!All && lo > hi) return 0x88888888u;  // no numbers of the row
  const float span = __fmul_rn(__fsub_rn(hi, lo), 8.f);
  float part = quotient(span, 15.f, 1.f / 15.f);
  if (span < 0x1p-90f) part = __fdiv_rn(span, 15.f);
  const float sum = __fadd_rn(lo, part);
  const __nv_bfloat162 middle = __floats2bfloat162_rn(sum, sum);
  const uint32_t mid_bits = *reinterpret_cast<const uint32_t*>(&middle) & 0xffff0000u;
  const float mid = __uint_as_float(mid_bits);
  // (Quotients below 2^-102 make no step, whatever their last bits; above, Markstein's holds.)
  float step = largest(quotient(__fsub_rn(hi, mid), 7.f, 1.f / 7.f), __fmul_rn(__fsub_rn(mid, lo), 0.125f));
  step = __uint_as_float((__float_as_uint(step) + 0xffffu) & 0xffff0000u);
  const bool odd = !(fabsf(mid) < INFINITY) || !(step < INFINITY), none = step < kLeastStep;
  scale = odd ? 0x7fc07fc0u : (none ? 0u : __float_as_uint(step)) | mid_bits >> 16;
  if (odd || none) return 0x88888888u;
  const float inv = __frcp_rn(step);
  // t is in -8 .. 7 but for its rounding: t + 1.5 * 2^23 + 8 rounds it to a whole number, ties to
  // even, and has the code in its last bits; the bits above them add up to a constant.
  uint32_t codes = 0;
#pragma unroll
  for (int i = 6; i >= 0; i -= 2) {
    float a = 0.f, b = 0.f;
    if (All || n >= (i / 4 + 1) * 4) {
      const Two x = add({y[i], y[i + 1]}, {-mid, -mid}), q = mul(x, {inv, inv});
      const Two t = fma(fma(q, {-step, -step}, x), {inv, inv}, q);
      t.get(a, b);
    }
    float c, d;
    add({a, b}, {12582920.f, 12582920.f}).get(c, d);
    codes = (codes * 16 + __float_as_uint(d)) * 16 + __float_as_uint(c);
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

// Where a lane's two chunks of a row start.
struct Chunks {
  int at[2];
  bool pair;  // they are two sides
};
template <Turn R>
__device__ __forceinline__ Chunks chunks_of(int l, int half) {
  if (R == kSides) {
    const int over = l - half / 4;
    if (over < 0) return {{4 * l, half + 4 * l}, true};
    return {{2 * half + 8 * over, 2 * half + 8 * over + 4}, false};
  }
  return {{8 * l, 8 * l + 4}, false};
}
// Where the other number of the pair of number x = 8 l + i is, x / 8 further on for each
// number x so that a warp's numbers i are in banks of their own; less 9 l.
__device__ __forceinline__ int pair_at(int i, int half, bool is_first) {
  const int a = half / 8, b = half % 8;
  return is_first ? 9 * a + i + b + (i + b >= 8) : i - b - 9 * a - (i < b);
}

// Heads first + sub, first + sub + 32 / L, .. below end of one kind of rows.
template <typename T, int L, bool Q4, Turn R, Form F, Kind K>
__device__ __forceinline__ void run_rows(const QkArgs& a, const Token& t, int first, int end,
                                         const float2* turns, float* stage) {
  constexpr int kPer = 32 / L;
  // Steps whose loads are in flight, as many as 64 registers are good for.  1, 2, 3, 4: 64 prompts of 256 in f32 72,
  // 68, 72, 78 us; 32,768 tokens in bf16 139, 116, 109, 107; 16,384 into 4 bits and back 56, 51, 49, 50; pairs that
  // cross lanes (4,099 tokens, fp16) 14.8, 15.7, 16.1, 16.8.
  constexpr int kAhead = sizeof(T) == 4 || Q4 ? 2 : R == kOdd ? 3 : 4;
  constexpr Turn S = K == kValues ? kNone : R;
  constexpr bool kInARow = S != kSides;
  const int lane = threadIdx.x & 31, l = lane & (L - 1), sub = lane / L;
  const Rows& from = K == kQueries ? a.q : K == kKeys ? a.k : a.v;
  const Rows& to = K == kQueries ? a.q_out : a.k_out;
  const int dim = F == kWhole ? 8 * L : K == kValues ? a.dv : a.d;
  const int half = a.half;
  const Chunks c = chunks_of<S>(l, half);
  const bool in0 = F == kWhole || c.at[0] < dim, in1 = F == kWhole || c.at[1] < dim;
  const T* src = static_cast<const T*>(from.p) + t.at * from.row + (first + sub) * from.head;
  Four<T> raw[kAhead][2];
  auto load = [&](Four<T> (&r)[2], int h) {
    get8<T, F, kInARow>(r, src, c.at[0], c.at[1], h < end && in0, h < end && in1);
    src += kPer * from.head;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(raw[i], first + i * kPer + sub);

  // y_i = (x_i A_i + x_pair B_i) * inv.
  float fa[8], fb[8];
  float* mine = stage + sub * (9 * L + 1);  // this row's numbers, x at x + x / 8, and a 0 (kOdd)
  int pair[8];  // where the pairs' other numbers are there
  const float* weight = K == kQueries ? a.q_weight : a.k_weight;
  const bool turned[2] = {S == kSides ? c.pair : c.at[0] < 2 * half, S == kSides ? c.pair : c.at[1] < 2 * half};
  if (K != kValues) {
    const bool word = reinterpret_cast<uintptr_t>(weight) % 16 == 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float4 w = make_float4(1.f, 1.f, 1.f, 1.f);
      if (weight && (e == 0 ? in0 : in1)) {
        const float* p = weight + c.at[e];
        w = word ? *reinterpret_cast<const float4*>(p) : make_float4(p[0], p[1], p[2], p[3]);
      }
      fa[4 * e] = w.x, fa[4 * e + 1] = w.y, fa[4 * e + 2] = w.z, fa[4 * e + 3] = w.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) fb[i] = 0.f;
    if (S == kSides && c.pair) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 z = turns[4 * l + i];
        const float wa = fa[i], wb = fa[4 + i];
        fa[i] = wa * z.x;
        fb[i] = -(wb * z.y);
        fa[4 + i] = wb * z.x;
        fb[4 + i] = wa * z.y;
      }
    }
    if (S == kNext) {
#pragma unroll
      for (int i = 0; i < 8; i += 2)
        if (c.at[i / 4] + i % 4 < 2 * half) {
          const float2 z = turns[(c.at[i / 4] + i % 4) / 2];
          const float wa = fa[i], wb = fa[i + 1];
          fa[i] = wa * z.x;
          fb[i] = -(wb * z.y);
          fa[i + 1] = wb * z.x;
          fb[i + 1] = wa * z.y;
        }
    }
    if (S == kOdd) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) mine[9 * l + i] = fa[i];
      if (l == 0) mine[9 * L] = 0.f;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int x = 8 * l + i;
        pair[i] = x < 2 * half ? 9 * l + pair_at(i, half, x < half) : 9 * L;
        asm volatile("" : "+r"(pair[i]));  // (is kept, not made again for every row)
        if (x < 2 * half) {
          const float2 z = turns[x < half ? x : x - half];
          const float wp = mine[pair[i]];
          fa[i] *= z.x;
          fb[i] = x < half ? -(wp * z.y) : wp * z.y;
        }
      }
    }
  }
  const float inv_d = 1.f / (float)a.d;
  T* dst = to.p && K != kValues ? static_cast<T*>(to.p) + t.at * to.row + (first + sub) * to.head : nullptr;
  uint32_t* block = t.block + (int64_t)(first + sub) * a.page_blocks * (block4_bytes(a.groups) / 4);
  const int block_step = kPer * a.page_blocks * (block4_bytes(a.groups) / 4);
  const int code_at = K == kValues ? values4(a.groups) / 4 + value_word4(l / 8, t.in, l & 7) : key_word4(l / 8, t.in, l & 7);
  const int scale_at =
      (K == kValues ? value_scales4(a.groups) : key_scales4(a.groups)) / 4 + l / 8 * 16 + place4(t.in);
  T* page = nullptr;
  if (!Q4 && K != kQueries && t.slot >= 0)
    page = static_cast<T*>(K == kValues ? a.pool_v : a.pool_k) + (t.slot * a.kv_heads + first + sub) * dim;

  for (int base = first; base < end; base += kAhead * kPer) {
#pragma unroll
    for (int b = 0; b < kAhead; ++b) {
      const int h = base + b * kPer + sub;
      if (h - sub >= end) break;
      const bool row = kPer == 1 || h < end;
      if (K == kValues && !Q4) {
        put8<T, F, true>(raw[b], page, c.at[0], c.at[1], row && in0, row && in1);
        page += kPer * dim;
      } else {
        float y[8];
        widen(raw[b][0], y);
        widen(raw[b][1], y + 4);
        if (K != kValues) {
          float inv = 1.f;
          if (weight) {
            Two sums = mul({y[0], y[1]}, {y[0], y[1]});
#pragma unroll
            for (int i = 2; i < 8; i += 2) sums = fma({y[i], y[i + 1]}, {y[i], y[i + 1]}, sums);
            float ss, other;
            sums.get(ss, other);
            ss += other;
#pragma unroll
            for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, L);
            inv = rsqrtf(fmaf(ss, inv_d, a.eps));
          }
          float p[8];  // the other numbers of the pairs
          if (S == kSides || S == kNext) {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = y[S == kSides ? i ^ 4 : i ^ 1];
          } else if (S == kOdd) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) mine[9 * l + i] = y[i];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = mine[pair[i]];
          }
          // (Beyond 2 half there is no pair: what lies in its place may be infinite.)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (S == kOdd || (S != kNone && turned[e])) {
              if (S == kNext && !(c.at[e] + 2 < 2 * half)) p[4 * e + 2] = p[4 * e + 3] = 0.f;
#pragma unroll
              for (int i = 4 * e; i < 4 * e + 4; i += 2) {
                const Two z = mul({p[i], p[i + 1]}, {fb[i], fb[i + 1]});
                mul(fma({y[i], y[i + 1]}, {fa[i], fa[i + 1]}, z), {inv, inv}).get(y[i], y[i + 1]);
              }
            } else {
#pragma unroll
              for (int i = 4 * e; i < 4 * e + 4; i += 2)
                mul(mul({y[i], y[i + 1]}, {fa[i], fa[i + 1]}), {inv, inv}).get(y[i], y[i + 1]);
            }
          }
          const Four<T> z[2] = {narrow(y, T{}), narrow(y + 4, T{})};
          if (dst) {
            put8<T, F, kInARow>(z, dst, c.at[0], c.at[1], row && in0, row && in1);
            dst += kPer * to.head;
          }
          if (page) {
            put8<T, F, kInARow>(z, page, c.at[0], c.at[1], row && in0, row && in1);
            page += kPer * dim;
          }
        }
        if (Q4 && K != kQueries && t.slot >= 0) {
          const int n = dim - 8 * l;
          if (!kInARow) {  // from two sides to 8 numbers in a row
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (i == 0 ? in0 : in1)
                *reinterpret_cast<float4*>(stage + sub * 8 * L + c.at[i]) =
                    make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float4 z = *reinterpret_cast<const float4*>(stage + sub * 8 * L + 8 * l + 4 * i);
              y[4 * i] = z.x, y[4 * i + 1] = z.y, y[4 * i + 2] = z.z, y[4 * i + 3] = z.w;
            }
          }
          uint32_t scale;
          const uint32_t codes = quantize<F == kWhole>(y, n, scale);
          if (row && l / 8 < a.groups) {
            block[code_at] = codes;
            if ((l & 7) == 0) block[scale_at] = scale;
          }
          block += block_step;
        }
      }
      load(raw[b], h + kAhead * kPer);
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

// A warp takes part `w % parts` of token w / parts's steps of 32 / L rows.  4 CTAs an SM, for which forms that
// rotate spill 16 to 120 bytes a thread; with 3, where few spill and less, f32 prompts took 66.8 us instead of 67.7,
// but bf16 ones 115 instead of 107, 4 bits 55 instead of 51.
template <typename T, int L, bool Q4, Turn R, Form F>
__global__ void __launch_bounds__(kThreads, 4) qk_kernel(QkArgs a, int parts) {
  constexpr int kPer = 32 / L;
  __shared__ __align__(16) float2 s_turn[kWarps][kMaxHalf];
  __shared__ __align__(16) float s_stage[kWarps][292];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
  Token t{};
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
  if (R != kNone && s0 < sq + sk) {
    const uint64_t at = (uint64_t)((int64_t)a.positions[t.at] + a.shift);
    for (int i = lane; i < a.half; i += 32) {
      float2 z;  // cos, sin of the turn in [-1/2, 1/2)
      const float x = (float)(int32_t)(uint32_t)((at * a.turns[i]) >> 32) * 0x1p-31f;
      sincospif(x, &z.y, &z.x);
      s_turn[warp][i] = z;
    }
    __syncwarp();
  }
  float* stage = s_stage[warp];
  if (s0 < sq)
    run_rows<T, L, Q4, R, F, kQueries>(a, t, s0 * kPer, min(a.heads, s1 * kPer), s_turn[warp], stage);
  if (s1 > sq && s0 < sq + sk)
    run_rows<T, L, Q4, R, F, kKeys>(a, t, max(s0 - sq, 0) * kPer, min(a.kv_heads, (s1 - sq) * kPer), s_turn[warp],
                                 stage);
  if (s1 > sq + sk && t.slot >= 0)
    run_rows<T, L, Q4, R, F, kValues>(a, t, max(s0 - sq - sk, 0) * kPer, min(a.kv_heads, (s1 - sq - sk) * kPer),
                                   s_turn[warp], stage);
}

// How many warps a token's `steps` go over: one where the tokens fill the SMs (more would make
// each token's factors more than once: 4,099 tokens of 18 rows of 80, fp16, 21 -> 23 us with
// two, 16,576 rows of 2,048 numbers read from 4 bits 24 -> 30 us).
int64_t parts_of(int64_t tokens, int64_t steps) {
  const int64_t parts = 152 * 32 / tokens;
  return parts < 1 ? 1 : parts > steps ? steps : parts;
}

template <typename T, int L, bool Q4, Form F>
cudaError_t launch(const QkArgs& a, cudaStream_t stream) {
  constexpr int kPer = 32 / L;
  const int sk = (a.kv_heads + kPer - 1) / kPer;
  const int parts = (int)parts_of(a.tokens, (a.heads + kPer - 1) / kPer + sk + (a.v.p ? sk : 0));
  const unsigned ctas = (unsigned)((a.tokens * parts + kWarps - 1) / kWarps);
  if (a.half == 0) qk_kernel<T, L, Q4, kNone, F><<<ctas, kThreads, 0, stream>>>(a, parts);
  else if (a.interleaved) qk_kernel<T, L, Q4, kNext, F><<<ctas, kThreads, 0, stream>>>(a, parts);
  else if (a.half % 4 == 0) qk_kernel<T, L, Q4, kSides, F><<<ctas, kThreads, 0, stream>>>(a, parts);
  else qk_kernel<T, L, Q4, kOdd, F == kWhole ? kWords : F><<<ctas, kThreads, 0, stream>>>(a, parts);
  return cudaGetLastError();
}

template <typename T, bool Q4>
cudaError_t launch_of(const QkArgs& a, cudaStream_t stream) {
  const int most = a.d > a.dv ? a.d : a.dv;
  const int lanes = most <= 64 ? 8 : most <= 128 ? 16 : 32;
  Form form = a.v.p && a.dv != a.d ? kWords : kWhole;
  const auto take = [&](const Rows& r, int dim) {
    if (!r.p) return;
    const Form f = form_of<T>(r.p, r.row, r.head, dim, lanes);
    form = form > f ? form : f;
  };
  take(a.q, a.d);
  take(a.k, a.d);
  take(a.v, a.dv);
  take(a.q_out, a.d);
  take(a.k_out, a.d);
  take({a.pool_k, a.d, a.d}, a.d);
  take({a.pool_v, a.dv, a.dv}, a.dv);
  // (Rows of no alignment take 32 lanes, whatever their length.)
  if (form == kAny) return launch<T, 32, Q4, kAny>(a, stream);
  if (lanes == 8) return form == kWhole ? launch<T, 8, Q4, kWhole>(a, stream) : launch<T, 8, Q4, kWords>(a, stream);
  if (lanes == 16) return form == kWhole ? launch<T, 16, Q4, kWhole>(a, stream) : launch<T, 16, Q4, kWords>(a, stream);
  return form == kWhole ? launch<T, 32, Q4, kWhole>(a, stream) : launch<T, 32, Q4, kWords>(a, stream);
}

// Rows of a 4-bit cache as the values they stand for; a slot outside it gives zeros.  Warps
// and lanes as above: a lane takes a code word of keys and one of values, four heads at a time, all their loads
// before the first is used (scattered words of 4 bytes: a token's lie 16 or 64 bytes apart).  16,384 tokens of 8
// rows in and out, two, four, eight heads at a time: 51.0, 51.2, 54.5 us.
template <typename T, int L, Form F>
__global__ void __launch_bounds__(kThreads) read4_kernel(Read4Args a, int parts) {
  constexpr int kPer = 32 / L, kHeads = 4;
  const int lane = threadIdx.x & 31, l = lane & (L - 1), sub = lane / L;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t at = parts == 1 ? w : w / parts;
  if (at >= a.tokens) return;
  const int part = (int)(w - at * parts), steps = (a.kv_heads + kPer - 1) / kPer;
  const int first = steps * part / parts * kPer, end = min(a.kv_heads, steps * (part + 1) / parts * kPer);
  const int64_t slot = a.slots[at];
  const bool there = slot >= 0 && slot < a.n_slots;
  const uint32_t* block = reinterpret_cast<const uint32_t*>(
      a.blocks + (there ? block_of(slot, a.kv_heads, a.page_blocks) * block4_bytes(a.groups) : 0));
  const int in = (int)(slot & 15), g = l / 8, x = l & 7;
  const int64_t stride = (int64_t)a.page_blocks * (block4_bytes(a.groups) / 4);
  const int n[2] = {a.d - 8 * l, a.dv - 8 * l};
  const int code_at[2] = {key_word4(g, in, x), values4(a.groups) / 4 + value_word4(g, in, x)};
  const int scale_at[2] = {key_scales4(a.groups) / 4 + g * 16 + place4(in),
                           value_scales4(a.groups) / 4 + g * 16 + place4(in)};
  T* dst[2] = {static_cast<T*>(a.k.p) + at * a.k.row + 8 * l, static_cast<T*>(a.v.p) + at * a.v.row + 8 * l};
#pragma unroll 1
  for (int base = first; base < end; base += kHeads * kPer) {
    uint32_t codes[kHeads][2], scale[kHeads][2];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int h = base + i * kPer + sub;
        codes[i][k] = scale[i][k] = 0;
        if (there && h < end && n[k] > 0) {
          codes[i][k] = block[h * stride + code_at[k]];
          scale[i][k] = block[h * stride + scale_at[k]];
        }
      }
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int h = base + i * kPer + sub;
        if (h - sub >= end) continue;
        const float step = __uint_as_float(scale[i][k] & 0xffff0000u), mid = __uint_as_float(scale[i][k] << 16);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          // 2^23 + code, less 2^23 + 8; the product is exact: 8 + 4 bits.
          const uint32_t c = e == 0 ? codes[i][k] : codes[i][k] >> (4 * e);
          const Two z = add({__uint_as_float((c & 15u) | 0x4b000000u), __uint_as_float((c >> 4 & 15u) | 0x4b000000u)},
                            {-8388616.f, -8388616.f});
          fma({step, step}, z, {mid, mid}).get(y[e], y[e + 1]);
        }
        const Four<T> z[2] = {narrow(y, T{}), narrow(y + 4, T{})};
        if (h < end && n[k] > 0)
          put8<T, F, true>(z, dst[k] + h * (k ? a.v.head : a.k.head), 0, 4, true, n[k] > 4);
      }
  }
}

template <typename T, int L, Form F>
cudaError_t launch_read(const Read4Args& a, cudaStream_t stream) {
  const int64_t parts = parts_of(a.tokens, (a.kv_heads + 32 / L - 1) / (32 / L));
  const int64_t ctas = (a.tokens * parts + kWarps - 1) / kWarps;
  read4_kernel<T, L, F><<<(unsigned)ctas, kThreads, 0, stream>>>(a, (int)parts);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_read_of(const Read4Args& a, cudaStream_t stream) {
  const int most = a.d > a.dv ? a.d : a.dv;
  const int lanes = most <= 64 ? 8 : most <= 128 ? 16 : 32;
  const Form k = form_of<T>(a.k.p, a.k.row, a.k.head, a.d, lanes);
  const Form v = form_of<T>(a.v.p, a.v.row, a.v.head, a.dv, lanes);
  const Form form = k > v ? k : v;
  if (form == kAny) return launch_read<T, 32, kAny>(a, stream);
  if (lanes == 8) return form == kWhole ? launch_read<T, 8, kWhole>(a, stream) : launch_read<T, 8, kWords>(a, stream);
  if (lanes == 16)
    return form == kWhole ? launch_read<T, 16, kWhole>(a, stream) : launch_read<T, 16, kWords>(a, stream);
  return form == kWhole ? launch_read<T, 32, kWhole>(a, stream) : launch_read<T, 32, kWords>(a, stream);
}

}  // namespace
}  // namespace nys
