// One token of attention for each request over a paged cache in 4 bits (flash form):
//
//   s_j = (q . k_j) / sqrt d,  out = sum_j e^{s_j} v_j / sum_j e^{s_j},
//   k_j = mid + step * code in groups of 64 numbers, so that a group's part of q . k_j is
//   step * (q . code) + mid * sum(q), and its part of the output
//   sum_j (p_j step_j) code_j + sum_j p_j mid_j.
//
// The products are mma.sync m16n8k16 in f16: what is multiplied is 4-bit codes by at most 8 heads, so the
// 128-row tensor-memory form would be empty for the most part.  They take codes and never see a scale: keys'
// scales multiply a group's product, values' scales the weights.  The many go into the product's 16 rows (A:
// 16 tokens of keys, 16 numbers of values), the heads into its 8 columns (B): 4 products a block and group for
// the scores, 4 for the results.  Weights come out of the scores' product with a token a row and go into the
// other with a token a row of B, which movmatrix turns them to.
//
// Codes become f16 centred: keys' as c - 8, from 1024 + c less 1032 (bits 0-3) and 64 + c less 72 (bits 4-7),
// a mask and a difference for two, and a shift for every second byte; values' as 2c - 15, in the same way after a
// shift for every byte.  As they lie they are numbers too, c 2^-24 and c 2^-20, below the smallest normal one,
// which the matrix units take, and faster (128 requests as below: 82 us).  But the units cut every sum
// towards zero, and scores of such small numbers are off by 2e-6 of the row instead of 1e-7.  Sums of one sign
// over very many values show the cuts, because the result is small beside them: of codes as they lie 8e-4 of the
// result over 200,000 keys, of c - 8, which is -1/2 on average, 3e-5.  So values' codes have a mean of 0, as far as
// numbers lie evenly about a group's middle, and the products' sums end after 32 tokens, where f32 additions take
// them: 2e-7, as elsewhere (the two long requests as below 60 -> 61 us, the 128 91 -> 94; sums of c - 8 that end
// after 32 tokens were off by 2e-6).
//
// Queries of 16-bit types go in as they are, of f32 as two f16 pieces (22 bits), after a power of two that fits
// the row; the second pieces have products of their own.  Weights p_j step_j are two f16 pieces (22 bits) after
// a power of two that follows the largest step so far, so that a weight is held to 2^-35 of the largest.
// Columns are heads; where there are at most 4, the other columns are the weights' second pieces, for which there
// is a second product else; where at most 2, columns are halves of the groups too, so that a lane scales half of
// them.  Sums, maxima and the middles' part are f32.
//
// A warp works by itself: it streams pairs of blocks of 16 tokens (1,152 bytes a group of 64
// each) through a ring of its own in shared memory (three pairs; two of more than 192 numbers) with cp.async,
// and takes a range of one or more requests' blocks.  Ranges come from the lengths, on the GPU, by either of two rules:
// few (request, KV head) units are cut into pieces of up to 32 blocks for a CTA, whose warps join their
// results in shared memory; else the units are laid end to end and every warp takes an even share
// (joined in the CTA where all four are of one unit).  What cuts leave is joined by a second launch.
//
// What bounds it: instructions, not memory.  128 requests of 517 to 8,192 tokens, 16 heads over 8 of 128
// numbers, bf16 (412 MB): 94 us, 4.4 TB/s of the 6.7 of a copy; counters at such a size: ALU pipe 52%, tensor 24%,
// DRAM 58% busy.  2 requests of 131,075 and 200,000, 32 heads over 4 (191 MB): 61 us, 3.1 TB/s: 8 heads need the second
// products.  64 chats of 97 to 3,025 in f32 (65 MB): 35 us, where ranges are 20 blocks and start, drain and join
// weigh; 4 young requests: 8.5 us, a launch and one range's chain of loads.  64 of 517 to 8,192 with 8 heads over 1
// of 256 numbers (52 MB): 40 us, 1.3 TB/s: two pairs in the ring, so that a warp's copies and products take turns.
//
// Blocks outside the pool are zeros, tokens past the length have weight 0 whatever their
// bytes are.
#pragma once

#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nys_attn_tc.h"
#include "nys_kv4.h"

namespace nys {
namespace {

constexpr int kHeads = 8;       // heads of a unit
// Blocks of a warp's part of a CTA's piece, at most (4, 16 and 32, against 8: 4 young requests 10.1, 8.1, 8.1 and
// 8.0 us, one of 1,500 tokens 10.4, 12.6, 13.5 and 11.6).
constexpr int kPiece = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 5.f;    // weights stay below 2^kLazy of the followed maximum's
// Beyond this a product's rounding (2^-24 of it) may not be left in the difference to the maximum.
constexpr float kFar = 0x1p20f;
constexpr int kSms = 152;
constexpr float kLeastStep4 = 0x1p-100f;  // but for 0
constexpr uint32_t kUnits = 11;           // steps times up stay below 2^kUnits, weights (half of that) below 2^15

constexpr int kBoth = 2;        // blocks that are multiplied together: 32 tokens

template <int G>
struct Shape {
  static constexpr int kStages = G <= 3 ? 3 : 2;
  static constexpr int kStage = kBoth * block4_bytes(G);
  static constexpr int kRoom = kStages * kStage;  // of a warp
  // The query's rows go through one stage, and what a warp leaves (Left) takes the ring's place.
  static_assert(kStage >= kHeads * 64 * G * 4 && kStages >= 2, "a stage holds 8 rows of 64 G floats");
};
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// CTAs of an SM: as many as its registers take.
template <int G>
constexpr int kOfSm = G <= 2 ? 3 : 2;
constexpr int kPieceBlocks = kWarps * kPiece;

// Pieces of cut units: in the workspace, first the units' records, then each piece's
// [heads] maxima and sums, then its results [heads][64 G].
struct Cut4 {
  int32_t first, pieces;  // pieces < 0: the second rule's, -pieces of them
};
struct Work4 {
  Cut4* units;
  float2* sums;
  float* results;
  int32_t heads;  // of a piece
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool fill, bool here) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16, %2;\n\t}" ::"r"(
          dst),
      "l"(src), "r"(fill ? 16 : 0), "r"((uint32_t)here)
      : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(const unsigned char* at) { return *reinterpret_cast<const uint4*>(at); }
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// c = a b (first) or c + a b; first is known where loops are unrolled.
__device__ __forceinline__ void mma_f16(bool first, float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (first)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// (x & mask) | bits, less `less`: codes in the mantissas of a power of two, and whole numbers (a widely known step).
__device__ __forceinline__ uint32_t centred(uint32_t x, uint32_t mask, uint32_t bits, uint16_t less) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(mask), "r"(bits));
  const __half2 z = __hsub2(*reinterpret_cast<const __half2*>(&y), __half2half2(__ushort_as_half(less)));
  return *reinterpret_cast<const uint32_t*>(&z);
}
// The two codes at bits 0-3, and at bits 4-7, of the halves as f16, less 8: from 1024 + code less 1032, and
// 64 + code less 72.
__device__ __forceinline__ uint32_t low(uint32_t x) { return centred(x, 0x000f000fu, 0x64006400u, 0x6408); }
__device__ __forceinline__ uint32_t high(uint32_t x) { return centred(x, 0x00f000f0u, 0x54005400u, 0x5480); }
// Those of bits 1-4, and 5-8, less 7.5 and times 2: from 1024 + 2 code less 1039, and 64 + 2 code less 79.
__device__ __forceinline__ uint32_t twice_low(uint32_t x) { return centred(x, 0x001e001eu, 0x64006400u, 0x640f); }
__device__ __forceinline__ uint32_t twice_high(uint32_t x) { return centred(x, 0x01e001e0u, 0x54005400u, 0x54f0); }
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 z = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&z);
}
__device__ __forceinline__ Two unpack_f16(uint32_t x) {
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&x));
  return {y.x, y.y};
}
__device__ __forceinline__ float from_of(float m) { return m == -INFINITY ? 0.f : -m; }
__device__ __forceinline__ float step_of(uint32_t scale) { return __uint_as_float(scale & 0xffff0000u); }
__device__ __forceinline__ float mid_of(uint32_t scale) { return __uint_as_float(scale << 16); }

__device__ __forceinline__ float read_as(const void* p, int64_t i, int dtype) {
  return dtype == NYS_F32    ? static_cast<const float*>(p)[i]
         : dtype == NYS_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
                             : __half2float(static_cast<const __half*>(p)[i]);
}
// Four numbers at p + i: one word where that is aligned.
__device__ __forceinline__ float4 read4_as(const void* p, int64_t i, int dtype) {
  if (dtype == NYS_F32) {
    const float* x = static_cast<const float*>(p) + i;
    if (reinterpret_cast<uintptr_t>(x) % 16 == 0) return *reinterpret_cast<const float4*>(x);
  } else {
    const uint16_t* x = static_cast<const uint16_t*>(p) + i;
    if (reinterpret_cast<uintptr_t>(x) % 8 == 0) {
      const uint2 y = *reinterpret_cast<const uint2*>(x);
      if (dtype == NYS_BF16)
        return make_float4(__uint_as_float(y.x << 16), __uint_as_float(y.x & 0xffff0000u),
                           __uint_as_float(y.y << 16), __uint_as_float(y.y & 0xffff0000u));
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&y.x));
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&y.y));
      return make_float4(a.x, a.y, b.x, b.y);
    }
  }
  return make_float4(read_as(p, i, dtype), read_as(p, i + 1, dtype), read_as(p, i + 2, dtype),
                     read_as(p, i + 3, dtype));
}
__device__ __forceinline__ void write4_as(void* p, int64_t i, int dtype, float4 y) {
  if (dtype == NYS_F32) {
    float* x = static_cast<float*>(p) + i;
    if (reinterpret_cast<uintptr_t>(x) % 16 == 0) {
      *reinterpret_cast<float4*>(x) = y;
    } else {
      x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
    }
    return;
  }
  uint32_t lo, hi;
  if (dtype == NYS_BF16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(y.x, y.y), b = __floats2bfloat162_rn(y.z, y.w);
    lo = *reinterpret_cast<const uint32_t*>(&a);
    hi = *reinterpret_cast<const uint32_t*>(&b);
  } else {
    lo = pack_f16(y.x, y.y);
    hi = pack_f16(y.z, y.w);
  }
  uint16_t* x = static_cast<uint16_t*>(p) + i;
  if (reinterpret_cast<uintptr_t>(x) % 8 == 0) {
    *reinterpret_cast<uint2*>(x) = make_uint2(lo, hi);
  } else {
    x[0] = (uint16_t)lo, x[1] = (uint16_t)(lo >> 16), x[2] = (uint16_t)hi, x[3] = (uint16_t)(hi >> 16);
  }
}

// Request b's length, held inside its table, and its blocks (one at least: a request
// without keys is written too).
__device__ __forceinline__ int len_of(const Attn4Args& a, int b, bool report) {
  const int len = a.lens[b];
  const int64_t cap = (int64_t)a.width * a.page_blocks * kBlock4;
  if (report && (len < 0 || len > cap)) attn_report(a.status, NYS_ATTN_BAD_LENGTH);
  return len < 0 ? 0 : (int)(len > cap ? cap : len);
}
__device__ __forceinline__ int blocks_of(int len) { return len > 0 ? (len + kBlock4 - 1) / kBlock4 : 1; }

// What joins a result to the one over other keys: this one's and that one's factors and
// the log-sum of both, from the maximum (base 2) and the sum.
struct Joint {
  float mine, other, lse;
};
// (Its log-sum is read before anything is written, which may lie in the same place.)
__device__ __forceinline__ float first_sum(const Attn4Args& a, int b, int h) {
  return a.first.p ? a.first_lse[(int64_t)b * a.heads + h] * kLog2e : -INFINITY;
}
__device__ __forceinline__ Joint join_first(const Attn4Args& a, int b, float wide, float m, float l) {
  const float top = fmaxf(m, wide);
  // (The maximum passes over a log-sum of NaN, which has to arrive.)
  if (m == -INFINITY && wide == -INFINITY && l == 0.f) {
    // No keys; or all scores below what fp32 holds.
    const float nan = __uint_as_float(0x7fc00000u);
    return len_of(a, b, false) > 0 ? Joint{nan, 0.f, nan} : Joint{0.f, 0.f, -INFINITY};
  }
  const float mine = m == -INFINITY ? 0.f : exp2f(m - top);
  const float other = wide == -INFINITY ? 0.f : exp2f(wide - top);
  const float sum = l * mine + other;
  // (A sum of NaN leaves a factor of 0 alone: there may be no other result to read.)
  return {mine / sum, other == 0.f ? 0.f : other / sum, (top + log2f(sum)) * kLn2};
}
__device__ __forceinline__ void put_result(const Attn4Args& a, int b, int h, int c, float4 y,
                                           const Joint& z) {
  y.x *= z.mine, y.y *= z.mine, y.z *= z.mine, y.w *= z.mine;
  if (a.first.p && z.other != 0.f) {
    const float4 w = read4_as(a.first.p, b * a.first.row + h * a.first.head + c, a.dtype);
    y.x += z.other * w.x, y.y += z.other * w.y, y.z += z.other * w.z, y.w += z.other * w.w;
  }
  write4_as(a.out.p, b * a.out.row + h * a.out.head + c, a.dtype, y);
}

// What row r of the products is: a head; second pieces of weights from row 4 on (not of 5 to 8 heads);
// and, of up to 2 heads with more groups than one, groups g = slot + 2 x only.
enum Rows4 { kEight, kFour, kTwo };
template <int G, Rows4 R>
struct Lane {
  static constexpr int kHeadRows = R == kEight ? 8 : R == kFour ? 4 : 2;
  static constexpr int kSlots = R == kTwo ? 2 : 1;
  static constexpr int kOwn = (G + kSlots - 1) / kSlots;  // groups of a lane
  static __device__ __forceinline__ int head(int r) { return r & (kHeadRows - 1); }
  static __device__ __forceinline__ int slot(int r) { return R == kTwo ? r >> 1 & 1 : 0; }
};
// (A lane's place: r = lane / 4, c = lane % 4.  It makes the B operands of column r, and has the products'
// columns 2c and 2c + 1, whose slot is the same.)

// Query rows in pieces: this lane's B operands (of column r), and what goes with columns 2c and 2c + 1.
template <int G, Rows4 R, bool F32>
struct Query {
  uint32_t b[G][2][2][F32 ? 4 : 2];     // first pieces for low and high codes, then second ones
  float sum[Lane<G, R>::kOwn][2];       // of the own groups' numbers, in the products' units
  float scale[2];                       // of the scores, to base 2
};

// A unit's query rows on their way to shared memory: 4 numbers a lane and chunk, as they are or, where rows
// are not aligned to them, as f32.
template <int G, Rows4 R>
struct RawQuery {
  static constexpr int kChunks = Lane<G, R>::kHeadRows * G / 2 + (Lane<G, R>::kHeadRows * G % 2);
  uint4 w[kChunks];
  bool f32;
};
template <int G, Rows4 R>
__device__ __forceinline__ void load_query(RawQuery<G, R>& q, const Attn4Args& a, int b, int head0, int n_heads) {
  const int lane = threadIdx.x & 31, size = a.dtype == NYS_F32 ? 4 : 2;
  const char* row = static_cast<const char*>(a.q.p) + (b * a.q.row + head0 * a.q.head) * size;
  const bool word = ((reinterpret_cast<uintptr_t>(a.q.p) | (uintptr_t)(a.q.row * size) | (uintptr_t)(a.q.head * size)) &
                     (uintptr_t)(4 * size - 1)) == 0;
  q.f32 = a.dtype == NYS_F32 || !word;
#pragma unroll
  for (int k = 0; k < RawQuery<G, R>::kChunks; ++k) {
    const int i = lane + 32 * k, head = i / (16 * G), d = 4 * (i - head * 16 * G);
    q.w[k] = make_uint4(0, 0, 0, 0);
    if (head < n_heads && d < a.d) {
      const char* p = row + (head * a.q.head + d) * size;
      if (word && size == 4) {
        q.w[k] = *reinterpret_cast<const uint4*>(p);
      } else if (word) {
        const uint2 y = *reinterpret_cast<const uint2*>(p);
        q.w[k].x = y.x, q.w[k].y = y.y;
      }
    }
  }
  if (word) return;
#pragma unroll
  for (int k = 0; k < RawQuery<G, R>::kChunks; ++k) {
    const int i = lane + 32 * k, head = i / (16 * G), d = 4 * (i - head * 16 * G);
    if (head < n_heads && d < a.d) {
      const char* p = row + (head * a.q.head + d) * size;
      q.w[k] = make_uint4(__float_as_uint(read_as(p, 0, a.dtype)), __float_as_uint(read_as(p, 1, a.dtype)),
                          __float_as_uint(read_as(p, 2, a.dtype)), __float_as_uint(read_as(p, 3, a.dtype)));
    }
  }
}
// By way of `room` in shared memory (8 heads of 64 G numbers).
template <int G, Rows4 R, bool F32>
__device__ __forceinline__ void make_query(Query<G, R, F32>& q, const RawQuery<G, R>& raw, const Attn4Args& a,
                                           int n_heads, float* room) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int h = Lane<G, R>::head(r), slot = Lane<G, R>::slot(r);
#pragma unroll
  for (int k = 0; k < RawQuery<G, R>::kChunks; ++k) {
    uint4 y = raw.w[k];
    if (!raw.f32) {
      if (a.dtype == NYS_BF16) {
        y = make_uint4(y.x << 16, y.x & 0xffff0000u, y.y << 16, y.y & 0xffff0000u);
      } else {
        const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&y.x));
        const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&y.y));
        y = make_uint4(__float_as_uint(lo.x), __float_as_uint(lo.y), __float_as_uint(hi.x), __float_as_uint(hi.y));
      }
    }
    if (lane + 32 * k < Lane<G, R>::kHeadRows * 16 * G) *reinterpret_cast<uint4*>(room + 4 * (lane + 32 * k)) = y;
  }
  __syncwarp();
  float x[G][2][8];
  float most = 0.f;
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (h < n_heads) y = *reinterpret_cast<const float4*>(room + h * 64 * G + 64 * g + 32 * e + 8 * c + 4 * s);
        x[g][e][4 * s] = y.x, x[g][e][4 * s + 1] = y.y, x[g][e][4 * s + 2] = y.z, x[g][e][4 * s + 3] = y.w;
        most = largest(most, largest(fabsf(y.x), fabsf(y.y)), largest(fabsf(y.z), fabsf(y.w)));
      }
  most = largest(most, __shfl_xor_sync(0xffffffffu, most, 1));
  most = largest(most, __shfl_xor_sync(0xffffffffu, most, 2));
  // Numbers below 2^15, and a scale that is no subnormal number (of 0 it would make NaN of masked scores); a row
  // that is not finite, or whose units' factor is not, has no scores.
  constexpr int kOwn = Lane<G, R>::kOwn, kSlots = Lane<G, R>::kSlots;
  const int exp = (int)(__float_as_uint(most) >> 23 & 255);
  const float to_two = a.scale * kLog2e;
  const int fit = min(126, isfinite(to_two) ? 126 + ilogbf(to_two) : 126);
  const float up = __uint_as_float((uint32_t)(min(14 - (exp - 127), fit) + 127) << 23);
  float scale = to_two / up;
  if (exp == 255 || !isfinite(scale)) scale = __uint_as_float(0x7fc00000u);
  float sums[kOwn] = {};
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const bool own = g % kSlots == slot;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float y[8], low[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] = own ? x[g][e][i] * up : 0.f;
        sums[g / kSlots] += y[i];
        low[i] = (y[i] - __half2float(__float2half_rn(y[i]))) * 2048.f;
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          q.b[g][e][s][i] = pack_f16(y[2 * s + i], y[2 * s + i + 4]);
          if (F32) q.b[g][e][s][F32 ? 2 + i : 0] = pack_f16(low[2 * s + i], low[2 * s + i + 4]);
        }
    }
  }
#pragma unroll
  for (int o = 0; o < kOwn; ++o) {
    sums[o] += __shfl_xor_sync(0xffffffffu, sums[o], 1);
    sums[o] += __shfl_xor_sync(0xffffffffu, sums[o], 2);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // from the columns' lanes
    q.scale[i] = __shfl_sync(0xffffffffu, scale, 8 * c + 4 * i);
#pragma unroll
    for (int o = 0; o < kOwn; ++o) q.sum[o][i] = __shfl_sync(0xffffffffu, sums[o], 8 * c + 4 * i);
  }
}

// A token's scale word of group g, r = token % 8, of the first or second 8 of a block.
__device__ __forceinline__ uint32_t scale_at(const unsigned char* scales, int g, int r, int second) {
  return reinterpret_cast<const uint32_t*>(scales)[g * 16 + r / 2 * 4 + second * 2 + (r & 1)];
}

// Scores s[token r, r + 8][column 2c, 2c + 1] of a block, unscaled: the keys' codes are the product's A
// operand, 16 tokens, so that the block takes 4 products a group.
template <int G, Rows4 R, bool F32>
__device__ __forceinline__ void scores(const Query<G, R, F32>& q, const unsigned char* at, int lane, float (&s)[2][2]) {
  constexpr int kSlots = Lane<G, R>::kSlots, kOwn = Lane<G, R>::kOwn;
  const int r = lane >> 2, slot = Lane<G, R>::slot(2 * (lane & 3));
  s[0][0] = s[0][1] = s[1][0] = s[1][1] = 0.f;
#pragma unroll
  for (int o = 0; o < kOwn; ++o) {
    float acc[4], low_acc[4];
#pragma unroll
    for (int x = 0; x < kSlots; ++x) {
      const int g = o * kSlots + x;
      if (g >= G) continue;
      const uint4 k = lds128(at + g * 512 + lane * 16);
      const uint32_t words[2][2] = {{k.x, k.z}, {k.y, k.w}};  // [e][token r, r + 8]
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const uint32_t y0 = z ? words[e][0] >> 8 : words[e][0], y1 = z ? words[e][1] >> 8 : words[e][1];
          const uint32_t av[4] = {low(y0), low(y1), high(y0), high(y1)};
          const bool first = x == 0 && e == 0 && z == 0;
          mma_f16(first, acc, av, q.b[g][e][z][0], q.b[g][e][z][1]);
          if (F32) mma_f16(first, low_acc, av, q.b[g][e][z][F32 ? 2 : 0], q.b[g][e][z][F32 ? 3 : 0]);
        }
    }
    // (A last group that there is not: the column is 0, any scales do.)
    const int g = o * kSlots + (G % kSlots && o == kOwn - 1 ? 0 : slot);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint32_t word = scale_at(at + key_scales4(G), g, r, t);
      const float step = step_of(word), mid = mid_of(word);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float dot = F32 ? fmaf(low_acc[2 * t + i], 0x1p-11f, acc[2 * t + i]) : acc[2 * t + i];
        s[t][i] = fmaf(step, dot, fmaf(mid, q.sum[o][i], s[t][i]));
      }
    }
  }
  if (R == kTwo) {  // the other groups' columns
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) s[t][i] += __shfl_xor_sync(0xffffffffu, s[t][i], 1);
  }
}

// An 8 x 8 matrix of f16, a row over 4 lanes, turned round.
__device__ __forceinline__ uint32_t turned(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// What a warp leaves in shared memory of its range: results [heads][64 G] without the middles' part,
// that part [heads][G], and each head's maximum and sum.  (And a log-sum that was read before any
// is written, which may be in its place.)
template <int G>
struct Left {
  float result[kHeads][64 * G];
  float mid[kHeads][G];
  float2 sum[kHeads];
  float first[kHeads];  // the log-sum of what is joined in
};
template <int G>
constexpr bool left_fits = sizeof(Left<G>) <= Shape<G>::kRoom;
static_assert(left_fits<1> && left_fits<2> && left_fits<3> && left_fits<4>, "Left has a warp's ring");

// Blocks [t0, t1) of unit (b, kvh, heads h0 ..) -> `left`, which is the ring's place.
template <int G, Rows4 R, bool F32>
__device__ __forceinline__ void run_range(const Attn4Args& a, unsigned char* room, int b, int kvh, int h0,
                                          int t0, int t1) {
  constexpr int kStages = Shape<G>::kStages, kBytes = block4_bytes(G), kStage = Shape<G>::kStage;
  constexpr int kWords = kBytes / 16, kSlots = Lane<G, R>::kSlots, kOwn = Lane<G, R>::kOwn;
  constexpr bool kColumns = R != kEight;  // second pieces are columns of their own
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int slot = Lane<G, R>::slot(2 * c);
  const uint32_t ring = tc::sptr(room);
  const int len = len_of(a, b, false);
  const int n_heads = min(kHeads, a.group - h0);
  // Without keys the rows count as 0: what is no number in them would meet the masked scores.
  const int q_heads = len > 0 ? n_heads : 0;

  RawQuery<G, R> raw;
  load_query(raw, a, b, kvh * a.group + h0, q_heads);

  // The next block's page is looked up one block ahead; blocks that there are none of are zeros.  (A
  // request without keys has no table to look into.)
  const int end = min(t1, (len + kBlock4 - 1) / kBlock4);
  int next = t0, in_page = t0 % a.page_blocks;
  const int32_t* page_at = next < end ? a.table + (int64_t)b * a.width + t0 / a.page_blocks : a.lens;
  int ahead = *page_at;
  bool bad = false;
  const uint32_t head_bytes = a.page_blocks * kBytes, page_bytes = a.kv_heads * head_bytes;  // (below 2^31)
  const uint8_t* head_at = a.blocks + kvh * head_bytes + lane * 16;
  const auto fetch = [&](uint32_t dst) {
#pragma unroll
    for (int e = 0; e < kBoth; ++e) {
      const bool wanted = next < end, there = wanted && (uint32_t)ahead < (uint32_t)a.n_pages;
      bad |= wanted && !there;
      // (Of a page that there is not, nothing is read: any address does.)
      const uint8_t* src = head_at + (uint64_t)(there ? ahead : 0) * page_bytes + in_page * kBytes;
      ++next;
      const bool turn = ++in_page == a.page_blocks;
      in_page = turn ? 0 : in_page;
      page_at += turn && next < end ? 1 : 0;
      ahead = *page_at;
#pragma unroll
      for (int i = 0; i < kWords; i += 32)
        cp16(dst + e * kBytes + (i + lane) * 16, src + i * 16, there, i + 32 <= kWords || i + lane < kWords);
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(ring + i * kStage);

  Query<G, R, F32> q;
  make_query<G, R, F32>(q, raw, a, q_heads, reinterpret_cast<float*>(room + (kStages - 1) * kStage));

  // Results: numbers 64 g + 8 r + 2 x (elements 2, 3: and one more) by columns 2c, 2c + 1 of the
  // product.  For each of the two columns: the maximum, from where on it is followed, and this lane's tokens'
  // weights and their middles' part.
  float o[G][4][4] = {};
  float o_mid[kOwn][2];
  Two l = {0.f, 0.f};
  float m[2] = {-INFINITY, -INFINITY}, m_next[2] = {-INFINITY, -INFINITY};
  bool far = false;      // one of them is, so that scores are rounded as the maximum was before it is taken off
  float up[kOwn];        // weights are p step up / 2,
  uint32_t limit[kOwn];  // where steps are below this (their bits)
#pragma unroll
  for (int x = 0; x < kOwn; ++x) {
    o_mid[x][0] = o_mid[x][1] = 0.f;
    limit[x] = __float_as_uint(kLeastStep4);
    up[x] = 1.f;
  }
  int stage = 0;
  for (int t = t0; t < t1; t += kBoth) {
    cp_wait<kStages - 2>();
    __syncwarp();
    const unsigned char* at = room + stage * kStage;
    float s[kBoth][2][2];
#pragma unroll
    for (int e = 0; e < kBoth; ++e) scores<G, R, F32>(q, at + e * kBytes, lane, s[e]);
    uint32_t v_scales[kBoth][kOwn][2];
#pragma unroll
    for (int e = 0; e < kBoth; ++e)
#pragma unroll
      for (int x = 0; x < kOwn; ++x)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int g = x * kSlots + slot;
          v_scales[e][x][u] = 0;
          if (G % kSlots == 0 || g < G) v_scales[e][x][u] = scale_at(at + e * kBytes + value_scales4(G), g, r, u);
        }
    // Tokens past the length, and blocks that are another warp's.
    if (t + kBoth > t1 || len - t * kBlock4 < kBoth * kBlock4) {
#pragma unroll
      for (int e = 0; e < kBoth; ++e) {
        const int left = t + e < t1 ? len - (t + e) * kBlock4 : 0;
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (r + 8 * u >= left) {
            s[e][u][0] = s[e][u][1] = -INFINITY;
#pragma unroll
            for (int x = 0; x < kOwn; ++x) v_scales[e][x][u] = 0;
          }
      }
    }
    // Whether a lane's scores pass what is followed; the columns' maxima are looked for only then.
    float top[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = fmaxf(s[0][0][i], s[0][1][i]);
#pragma unroll
      for (int e = 1; e < kBoth; ++e) top[i] = fmaxf(top[i], fmaxf(s[e][0][i], s[e][1][i]));
      top[i] = __fmul_rn(top[i], q.scale[i]);
    }
    bool follow = top[0] > m_next[0] || top[1] > m_next[1];
    uint32_t steps[kOwn];
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
      steps[x] = 0;
#pragma unroll
      for (int e = 0; e < kBoth; ++e) steps[x] = max(steps[x], max(v_scales[e][x][0], v_scales[e][x][1]));
      follow |= steps[x] >= limit[x];
    }
    if (__any_sync(0xffffffffu, follow)) {
      float by[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int u = 4; u < 32; u <<= 1) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], u));
        const float now = top[i] > m_next[i] ? fmaxf(m[i], top[i]) : m[i];
        by[i] = m[i] == -INFINITY ? 0.f : exp2_fast(m[i] - now);
        m[i] = now;
        m_next[i] = __fadd_rd(now, kLazy);  // (no more than kLazy also where that is less than a unit of m)
      }
      l = mul(l, {by[0], by[1]});
      far = __any_sync(0xffffffffu, fabsf(from_of(m[0])) > kFar || fabsf(from_of(m[1])) > kFar);
#pragma unroll
      for (int x = 0; x < kOwn; ++x) {
        uint32_t most = steps[x];
#pragma unroll
        for (int u = 4; u < 32; u <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, u));
        // The next power of two; a step of NaN has a middle of NaN, which decides.
        float less = 1.f;
        if (most >= limit[x] && most < 0x7f800000u) {
          const uint32_t exp = (most >> 23) + 1;
          limit[x] = exp << 23;
          const float was = up[x];
          up[x] = __uint_as_float((127u + 127u + kUnits - exp) << 23);
          less = up[x] / was;
        }
        const float f0 = by[0] * less, f1 = by[1] * less;
        o_mid[x][0] *= by[0], o_mid[x][1] *= by[1];
#pragma unroll
        for (int g = x * kSlots; g < x * kSlots + kSlots && g < G; ++g)
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            o[g][z][0] *= f0, o[g][z][2] *= f0;
            o[g][z][1] *= f1, o[g][z][3] *= f1;
          }
      }
    }
    const float from[2] = {from_of(m[0]), from_of(m[1])};
#pragma unroll
    for (int e = 0; e < kBoth; ++e)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (far) {
          s[e][u][0] = __fadd_rn(__fmul_rn(s[e][u][0], q.scale[0]), from[0]);
          s[e][u][1] = __fadd_rn(__fmul_rn(s[e][u][1], q.scale[1]), from[1]);
        } else {
          fma({s[e][u][0], s[e][u][1]}, {q.scale[0], q.scale[1]}, {from[0], from[1]}).get(s[e][u][0], s[e][u][1]);
        }
        s[e][u][0] = exp2_fast(s[e][u][0]);
        s[e][u][1] = exp2_fast(s[e][u][1]);
        l = add(l, {s[e][u][0], s[e][u][1]});
      }
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
      uint32_t pb[kBoth][2][2];
#pragma unroll
      for (int e = 0; e < kBoth; ++e)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t word = v_scales[e][x][u];
          // Of codes less 7.5, for which the middle is half a step lower.
          const float mid = fmaf(-0.5f, step_of(word), mid_of(word)), f = step_of(word) * (0.5f * up[x]);
          o_mid[x][0] = fmaf(s[e][u][0], mid, o_mid[x][0]);
          o_mid[x][1] = fmaf(s[e][u][1], mid, o_mid[x][1]);
          const float x0 = s[e][u][0] * f, x1 = s[e][u][1] * f;
          uint32_t y = pack_f16(x0, x1);
          // The second piece: less what was taken (exact).
          const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&y));
          const uint32_t second = pack_f16(x0 - z.x, x1 - z.y);
          if (kColumns) y = c >= 2 ? second : y;
          pb[e][0][u] = turned(y);
          if (!kColumns) pb[e][1][u] = turned(second);
        }
#pragma unroll
      for (int g = x * kSlots; g < x * kSlots + kSlots && g < G; ++g) {
        float acc[4][4];
#pragma unroll
        for (int e = 0; e < kBoth; ++e) {
          const uint4 v = lds128(at + e * kBytes + values4(G) + g * 512 + lane * 16);
          const uint32_t va[2] = {__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632)};
          const uint32_t vb[2] = {__byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632)};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const uint32_t wa = z & 1 ? va[z / 2] >> 7 : va[z / 2] << 1, wb = z & 1 ? vb[z / 2] >> 7 : vb[z / 2] << 1;
            const uint32_t av[4] = {twice_low(wa), twice_high(wa), twice_low(wb), twice_high(wb)};
            // (Second pieces first: what is cut goes by the sum so far.)
            if (!kColumns) mma_f16(e == 0, acc[z], av, pb[e][1][0], pb[e][1][1]);
            mma_f16(kColumns && e == 0, acc[z], av, pb[e][0][0], pb[e][0][1]);
          }
        }
        // (Added up here, rounded to the nearest, not by the products.)
#pragma unroll
        for (int z = 0; z < 4; ++z)
#pragma unroll
          for (int i = 0; i < 4; i += 2)
            add({o[g][z][i], o[g][z][i + 1]}, {acc[z][i], acc[z][i + 1]}).get(o[g][z][i], o[g][z][i + 1]);
      }
    }
    __syncwarp();
    fetch(ring + (stage == 0 ? kStages - 1 : stage - 1) * kStage);
    stage = stage == kStages - 1 ? 0 : stage + 1;
  }
  cp_wait<0>();
  __syncwarp();
  if (bad && lane == 0) attn_report(a.status, NYS_ATTN_BAD_PAGE);

  // The ring is done with.
  Left<G>& left = *reinterpret_cast<Left<G>*>(room);
  const auto sum_of = [](float x) {
#pragma unroll
    for (int u = 4; u < 32; u <<= 1) x += __shfl_xor_sync(0xffffffffu, x, u);
    return x;
  };
  float sums[2];
  l.get(sums[0], sums[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int column = 2 * c + i, head = Lane<G, R>::head(column);
    const bool mine = head < n_heads && r == 0 && (!kColumns || column < 4);
    const float l_sum = sum_of(sums[i]);
    if (mine && slot == 0) {
      left.sum[head] = make_float2(m[i], l_sum);
      left.first[head] = first_sum(a, b, kvh * a.group + h0 + head);
    }
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
      const float y = sum_of(o_mid[x][i]);
      const int g = x * kSlots + slot;
      if (mine && g < G) left.mid[head][g] = y;
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const float down = 1.f / up[g / kSlots];  // (of columns whose slot has the group)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float y[8];
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        y[z] = o[g][z / 2][i + 2 * (z & 1)] * down;
        if (kColumns) y[z] += __shfl_xor_sync(0xffffffffu, y[z], 2);  // the second pieces' columns
      }
      const int column = 2 * c + i, h = Lane<G, R>::head(column);
      if (h < n_heads && (!kColumns || column < 4) && slot == g % kSlots) {
#pragma unroll
        for (int z = 0; z < 8; z += 4)
          *reinterpret_cast<float4*>(&left.result[h][64 * g + 8 * r + z]) =
              make_float4(y[z], y[z + 1], y[z + 2], y[z + 3]);
      }
    }
  }
}

// What `warps` warps left (Left, `apart` bytes apart) of one unit, joined by threads `thread` of
// `threads`: the final result (piece < 0) or piece `piece`.
template <int G>
__device__ __forceinline__ void emit(const Attn4Args& a, const Work4& w, const unsigned char* room, int apart, int warps,
                                     int b, int head0, int n_heads, int64_t piece, int thread, int threads) {
#pragma unroll 1
  for (int i = thread; i < n_heads * 16 * G; i += threads) {
    const int h = i / (16 * G), d = 4 * (i - h * 16 * G);
    float top = -INFINITY, l = 0.f;
    const float2* sums = &reinterpret_cast<const Left<G>*>(room)->sum[h];
#pragma unroll 4
    for (int x = 0; x < warps; ++x)
      top = fmaxf(top, reinterpret_cast<const float2*>(reinterpret_cast<const char*>(sums) + x * apart)->x);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = 0; x < warps; ++x) {
      const Left<G>& left = *reinterpret_cast<const Left<G>*>(room + x * apart);
      const float2 s = left.sum[h];
      // (A sum of NaN has any maximum, and has to arrive.)
      const float by = s.x == top ? 1.f : s.x == -INFINITY ? s.y : exp2_fast(s.x - top);
      const float4 z = *reinterpret_cast<const float4*>(&left.result[h][d]);
      const float mid = left.mid[h][d / 64];
      l = fmaf(s.y, by, l);
      y.x = fmaf(z.x + mid, by, y.x), y.y = fmaf(z.y + mid, by, y.y);
      y.z = fmaf(z.z + mid, by, y.z), y.w = fmaf(z.w + mid, by, y.w);
    }
    if (piece >= 0) {
      if (d == 0) w.sums[piece * w.heads + h] = make_float2(top, l);
      *reinterpret_cast<float4*>(w.results + (piece * w.heads + h) * (64 * G) + d) = y;
      continue;
    }
    const Joint z = join_first(a, b, reinterpret_cast<const Left<G>*>(room)->first[h], top, l);
    if (d < a.dv) put_result(a, b, head0 + h, d, y, z);
    if (a.lse && d == 0) a.lse[(int64_t)b * a.heads + head0 + h] = z.lse;
  }
}

template <int G, Rows4 R, bool F32>
__global__ void __launch_bounds__(kThreads, kOfSm<G>) attn4_kernel(Attn4Args a, Work4 w) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int kRoom = Shape<G>::kRoom;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tiles = (a.group + kHeads - 1) / kHeads, per_request = a.kv_heads * tiles;
  const int64_t units = (int64_t)a.n * per_request;
  let_next_start();

  // All blocks, which every warp counts for itself (no step of the CTA's: 128 lengths a round), and where
  // the prefix sum of `weight` passes x: the request, and the sum before it.
  const auto blocks_at = [&](int b, bool report) { return b < a.n ? blocks_of(len_of(a, b, report)) : 0; };
  int first[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) first[i] = blocks_at(4 * lane + i, blockIdx.x == 0 && warp == 0);
  int64_t sum = (int64_t)first[0] + first[1] + first[2] + first[3];
  for (int c0 = 128; c0 < a.n; c0 += 128)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += blocks_at(c0 + 4 * lane + i, blockIdx.x == 0 && warp == 0);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int64_t total = sum * per_request;
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  // The first rule: pieces of a CTA; the second: even shares of the warps, `share` blocks and one more in
  // the first `more` warps.
  const bool pieces = total / kPieceBlocks + units <= gridDim.x;
  const int64_t share = total > UINT32_MAX ? total / warps : (uint32_t)total / (uint32_t)warps;
  const int64_t more = total - share * warps;
  const int64_t first_warp = (int64_t)blockIdx.x * kWarps;
  // Where a warp begins, in pieces or in blocks.
  const auto begin_of = [&](int64_t i) { return i * share + (i < more ? i : more); };
  const auto find = [&](int64_t x, int64_t& before) {
    int64_t carry = 0;
    for (int c0 = 0; c0 < a.n; c0 += 128) {
      int64_t mine[4], all = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = c0 == 0 ? first[i] : blocks_at(c0 + 4 * lane + i, false);
        mine[i] = all;
        all += (int64_t)per_request * (pieces ? (t + kPieceBlocks - 1) / kPieceBlocks : t);
      }
      int64_t scan = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += y;
      }
      const int64_t from = carry + scan - all;
      const uint32_t here = __ballot_sync(0xffffffffu, x >= from && x < from + all);
      if (here) {
        int in = 0;
        int64_t to = from;
#pragma unroll
        for (int i = 1; i < 4; ++i)
          if (x >= from + mine[i] && 4 * lane + i + c0 < a.n) in = i, to = from + mine[i];
        const int who = __ffs(here) - 1;
        before = __shfl_sync(0xffffffffu, to, who);
        return c0 + 4 * who + __shfl_sync(0xffffffffu, in, who);
      }
      carry += __shfl_sync(0xffffffffu, scan, 31);
    }
    return -1;
  };
  // 64-bit numbers that are small, mostly.
  const auto div = [](int64_t x, int y) { return (int)(x <= UINT32_MAX ? (uint32_t)x / (uint32_t)y : x / y); };

  unsigned char* room = smem + warp * kRoom;
  int64_t x = pieces ? blockIdx.x : begin_of(first_warp), end = pieces ? x + 1 : begin_of(first_warp + kWarps), before = 0;
  if (x >= end) return;
  int b = find(x, before);
  if (b < 0) return;  // (the CTA's all, as what is left of a piece's CTA)
  int t = blocks_at(b, false);
  int64_t at = x - before;  // in request b
  // The second rule's warps of one unit join too: what the CTA has is inside a unit.
  const bool together = pieces || (share > 0 && end - x <= t - (at - (int64_t)div(at, t) * t));
  if (!together) {
    x = begin_of(first_warp + warp), end = begin_of(first_warp + warp + 1);
    if (x >= end) return;
    b = find(x, before);
    t = blocks_at(b, false);
    at = x - before;
  }
  const int np = pieces ? (t + kPieceBlocks - 1) / kPieceBlocks : 1;
  while (x < end) {
    // Unit u's blocks [lo, hi), this warp's of them [mine, mine_end).
    const int per = pieces ? np : t;
    const int u = div(at, per), i = (int)(at - (int64_t)u * per);
    int lo = i, hi = (int)(end - x < t - lo ? lo + (end - x) : t);
    if (pieces) {
      lo = (int)((int64_t)t * i / np);
      hi = (int)((int64_t)t * (i + 1) / np);
    }
    int mine = lo, mine_end = hi;
    if (together) {
      const int pairs = (hi - lo + 1) / 2;
      mine = lo + 2 * (pairs * warp / kWarps);
      mine_end = min(hi, lo + 2 * (pairs * (warp + 1) / kWarps));
    }
    const int kvh = u / tiles, h0 = (u - kvh * tiles) * kHeads;
    const bool whole = lo == 0 && hi == t;
    const int64_t id = together ? first_warp : first_warp + warp;
    // Where the unit's pieces are: x .. of the first rule; of the second 2 id + 1 in the first
    // warp that has some of it, 2 id in later ones.
    const int64_t piece = whole ? -1 : pieces ? x : lo == 0 ? 2 * id + 1 : 2 * id;
    if (w.units && lo == 0 && lane == 0 && (!together || warp == 0)) {
      int32_t count = np;
      if (!pieces && !whole) {
        const int64_t end_at = x + t, fat = more * (share + 1);  // the warp that has the unit's last block
        const int64_t last_id = end_at <= fat ? (end_at - 1) / (share + 1) : more + (end_at - 1 - fat) / share;
        count = -(int32_t)(last_id - id + 1);
      }
      w.units[(int64_t)b * per_request + u] = {(int32_t)(pieces ? x : 2 * id + 1), count};
    }
    run_range<G, R, F32>(a, room, b, kvh, h0, mine, mine_end);
    const int n_heads = min(kHeads, a.group - h0);
    if (together) __syncthreads();
    else __syncwarp();
    emit<G>(a, w, together ? smem : room, kRoom, together ? kWarps : 1, b, kvh * a.group + h0, n_heads, piece,
            together ? tid : lane, together ? kThreads : 32);
    if (together) {
      // The other warps' places among the unit's pieces hold nothing.
      if (!pieces && tid < (kWarps - 1) * n_heads) {
        const int64_t other = first_warp + 1 + tid / n_heads;
        w.sums[2 * other * w.heads + tid % n_heads] = make_float2(-INFINITY, 0.f);
      }
      return;
    }
    __syncwarp();
    x += hi - lo;
    at += hi - lo;
    if (at == (int64_t)t * per_request && x < end) {
      at = 0;
      t = blocks_of(len_of(a, ++b, false));
    }
  }
}

// Joins the pieces of cut units: a CTA's warps over one head's pieces, or (Alone: many heads, of few
// pieces each) a warp each.  A lane has numbers 4 lane .. of the head.
constexpr int kJoinWarps = 8;

template <int G, bool Alone>
__global__ void __launch_bounds__(kJoinWarps * 32) join4_kernel(Attn4Args a, Work4 w) {
  __shared__ float s_o[Alone ? 1 : kJoinWarps][64 * G];
  __shared__ float2 s_sum[kJoinWarps];
  constexpr int kEach = (G + 1) / 2;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tiles = (a.group + kHeads - 1) / kHeads, per_request = a.kv_heads * tiles;
  const int64_t rows = (int64_t)a.n * per_request * w.heads;
  const int64_t stride = Alone ? (int64_t)gridDim.x * kJoinWarps : gridDim.x;
  wait_for_previous();
  for (int64_t x = Alone ? (int64_t)blockIdx.x * kJoinWarps + warp : blockIdx.x; x < rows; x += stride) {
    const int64_t u = rows <= INT32_MAX ? (uint32_t)x / (uint32_t)w.heads : x / w.heads;
    const int h = (int)(x - u * w.heads);
    const Cut4 unit = w.units[u];
    if (unit.pieces == 1) continue;
    const int b = (int)(rows <= INT32_MAX ? (uint32_t)u / (uint32_t)per_request : u / per_request);
    const int in = (int)(u - (int64_t)b * per_request);
    const int kvh = in / tiles, h0 = (in - kvh * tiles) * kHeads;
    if (h0 + h >= a.group) continue;
    const int n = unit.pieces < 0 ? -unit.pieces : unit.pieces;
    const auto piece = [&](int i) {
      return (int64_t)(unit.pieces > 0 || i == 0 ? unit.first + i : unit.first + 2 * i - 1) * w.heads + h;
    };
    float top = -INFINITY;
    for (int i = Alone ? lane : tid; i < n; i += Alone ? 32 : kJoinWarps * 32) top = fmaxf(top, w.sums[piece(i)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!Alone) {
      __syncthreads();
      if (lane == 0) s_sum[warp].x = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kJoinWarps; ++i) top = fmaxf(top, s_sum[i].x);
    }
    const int head = kvh * a.group + h0 + h;
    // This warp's pieces [lo, hi): their weights a lane each, and then those that there are (a CTA's
    // warps that joined left one of four) four at a time.
    float4 o[kEach] = {};
    float l = 0.f;
    const int lo = Alone ? 0 : (int)((int64_t)n * warp / kJoinWarps);
    const int hi = Alone ? n : (int)((int64_t)n * (warp + 1) / kJoinWarps);
    for (int base = lo; base < hi; base += 32) {
      float by = 0.f;
      if (base + lane < hi) {
        const float2 s = w.sums[piece(base + lane)];
        by = s.x == -INFINITY ? s.y : exp2_fast(s.x - top);  // (of a sum of NaN: NaN)
        l += s.y * by;
      }
      uint32_t left = __ballot_sync(0xffffffffu, by != 0.f);
      while (left) {
        float4 y[4][kEach];
        float f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = left ? __ffs(left) - 1 : -1;
          left &= left - 1;
          f[k] = __shfl_sync(0xffffffffu, by, i < 0 ? 0 : i);
#pragma unroll
          for (int e = 0; e < kEach; ++e) {
            y[k][e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i >= 0 && 128 * e + 4 * lane < 64 * G)
              y[k][e] = *reinterpret_cast<const float4*>(w.results + piece(base + i) * (64 * G) + 128 * e + 4 * lane);
          }
          if (i < 0) f[k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int e = 0; e < kEach; ++e) {
            o[e].x = fmaf(y[k][e].x, f[k], o[e].x), o[e].y = fmaf(y[k][e].y, f[k], o[e].y);
            o[e].z = fmaf(y[k][e].z, f[k], o[e].z), o[e].w = fmaf(y[k][e].w, f[k], o[e].w);
          }
      }
    }
#pragma unroll
    for (int i = 16; i; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
    const float wide = first_sum(a, b, head);  // before any log-sum is written
    if (Alone) {
      __syncwarp();
      const Joint z = join_first(a, b, wide, top, l);
      if (a.lse && lane == 0) a.lse[(int64_t)b * a.heads + head] = z.lse;
#pragma unroll
      for (int e = 0; e < kEach; ++e)
        if (128 * e + 4 * lane < a.dv) put_result(a, b, head, 128 * e + 4 * lane, o[e], z);
      continue;
    }
    if (lane == 0) s_sum[warp].y = l;
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (128 * e + 4 * lane < 64 * G)
        *reinterpret_cast<float4*>(&s_o[Alone ? 0 : warp][128 * e + 4 * lane]) = o[e];
    __syncthreads();
    if (tid * 4 < 64 * G) {
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      l = 0.f;
#pragma unroll
      for (int i = 0; i < kJoinWarps; ++i) {
        const float4 z = *reinterpret_cast<const float4*>(&s_o[Alone ? 0 : i][4 * tid]);
        y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
        l += s_sum[i].y;
      }
      const Joint z = join_first(a, b, wide, top, l);
      if (a.lse && tid == 0) a.lse[(int64_t)b * a.heads + head] = z.lse;
      if (4 * tid < a.dv) put_result(a, b, head, 4 * tid, y, z);
    }
  }
}

struct Plan4 {
  unsigned ctas;
  int64_t units, pieces;  // pieces: 0 where no unit can be cut
  int heads;
};
template <int G>
Plan4 plan(int64_t n, int kv_heads, int group, int64_t keys) {
  Plan4 p;
  const int tiles = (group + kHeads - 1) / kHeads;
  p.units = n * kv_heads * tiles;
  p.heads = group < kHeads ? group : kHeads;
  const int64_t blocks = keys > kBlock4 ? (keys + kBlock4 - 1) / kBlock4 : 1;
  // CTAs that run at once; fewer only where the pieces of the longest requests need fewer.
  const int64_t most = kSms * kOfSm<G>;
  const int64_t cut = (blocks + kPieceBlocks - 1) / kPieceBlocks;
  const int64_t ctas = cut > most ? most : p.units * (cut + 1);
  p.ctas = (unsigned)(ctas < most ? ctas : most);
  // (Units of one piece, and a CTA more for each: the first rule, and no cut.)
  const bool never = cut == 1 && p.units * 2 <= p.ctas;
  p.pieces = never ? 0 : 2 * (int64_t)p.ctas * kWarps;
  return p;
}
Plan4 plan_of(int G, int64_t n, int kv_heads, int group, int64_t keys) {
  switch (G) {
    case 1: return plan<1>(n, kv_heads, group, keys);
    case 2: return plan<2>(n, kv_heads, group, keys);
    case 3: return plan<3>(n, kv_heads, group, keys);
    default: return plan<4>(n, kv_heads, group, keys);
  }
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

template <int G, Rows4 R, bool F32>
cudaError_t launch(const Attn4Args& a, void* workspace, cudaStream_t stream) {
  const Plan4 p = plan<G>(a.n, a.kv_heads, a.group, (int64_t)a.width * a.page_blocks * kBlock4);
  Work4 w{};
  w.heads = p.heads;
  if (p.pieces > 0) {
    unsigned char* at = static_cast<unsigned char*>(workspace);
    w.units = reinterpret_cast<Cut4*>(at);
    at += up256(p.units * sizeof(Cut4));
    w.sums = reinterpret_cast<float2*>(at);
    at += up256(p.pieces * p.heads * sizeof(float2));
    w.results = reinterpret_cast<float*>(at);
  }
  constexpr int kSmem = kWarps * Shape<G>::kRoom;
  cudaError_t e = ensure_smem<attn4_kernel<G, R, F32>>(kSmem);
  if (e != cudaSuccess) return e;
  attn4_kernel<G, R, F32><<<p.ctas, kThreads, kSmem, stream>>>(a, w);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.pieces == 0) return e;
  const int64_t rows = p.units * p.heads;
  // A CTA a head where there are few, of many pieces each (2 very long requests 61 us, a warp a head 74); a warp a
  // head else (128 requests of 517 to 8,192 94 us, a CTA a head 98).
  if (rows <= kSms * 4)
    return launch_dependent(join4_kernel<G, false>, dim3((unsigned)rows), kJoinWarps * 32, 0, stream, a, w);
  const int64_t ctas = (rows + kJoinWarps - 1) / kJoinWarps;
  return launch_dependent(join4_kernel<G, true>, dim3((unsigned)(ctas < kSms * 8 ? ctas : kSms * 8)), kJoinWarps * 32, 0,
                          stream, a, w);
}

template <int G, bool F32>
cudaError_t launch_of(const Attn4Args& a, void* workspace, cudaStream_t stream) {
  if (a.group > 4) return launch<G, kEight, F32>(a, workspace, stream);
  if (a.group > 2 || G == 1) return launch<G, kFour, F32>(a, workspace, stream);
  return launch<G, G == 1 ? kFour : kTwo, F32>(a, workspace, stream);
}
template <bool F32>
cudaError_t launch_any(const Attn4Args& a, void* workspace, cudaStream_t stream) {
  switch (groups4(a.d, a.dv)) {
    case 1: return launch_of<1, F32>(a, workspace, stream);
    case 2: return launch_of<2, F32>(a, workspace, stream);
    case 3: return launch_of<3, F32>(a, workspace, stream);
    default: return launch_of<4, F32>(a, workspace, stream);
  }
}

}  // namespace
}  // namespace nys
