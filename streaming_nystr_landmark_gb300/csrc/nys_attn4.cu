// One token of attention for each request over a paged cache in 4 bits (flash form):
//
//   s_j = (q . k_j) / sqrt d,  out = sum_j e^{s_j} v_j / sum_j e^{s_j},
//   k_j = mid + step * code in groups of 64 numbers, so that a group's part of q . k_j is
//   step * (q . code) + mid * sum(q), and its part of the output
//   sum_j (p_j step_j) code_j + sum_j p_j mid_j.
//
// The products take codes (whole numbers from -8 to 7, exact in 16 bits) and never see a
// scale: keys' scales multiply a group's product, values' scales the weights.  q goes in
// as two fp16 pieces (22 bits, after a power of two that fits its row), which are rows
// 0-7 and 8-15 of mma.sync m16n8k16; weights go in as two bf16 pieces (16 bits), in f32
// calls three.  Sums, maxima and the middles' part are f32.  A group of up to 8 heads
// fills the products' 8 columns at best, and memory sets the time: the 128-row
// tensor-memory form would be empty for the most part.
//
// A warp works by itself: it streams blocks of 16 tokens (1,152 bytes a group of 64) through
// a ring of its own in shared memory with cp.async, and takes a range of one or more
// requests' blocks.  Ranges come from the lengths, on the GPU, by either of two rules:
// few (request, KV head) units are cut evenly into as many pieces as there are warps for;
// many units are laid end to end and every warp takes an even share.  What cuts leave is
// joined by a second launch.
//
// Blocks outside the pool are zeros, tokens past the length have weight 0 whatever their
// bytes are.
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nys_attn_tc.h"
#include "nys_kv4.h"

namespace nys {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kHeads = 8;       // heads of a unit
constexpr int kLeast = 8;       // blocks of a piece of a cut unit, at least
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.f;
constexpr int kSms = 152;

template <int G>
struct Shape {
  static constexpr int kStages = G <= 2 ? 4 : 3;
  static constexpr int kCtas = G <= 2 ? 4 : G == 3 ? 3 : 2;  // of an SM
  static constexpr int kSmem = kWarps * kStages * block4_bytes(G);
};

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

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool fill) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(fill ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(at)
               : "memory");
  return x;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// (x & mask) | bits: a code into the mantissa of a power of two.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(mask), "r"(bits));
  return y;
}
// The two codes at bits 0-3 of the halves as fp16 code - 8: 1024 + code, less 1032.
__device__ __forceinline__ uint32_t low_f16(uint32_t x) {
  const uint32_t y = and_or(x, 0x000f000fu, 0x64006400u);
  const __half2 z = __hsub2(*reinterpret_cast<const __half2*>(&y), __half2half2(__ushort_as_half(0x6408)));
  return *reinterpret_cast<const uint32_t*>(&z);
}
// The two at bits 4-7: 64 + code, less 72.
__device__ __forceinline__ uint32_t high_f16(uint32_t x) {
  const uint32_t y = and_or(x, 0x00f000f0u, 0x54005400u);
  const __half2 z = __hsub2(*reinterpret_cast<const __half2*>(&y), __half2half2(__ushort_as_half(0x5480)));
  return *reinterpret_cast<const uint32_t*>(&z);
}
// The two at bits 0-3 as bf16: 128 + code, less 136.
__device__ __forceinline__ uint32_t low_bf16(uint32_t x) {
  const uint32_t y = and_or(x, 0x000f000fu, 0x43004300u);
  const __nv_bfloat162 z = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&y),
                                   __bfloat162bfloat162(__ushort_as_bfloat16(0x4308)));
  return *reinterpret_cast<const uint32_t*>(&z);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 z = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&z);
}
// Two numbers as bf16, which are taken off them.
__device__ __forceinline__ uint32_t take_bf16(float& lo, float& hi) {
  const __nv_bfloat162 z = __floats2bfloat162_rn(lo, hi);
  const uint32_t y = *reinterpret_cast<const uint32_t*>(&z);
  lo -= __uint_as_float(y << 16);
  hi -= __uint_as_float(y & 0xffff0000u);
  return y;
}
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
__device__ __forceinline__ Joint join_first(float wide, float m, float l) {
  const float top = fmaxf(m, wide);
  if (top == -INFINITY && l == 0.f) return {0.f, 0.f, -INFINITY};
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

// Blocks [t0, t1) of unit (b, kvh, heads h0 ..) -> the final result, or piece `piece`.
template <int G, bool F32>
__device__ __forceinline__ void run_range(const Attn4Args& a, const Work4& w, uint32_t ring, int b,
                                          int kvh, int h0, int t0, int t1, int piece) {
  constexpr int kStages = Shape<G>::kStages, kBytes = block4_bytes(G);
  constexpr int kWords = kBytes / 16;
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int len = len_of(a, b, false);
  const int32_t* pages = a.table + (int64_t)b * a.width;
  const int n_heads = min(kHeads, a.group - h0);
  const int head0 = kvh * a.group + h0;

  // Block t's place; the page's number is looked up one block ahead.
  auto page_of = [&](int t) {
    if (t >= t1 || t * kBlock4 >= len) return -1;
    const int32_t pg = pages[t / a.page_blocks];
    if (pg < 0 || pg >= a.n_pages) {
      if (lane == 0) attn_report(a.status, NYS_ATTN_BAD_PAGE);
      return -1;
    }
    return pg;
  };
  int ahead = page_of(t0);
  auto fetch = [&](int t, int stage) {
    const int pg = ahead;
    ahead = page_of(t + 1);
    if (t < t1) {
      const uint8_t* src = a.blocks;
      if (pg >= 0)
        src += (((int64_t)pg * a.kv_heads + kvh) * a.page_blocks + t % a.page_blocks) * kBytes;
      const uint32_t dst = ring + stage * kBytes;
#pragma unroll
      for (int i = 0; i < kWords; i += 32)
        if (i + 32 <= kWords || i + lane < kWords)
          cp16(dst + (i + lane) * 16, src + (i + lane) * 16, pg >= 0);
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(t0 + i, i);

  // The query: pieces of its row's numbers times a power of two, and their sums.
  uint32_t qa[G][2][2][4];
  float q_sum[G];
  float scale;
  {
    float4 x[G][2][2];
    float most = 0.f;
    const bool mine = r < n_heads;
    const int64_t at = b * a.q.row + (head0 + r) * a.q.head;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int d = 64 * g + 32 * h + 8 * c + 4 * s;
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
          if (mine && d < a.d) y = read4_as(a.q.p, at + d, a.dtype);
          x[g][h][s] = y;
          most = fmaxf(most, fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w))));
        }
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
    // 2^14 <= most * up < 2^15; a row that is not finite stays as it is.
    const int e = (int)(__float_as_uint(most) >> 23);
    const int raise = e == 255 ? 0 : min(14 - (e - 127), 126);
    const float up = e == 0 && most == 0.f ? 1.f : __uint_as_float((uint32_t)(raise + 127) << 23);
    scale = a.scale * kLog2e / up;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      q_sum[g] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float y[8] = {x[g][h][0].x, x[g][h][0].y, x[g][h][0].z, x[g][h][0].w,
                      x[g][h][1].x, x[g][h][1].y, x[g][h][1].z, x[g][h][1].w};
        float low[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i] *= up;
          q_sum[g] += y[i];
          low[i] = (y[i] - __half2float(__float2half_rn(y[i]))) * 2048.f;
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          qa[g][h][s][0] = pack_f16(y[2 * s], y[2 * s + 4]);
          qa[g][h][s][1] = pack_f16(low[2 * s], low[2 * s + 4]);
          qa[g][h][s][2] = pack_f16(y[2 * s + 1], y[2 * s + 5]);
          qa[g][h][s][3] = pack_f16(low[2 * s + 1], low[2 * s + 5]);
        }
      }
      q_sum[g] += __shfl_xor_sync(0xffffffffu, q_sum[g], 1);
      q_sum[g] += __shfl_xor_sync(0xffffffffu, q_sum[g], 2);
    }
  }

  float o[G][4][4] = {}, o_mid[G] = {};
  float m = -INFINITY, l = 0.f;
  int stage = 0;
  for (int t = t0; t < t1; ++t) {
    cp_wait<kStages - 2>();
    __syncwarp();
    const uint32_t at = ring + stage * kBytes;
    // Scores of head r for the tokens 2c, 2c + 1, 2c + 8, 2c + 9.
    float s[4] = {};
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint4 k = lds128(at + g * 512 + lane * 16);
      const uint4 sc = lds128(at + key_scales4(G) + g * 64 + c * 16);
      const uint32_t words[2][2] = {{k.x, k.y}, {k.z, k.w}};
      const uint32_t scales[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float acc[4] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = words[j][h], y = x >> 8;
          mma_f16(acc, qa[g][h][0][0], qa[g][h][0][1], qa[g][h][0][2], qa[g][h][0][3], low_f16(x),
                  high_f16(x));
          mma_f16(acc, qa[g][h][1][0], qa[g][h][1][1], qa[g][h][1][2], qa[g][h][1][3], low_f16(y),
                  high_f16(y));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t z = scales[2 * j + i];
          const float dot = fmaf(acc[2 + i], 0x1p-11f, acc[i]);
          s[2 * j + i] = fmaf(step_of(z), dot, fmaf(mid_of(z), q_sum[g], s[2 * j + i]));
        }
      }
    }
    uint32_t v_scales[G][4];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint4 sc = lds128(at + value_scales4(G) + g * 64 + c * 16);
      v_scales[g][0] = sc.x, v_scales[g][1] = sc.y, v_scales[g][2] = sc.z, v_scales[g][3] = sc.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] *= scale;
    const int left = len - t * kBlock4;  // tokens of this block that count
    if (left < kBlock4) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (2 * c + (i & 1) + (i >> 1) * 8 >= left) {
          s[i] = -INFINITY;
#pragma unroll
          for (int g = 0; g < G; ++g) v_scales[g][i] = 0;
        }
    }
    float top = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (__any_sync(0xffffffffu, top > m + kLazy || (m == -INFINITY && top > m))) {
      const float now = fmaxf(m, top);
      const float by = m == -INFINITY ? 0.f : exp2_fast(m - now);
      m = now;
      l *= by;
#pragma unroll
      for (int g = 0; g < G; ++g) o_mid[g] *= by;
      const float by0 = __shfl_sync(0xffffffffu, by, 8 * c), by1 = __shfl_sync(0xffffffffu, by, 8 * c + 4);
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          o[g][x][0] *= by0, o[g][x][2] *= by0;
          o[g][x][1] *= by1, o[g][x][3] *= by1;
        }
    }
    const float from = m == -INFINITY ? 0.f : m;
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = exp2_fast(s[i] - from);
      l += p[i];
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = p[i] * step_of(v_scales[g][i]);
        o_mid[g] = fmaf(p[i], mid_of(v_scales[g][i]), o_mid[g]);
      }
      uint32_t pb[3][2];
#pragma unroll
      for (int i = 0; i < (F32 ? 3 : 2); ++i) {
        pb[i][0] = take_bf16(x[0], x[1]);
        pb[i][1] = take_bf16(x[2], x[3]);
      }
      const uint4 v = lds128(at + values4(G) + g * 512 + lane * 16);
      const uint32_t va[2] = {__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632)};
      const uint32_t vb[2] = {__byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632)};
#pragma unroll
      for (int x4 = 0; x4 < 4; ++x4) {
        const int half = x4 / 2, sh = (x4 & 1) * 8;
        const uint32_t a0 = low_bf16(va[half] >> sh), a1 = low_bf16(va[half] >> (sh + 4));
        const uint32_t a2 = low_bf16(vb[half] >> sh), a3 = low_bf16(vb[half] >> (sh + 4));
#pragma unroll
        for (int i = 0; i < (F32 ? 3 : 2); ++i) mma_bf16(o[g][x4], a0, a1, a2, a3, pb[i][0], pb[i][1]);
      }
    }
    __syncwarp();
    fetch(t + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
    stage = stage == kStages - 1 ? 0 : stage + 1;
  }
  cp_wait<0>();
  __syncwarp();

  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    o_mid[g] += __shfl_xor_sync(0xffffffffu, o_mid[g], 1);
    o_mid[g] += __shfl_xor_sync(0xffffffffu, o_mid[g], 2);
  }
  // This lane's results are heads 2c and 2c + 1, numbers 64 g + 8 r ...
  float wide[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) wide[i] = 2 * c + i < n_heads ? first_sum(a, b, head0 + 2 * c + i) : 0.f;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int h = 2 * c + i, from = 4 * h;
    const float hm = __shfl_sync(0xffffffffu, m, from), hl = __shfl_sync(0xffffffffu, l, from);
    float mids[G];
#pragma unroll
    for (int g = 0; g < G; ++g) mids[g] = __shfl_sync(0xffffffffu, o_mid[g], from);
    if (h >= n_heads) continue;
    Joint z{};
    if (piece < 0) {
      z = join_first(wide[i], hm, hl);
      if (a.lse && r == 0) a.lse[(int64_t)b * a.heads + head0 + h] = z.lse;
    } else if (r == 0) {
      w.sums[(int64_t)piece * w.heads + h] = make_float2(hm, hl);
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int d = 64 * g + 8 * r + 4 * s;
        const float4 y = make_float4(o[g][2 * s][i] + mids[g], o[g][2 * s][2 + i] + mids[g],
                                     o[g][2 * s + 1][i] + mids[g], o[g][2 * s + 1][2 + i] + mids[g]);
        if (piece >= 0)
          *reinterpret_cast<float4*>(w.results + ((int64_t)piece * w.heads + h) * (64 * G) + d) = y;
        else if (d < a.dv)
          put_result(a, b, head0 + h, d, y, z);
      }
  }
}

template <int G, bool F32>
__global__ void __launch_bounds__(kThreads, Shape<G>::kCtas) attn4_kernel(Attn4Args a, Work4 w) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_sum[kWarps];
  __shared__ int s_request[kWarps];
  __shared__ int64_t s_before[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tiles = (a.group + kHeads - 1) / kHeads, per_request = a.kv_heads * tiles;
  const int64_t units = (int64_t)a.n * per_request;
  let_next_start();

  // All blocks.
  int64_t sum = 0;
  for (int b = tid; b < a.n; b += kThreads) sum += blocks_of(len_of(a, b, blockIdx.x == 0));
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  if (tid < kWarps) s_request[tid] = -1;
  __syncthreads();
  sum = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) sum += s_sum[i];
  const int64_t total = sum * per_request;
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  // The first rule: pieces of at most `most` blocks; the second: even shares.
  const bool pieces = units <= warps / 2;
  int64_t most = (total + warps - units - 1) / (warps - units);
  most = most < kLeast ? kLeast : most;
  const int64_t shares = total < warps ? total : warps;
  const int64_t id = (int64_t)blockIdx.x * kWarps + warp;
  // Where each warp of the CTA begins, in pieces or in blocks.
  auto begin_of = [&](int64_t i) { return pieces ? i : i < shares ? i * total / shares : total; };
  int64_t carry = 0;
  const int64_t last = begin_of((int64_t)blockIdx.x * kWarps + kWarps - 1);
  for (int c0 = 0; c0 < a.n; c0 += kThreads) {
    const int b = c0 + tid;
    int64_t mine = 0;
    if (b < a.n) {
      const int t = blocks_of(len_of(a, b, false));
      mine = (int64_t)per_request * (pieces ? (t + most - 1) / most : t);
    }
    int64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = scan;
    __syncthreads();
    int64_t before = carry;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before += s_sum[i];
      carry += s_sum[i];
    }
    before += scan - mine;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int64_t x = begin_of((int64_t)blockIdx.x * kWarps + i);
      if (x >= before && x < before + mine) {
        s_request[i] = b;
        s_before[i] = before;
      }
    }
    if (carry > last) break;
  }
  __syncthreads();
  int b = s_request[warp];
  if (b < 0) return;
  const int64_t before = s_before[warp];
  const uint32_t ring = tc::sptr(smem) + warp * Shape<G>::kStages * block4_bytes(G);

  if (pieces) {
    const int t = blocks_of(len_of(a, b, false)), np = (int)((t + most - 1) / most);
    const int in = (int)(id - before), u = in / np, i = in - u * np;
    const int kvh = u / tiles, h0 = (u - kvh * tiles) * kHeads;
    if (w.units && i == 0 && lane == 0)
      w.units[(int64_t)b * per_request + u] = {(int32_t)id, np};
    run_range<G, F32>(a, w, ring, b, kvh, h0, (int)((int64_t)t * i / np),
                      (int)((int64_t)t * (i + 1) / np), np == 1 ? -1 : (int)id);
    return;
  }
  int64_t x = begin_of(id);
  const int64_t end = begin_of(id + 1);
  int t = blocks_of(len_of(a, b, false));
  int64_t at = x - before;  // in request b
  while (x < end) {
    const int u = (int)(at / t), lo = (int)(at - (int64_t)u * t);
    const int hi = (int)(end - x < t - lo ? lo + (end - x) : t);
    const int kvh = u / tiles, h0 = (u - kvh * tiles) * kHeads;
    const bool whole = lo == 0 && hi == t;
    // The unit's piece in its first warp is that one's 2 id + 1, in later ones 2 id.
    if (w.units && lo == 0 && lane == 0) {
      const int64_t stop = x + t;  // the last warp that has some of it
      const int64_t last_id = (stop * shares + total - 1) / total - 1;
      w.units[(int64_t)b * per_request + u] = {(int32_t)(2 * id + 1),
                                               whole ? 1 : -(int32_t)(last_id - id + 1)};
    }
    run_range<G, F32>(a, w, ring, b, kvh, h0, lo, hi,
                      whole ? -1 : (int)(lo == 0 ? 2 * id + 1 : 2 * id));
    x += hi - lo;
    at += hi - lo;
    if (at == (int64_t)t * per_request && x < end) {
      at = 0;
      t = blocks_of(len_of(a, ++b, false));
    }
  }
}

// Joins the pieces of a cut unit: a CTA a unit, its warps over the pieces, a lane's numbers
// 4 lane .. of each head.
constexpr int kJoinWarps = 8;

template <int G>
__global__ void __launch_bounds__(kJoinWarps * 32) join4_kernel(Attn4Args a, Work4 w) {
  __shared__ float s_o[kJoinWarps][64 * G];
  __shared__ float2 s_sum[kJoinWarps];
  wait_for_previous();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tiles = (a.group + kHeads - 1) / kHeads, per_request = a.kv_heads * tiles;
  const int64_t units = (int64_t)a.n * per_request;
  for (int64_t x = blockIdx.x; x < units * w.heads; x += gridDim.x) {
    const int64_t u = x / w.heads;
    const int h = (int)(x - u * w.heads);
    const Cut4 unit = w.units[u];
    const int b = (int)(u / per_request), in = (int)(u - (int64_t)b * per_request);
    const int kvh = in / tiles, h0 = (in - kvh * tiles) * kHeads;
    if (unit.pieces == 1 || h0 + h >= a.group) continue;
    const int n = unit.pieces < 0 ? -unit.pieces : unit.pieces;
    auto piece = [&](int i) {
      return (int64_t)(unit.pieces > 0 || i == 0 ? unit.first + i : unit.first + 2 * i - 1) * w.heads + h;
    };
    float top = -INFINITY;
    for (int i = tid; i < n; i += kJoinWarps * 32) top = fmaxf(top, w.sums[piece(i)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    __syncthreads();
    if (lane == 0) s_sum[warp].x = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) top = fmaxf(top, s_sum[i].x);
    __syncthreads();
    constexpr int kEach = (G + 1) / 2;
    float4 o[kEach] = {};
    float l = 0.f;
#pragma unroll 4
    for (int i = warp; i < n; i += kJoinWarps) {
      const int64_t p = piece(i);
      const float2 s = w.sums[p];
      const float by = s.x == -INFINITY ? 0.f : exp2_fast(s.x - top);
      l += s.y * by;
#pragma unroll
      for (int e = 0; e < kEach; ++e)
        if (128 * e + 4 * lane < 64 * G) {
          const float4 y = *reinterpret_cast<const float4*>(w.results + p * (64 * G) + 128 * e + 4 * lane);
          o[e].x = fmaf(y.x, by, o[e].x), o[e].y = fmaf(y.y, by, o[e].y);
          o[e].z = fmaf(y.z, by, o[e].z), o[e].w = fmaf(y.w, by, o[e].w);
        }
    }
    if (lane == 0) s_sum[warp].y = l;
    const int head = kvh * a.group + h0 + h;
    const float wide = first_sum(a, b, head);
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (128 * e + 4 * lane < 64 * G) *reinterpret_cast<float4*>(&s_o[warp][128 * e + 4 * lane]) = o[e];
    __syncthreads();
    if (tid * 4 < 64 * G) {
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      l = 0.f;
#pragma unroll
      for (int i = 0; i < kJoinWarps; ++i) {
        const float4 z = *reinterpret_cast<const float4*>(&s_o[i][4 * tid]);
        y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
        l += s_sum[i].y;
      }
      const Joint z = join_first(wide, top, l);
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
  const int64_t most = kSms * Shape<G>::kCtas;
  const int64_t cut = (blocks + kLeast - 1) / kLeast;
  int64_t ctas = cut > most * kWarps ? most : (p.units * (cut + 2) * 2 + kWarps - 1) / kWarps;
  ctas = ctas < 1 ? 1 : ctas < most ? ctas : most;
  p.ctas = (unsigned)ctas;
  const bool never = cut == 1 && p.units <= ctas * kWarps / 2;
  p.pieces = never ? 0 : 2 * ctas * kWarps;
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

template <int G, bool F32>
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
  cudaError_t e = ensure_smem<attn4_kernel<G, F32>>(Shape<G>::kSmem);
  if (e != cudaSuccess) return e;
  attn4_kernel<G, F32><<<p.ctas, kThreads, Shape<G>::kSmem, stream>>>(a, w);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.pieces == 0) return e;
  const int64_t rows = p.units * p.heads, ctas = rows < kSms * 8 ? rows : kSms * 8;
  return launch_dependent(join4_kernel<G>, dim3((unsigned)ctas), kJoinWarps * 32, 0, stream, a, w);
}

template <bool F32>
cudaError_t launch_of(const Attn4Args& a, void* workspace, cudaStream_t stream) {
  switch (groups4(a.d, a.dv)) {
    case 1: return launch<1, F32>(a, workspace, stream);
    case 2: return launch<2, F32>(a, workspace, stream);
    case 3: return launch<3, F32>(a, workspace, stream);
    default: return launch<4, F32>(a, workspace, stream);
  }
}

}  // namespace

size_t attn4_workspace(const nys_attn_config& c, int64_t n, int64_t keys) {
  if (n == 0) return 0;
  const int G = groups4(c.d, c.dv);
  const Plan4 p = plan_of(G, n, c.kv_heads, c.heads / c.kv_heads, keys);
  if (p.pieces == 0) return 0;
  return up256(p.units * sizeof(Cut4)) + up256(p.pieces * p.heads * sizeof(float2)) +
         up256(p.pieces * p.heads * sizeof(float) * 64 * G);
}

cudaError_t launch_attn4(const Attn4Args& a, void* workspace, cudaStream_t stream) {
  return a.dtype == NYS_F32 ? launch_of<true>(a, workspace, stream)
                            : launch_of<false>(a, workspace, stream);
}

}  // namespace nys
