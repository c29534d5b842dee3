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
// Bound by HBM: a row is read and written once.  The sines of a token are made once for
// all its heads and kept in shared memory; a row lies over 16 or 32 lanes, 4 numbers a
// lane and chunk, and a pair's other half is fetched through shared memory.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nys_attn_tc.h"
#include "nys_kv4.h"

namespace nys {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 4;    // rows of a lane group that are loaded together
constexpr int kTile = 4;    // tokens of a CTA where there are many
constexpr float kLeastStep = 0x1p-100f;

template <typename T>
struct alignas(4 * sizeof(T)) Four {
  T x[4];
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T round_to(float x);
template <>
__device__ __forceinline__ float round_to<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half round_to<__half>(float x) {
  return __float2half_rn(x);
}

// Four numbers at p, as one word where that is aligned.
template <typename T>
__device__ __forceinline__ Four<T> load4(const T* p) {
  if (reinterpret_cast<uintptr_t>(p) % sizeof(Four<T>) == 0) return *reinterpret_cast<const Four<T>*>(p);
  return {p[0], p[1], p[2], p[3]};
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&y)[4]) {
  const Four<T> z = {round_to<T>(y[0]), round_to<T>(y[1]), round_to<T>(y[2]), round_to<T>(y[3])};
  if (reinterpret_cast<uintptr_t>(p) % sizeof(Four<T>) == 0) {
    *reinterpret_cast<Four<T>*>(p) = z;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = z.x[i];
  }
}

// A group of 64 numbers over 16 lanes, 4 a lane (`here`: these are numbers of the row),
// to its scale word and this lane's 4 codes.
__device__ __forceinline__ uint32_t quantize(const float (&y)[4], bool here, uint32_t& scale) {
  float lo = here ? fminf(fminf(y[0], y[1]), fminf(y[2], y[3])) : INFINITY;
  float hi = here ? fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) : -INFINITY;
  // fminf and fmaxf pass over NaN, a sum does not; infinities show in the step.
  float odd = here ? y[0] + y[1] + y[2] + y[3] : 0.f;
  odd = odd != odd ? 1.f : 0.f;
#pragma unroll
  for (int o = 8; o; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o, 16));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o, 16));
    odd += __shfl_xor_sync(0xffffffffu, odd, o, 16);
  }
  if (!(lo <= hi) && odd == 0.f) {  // no numbers of the row at all
    scale = 0;
    return 0x8888u;
  }
  const float m = __fadd_rn(lo, __fdiv_rn(__fmul_rn(__fsub_rn(hi, lo), 8.f), 15.f));
  const float mid = __bfloat162float(__float2bfloat16_rn(m));
  float step = fmaxf(__fdiv_rn(__fsub_rn(hi, mid), 7.f), __fmul_rn(__fsub_rn(mid, lo), 0.125f));
  step = __uint_as_float((__float_as_uint(step) + 0xffffu) & 0xffff0000u);
  if (odd != 0.f || !(fabsf(mid) < INFINITY) || !(step < INFINITY)) {
    scale = 0x7fc07fc0u;
    return 0x8888u;
  }
  if (step < kLeastStep) step = 0.f;
  scale = __float_as_uint(step) | __float_as_uint(mid) >> 16;
  if (step == 0.f) return 0x8888u;
  const float inv = __frcp_rn(step);
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = __fsub_rn(y[i], mid);
    float t = __fmul_rn(x, inv);
    t = __fmaf_rn(__fmaf_rn(-t, step, x), inv, t);
    const int c = (int)rintf(fminf(fmaxf(t, -8.f), 7.f)) + 8;
    codes |= (uint32_t)c << (4 * i);
  }
  return codes;
}

// L lanes a row, E chunks of 4 L numbers.  blockIdx.x: tokens, blockIdx.y: a part of
// their rows.
template <typename T, int L, int E, bool Q4>
__global__ void __launch_bounds__(kThreads) qk_kernel(QkArgs a, int tile) {
  constexpr int kPer = 32 / L;  // rows of a warp at once
  constexpr int kSpan = 4 * L;
  extern __shared__ __align__(16) unsigned char smem[];
  float* s_weight = reinterpret_cast<float*>(smem);                // [2][kSpan * E]
  float* s_stage = s_weight + 2 * kSpan * E;                       // [rows at once][kSpan * E]
  int64_t* s_slot = reinterpret_cast<int64_t*>(s_stage + kWarps * kPer * kSpan * E);  // [kTile]
  float2* s_turn = reinterpret_cast<float2*>(s_slot + kTile);      // [tile][half]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int l = lane & (L - 1), sub = lane / L;
  const int per_token = a.heads + a.kv_heads + (a.v.p ? a.kv_heads : 0);
  const int64_t t0 = (int64_t)blockIdx.x * tile;
  const int nt = (int)(t0 + tile < a.tokens ? tile : a.tokens - t0);
  const int all = nt * per_token;
  const int u0 = (int)((int64_t)all * blockIdx.y / gridDim.y);
  const int u1 = (int)((int64_t)all * (blockIdx.y + 1) / gridDim.y);

  Four<T> raw[kRows][E];
  auto load = [&](int base) {
#pragma unroll
    for (int b = 0; b < kRows; ++b) {
      const int u = base + (b * kWarps + warp) * kPer + sub;
      if (u < u1) {
        const int tok = u / per_token;
        int r = u - tok * per_token;
        const Rows* from = &a.q;
        int dim = a.d;
        if (r >= a.heads) {
          r -= a.heads;
          from = &a.k;
          if (r >= a.kv_heads) {
            r -= a.kv_heads;
            from = &a.v;
            dim = a.dv;
          }
        }
        const T* p = static_cast<const T*>(from->p) + (t0 + tok) * from->row + r * from->head;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (e * kSpan + 4 * l < dim) raw[b][e] = load4(p + e * kSpan + 4 * l);
      }
    }
  };
  load(u0);

  for (int i = tid; i < a.d; i += kThreads) {
    if (a.q_weight) s_weight[i] = a.q_weight[i];
    if (a.k_weight) s_weight[kSpan * E + i] = a.k_weight[i];
  }
  if (a.slots && tid < nt) s_slot[tid] = a.slots[t0 + tid];
  for (int i = tid; i < nt * a.half; i += kThreads) {
    const int tok = i / a.half, pair = i - tok * a.half;
    const int64_t at = (int64_t)a.positions[t0 + tok] + a.shift;
    const uint64_t turn = (uint64_t)at * a.turns[pair];
    float2 z;  // cos, sin of the turn in (-1/2, 1/2]
    sincospif((float)(int32_t)(uint32_t)(turn >> 32) * 0x1p-31f, &z.y, &z.x);
    s_turn[i] = z;
  }
  __syncthreads();

  float* stage = s_stage + (warp * kPer + sub) * kSpan * E;
  for (int base = u0; base < u1;) {
#pragma unroll
    for (int b = 0; b < kRows; ++b) {
      const int first = base + (b * kWarps + warp) * kPer;  // the same for the warp
      if (first >= u1) break;
      const int u = first + sub;
      const bool row = u < u1;
      const int tok = row ? u / per_token : 0;
      int r = row ? u - tok * per_token : 0;
      const bool is_q = r < a.heads, is_v = r >= a.heads + a.kv_heads;
      r -= is_q ? 0 : is_v ? a.heads + a.kv_heads : a.heads;
      const int dim = is_v ? a.dv : a.d;
      const bool norm = !is_v && (is_q ? a.q_weight : a.k_weight) != nullptr;
      const bool turn = !is_v && a.half > 0;
      float y[E][4];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool in = row && e * kSpan + 4 * l < dim;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[e][i] = in ? widen(raw[b][e].x[i]) : 0.f;
      }
      if (__any_sync(0xffffffffu, norm)) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) ss = fmaf(y[e][i], y[e][i], ss);
#pragma unroll
        for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, L);
        if (norm) {
          const float inv = rsqrtf(ss / (float)a.d + a.eps);
          const float* w = s_weight + (is_q ? 0 : kSpan * E) + 4 * l;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (e * kSpan + 4 * l >= dim) continue;
            const float4 z = *reinterpret_cast<const float4*>(w + e * kSpan);
            y[e][0] = y[e][0] * inv * z.x;
            y[e][1] = y[e][1] * inv * z.y;
            y[e][2] = y[e][2] * inv * z.z;
            y[e][3] = y[e][3] * inv * z.w;
          }
        }
      }
      if (__any_sync(0xffffffffu, turn)) {
        const float2* cs = s_turn + tok * a.half;
        if (a.interleaved) {
          if (turn) {
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                const int pair = (e * kSpan + 4 * l + i) / 2;
                if (pair < a.half) {
                  const float2 z = cs[pair];
                  const float p = y[e][i], q = y[e][i + 1];
                  y[e][i] = p * z.x - q * z.y;
                  y[e][i + 1] = p * z.y + q * z.x;
                }
              }
          }
        } else {
          __syncwarp();
#pragma unroll
          for (int e = 0; e < E; ++e)
            *reinterpret_cast<float4*>(stage + e * kSpan + 4 * l) =
                make_float4(y[e][0], y[e][1], y[e][2], y[e][3]);
          __syncwarp();
          if (turn) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const int at = e * kSpan + 4 * l;
              if (at >= 2 * a.half) continue;
              float other[4];
              float2 z[4];
              if ((a.half & 3) == 0) {  // four numbers on one side
                const int x = at < a.half ? at : at - a.half;
                const float4 o = *reinterpret_cast<const float4*>(stage + (at < a.half ? at + a.half : x));
                const float4 z0 = *reinterpret_cast<const float4*>(cs + x);
                const float4 z1 = *reinterpret_cast<const float4*>(cs + x + 2);
                other[0] = o.x, other[1] = o.y, other[2] = o.z, other[3] = o.w;
                z[0] = {z0.x, z0.y}, z[1] = {z0.z, z0.w}, z[2] = {z1.x, z1.y}, z[3] = {z1.z, z1.w};
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int c = at + i, x = c < a.half ? c : c - a.half;
                  const bool in = c < 2 * a.half;
                  other[i] = in ? stage[c < a.half ? c + a.half : x] : 0.f;
                  z[i] = in ? cs[x] : make_float2(1.f, 0.f);
                }
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)
                y[e][i] = at + i < a.half ? y[e][i] * z[i].x - other[i] * z[i].y
                                          : y[e][i] * z[i].x + other[i] * z[i].y;
            }
          }
        }
      }
      const Rows& to = is_q ? a.q_out : a.k_out;
      if (row && !is_v && to.p) {
        T* p = static_cast<T*>(to.p) + (t0 + tok) * to.row + r * to.head;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (e * kSpan + 4 * l < dim) store4(p + e * kSpan + 4 * l, y[e]);
      }
      const int64_t slot = row && !is_q && a.slots ? s_slot[tok] : -1;
      const bool held = slot >= 0 && slot < a.n_slots;
      if constexpr (Q4) {
        if (__any_sync(0xffffffffu, held)) {
          const int64_t block = slot >> 4, page = held ? block / a.page_blocks : 0;
          uint32_t* to4 = reinterpret_cast<uint32_t*>(
              a.blocks + ((page * a.kv_heads + r) * a.page_blocks + (block - page * a.page_blocks)) *
                             block4_bytes(a.groups));
          const int t = (int)(slot & 15);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            uint32_t scale, codes = quantize(y[e], e * kSpan + 4 * l < dim, scale);
            codes |= __shfl_xor_sync(0xffffffffu, codes, 1) << 16;
            const int g = (e * kSpan + 4 * l) / kGroup4, x = l / 2 % 8;
            if (held && g < a.groups) {
              if ((l & 1) == 0)
                to4[is_v ? values4(a.groups) / 4 + value_word4(g, t, x) : key_word4(g, t, x)] = codes;
              if ((l & 15) == 0)
                to4[(is_v ? value_scales4(a.groups) : key_scales4(a.groups)) / 4 + g * 16 + place4(t)] = scale;
            }
          }
        }
      } else if (held) {
        T* p = static_cast<T*>(is_v ? a.pool_v : a.pool_k) + (slot * a.kv_heads + r) * dim;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (e * kSpan + 4 * l < dim) store4(p + e * kSpan + 4 * l, y[e]);
      }
    }
    base += kRows * kWarps * kPer;
    if (base < u1) load(base);
  }
}

template <typename T, int L, int E, bool Q4>
cudaError_t launch(const QkArgs& a, cudaStream_t stream) {
  constexpr int kPer = 32 / L;
  const int per_token = a.heads + a.kv_heads + (a.v.p ? a.kv_heads : 0);
  // Few tokens: a row a lane group, over as many SMs as there are rows for.
  int parts = (per_token + kWarps * kPer - 1) / (kWarps * kPer), tile = 1;
  if (a.tokens * parts > 152 * 8) {
    tile = kTile;
    parts = 1;
  }
  const int64_t ctas = (a.tokens + tile - 1) / tile;
  const size_t smem = sizeof(float) * (2 + kWarps * kPer) * 4 * L * E + sizeof(int64_t) * kTile +
                      sizeof(float2) * tile * a.half;
  qk_kernel<T, L, E, Q4><<<dim3((unsigned)ctas, parts), kThreads, smem, stream>>>(a, tile);
  return cudaGetLastError();
}

template <typename T, bool Q4>
cudaError_t launch_of(const QkArgs& a, cudaStream_t stream) {
  const int most = a.d > a.dv ? a.d : a.dv;
  if (most <= 64) return launch<T, 16, 1, Q4>(a, stream);
  if (most <= 128) return launch<T, 32, 1, Q4>(a, stream);
  return launch<T, 32, 2, Q4>(a, stream);
}

// Rows of a 4-bit cache as the values they stand for; a slot outside it gives zeros.  A
// thread takes the 8 numbers of a code word; words of a row are consecutive lanes.
template <typename T>
__global__ void __launch_bounds__(kThreads) read4_kernel(Read4Args a) {
  const int words_k = (a.d + 7) / 8, words = words_k + (a.dv + 7) / 8;
  const int per = words * a.kv_heads;
  const int64_t total = a.tokens * per;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t tok = total <= INT32_MAX ? (int64_t)((uint32_t)i / (uint32_t)per) : i / per;
    const int in = (int)(i - tok * per), h = in / words;
    int x = in - h * words;
    const bool is_v = x >= words_k;
    if (is_v) x -= words_k;
    const int64_t slot = a.slots[tok];
    uint32_t codes = 0, scale = 0;
    if (slot >= 0 && slot < a.n_slots) {
      const int64_t block = slot >> 4, page = block / a.page_blocks;
      const uint32_t* from = reinterpret_cast<const uint32_t*>(
          a.blocks + ((page * a.kv_heads + h) * a.page_blocks + (block - page * a.page_blocks)) *
                         block4_bytes(a.groups));
      const int t = (int)(slot & 15), g = x / 8;
      codes = from[is_v ? values4(a.groups) / 4 + value_word4(g, t, x % 8) : key_word4(g, t, x % 8)];
      scale = from[(is_v ? value_scales4(a.groups) : key_scales4(a.groups)) / 4 + g * 16 + place4(t)];
    }
    const float step = __uint_as_float(scale & 0xffff0000u), mid = __uint_as_float(scale << 16);
    const Rows& to = is_v ? a.v : a.k;
    T* p = static_cast<T*>(to.p) + tok * to.row + h * to.head + 8 * x;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (8 * x + 4 * half >= (is_v ? a.dv : a.d)) break;
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)  // the product is exact: 8 + 4 bits
        y[e] = mid + step * (float)((int)(codes >> (16 * half + 4 * e) & 15) - 8);
      store4(p + 4 * half, y);
    }
  }
}

template <typename T>
cudaError_t launch_read(const Read4Args& a, cudaStream_t stream) {
  const int64_t threads = a.tokens * a.kv_heads * ((a.d + 7) / 8 + (a.dv + 7) / 8);
  int64_t ctas = (threads + kThreads - 1) / kThreads;
  if (ctas > 152 * 64) ctas = 152 * 64;
  read4_kernel<T><<<(unsigned)ctas, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
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
    case NYS_F32: return launch_read<float>(a, stream);
    case NYS_BF16: return launch_read<__nv_bfloat16>(a, stream);
    default: return launch_read<__half>(a, stream);
  }
}

}  // namespace nys
