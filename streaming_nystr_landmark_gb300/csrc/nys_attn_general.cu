// Exact attention, general path: any head dim up to 256, any strides and
// alignment, any type.
//
//   out_i = sum_j e^{s_ij - m_i} v_j / sum_j e^{s_ij - m_i},
//   s_ij = scale q_i . k_j,  m_i = max_j s_ij over the keys that i sees,
//
// in one pass over the keys with the running maximum and sum (flash form):
// a new maximum rescales what has been summed by e^{m_old - m_new}.
//
// One warp per (row, head).  32 keys at a time: lane = key for the dot
// products (the query in shared memory), then lane = value column for the
// weighted sum, each weight broadcast by a shuffle.  Nothing is reused
// between the rows of a group, so the caches carry the keys; this path is
// for the shapes that the tiled kernels do not take, and its arithmetic is
// all f32 whatever the stored type.
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nys_attn.h"

namespace nys {
namespace {

constexpr int kWarps = 4;

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <>
__device__ __forceinline__ float to_f<__half>(__half x) {
  return __half2float(x);
}
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f<__half>(float x) {
  return __float2half_rn(x);
}

// Running softmax of one row over a warp.  acc[c] is column lane + 32 c.
struct RowState {
  float m = -INFINITY, l = 0.f;
  float acc[kAttnMaxDim / 32];
  __device__ __forceinline__ RowState() {
#pragma unroll
    for (int c = 0; c < kAttnMaxDim / 32; ++c) acc[c] = 0.f;
  }
};

// Adds keys [0, nk) whose rows `at(j, kp, vp)` gives (false: no such row, all
// zeros).  q is the warp's query in shared memory, already scaled.
template <typename T, typename At>
__device__ __forceinline__ void add_keys(RowState& st, const float* q, int d, int dv, int nk,
                                         int lane, At at) {
  for (int j0 = 0; j0 < nk; j0 += 32) {
    const int j = j0 + lane;
    float s = -INFINITY;
    if (j < nk) {
      const T *kp, *vp;
      float x = 0.f;
      if (at(j, kp, vp))
        for (int c = 0; c < d; ++c) x = fmaf(q[c], to_f<T>(kp[c]), x);
      s = x;
    }
    float bm = s;
#pragma unroll
    for (int o = 16; o; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
    const float nm = fmaxf(st.m, bm);
    const float ref = nm == -INFINITY ? 0.f : nm;
    const float r = expf(st.m - ref);
    // A NaN score (its own key's or query's NaN) stays a NaN weight.
    const float p = j < nk ? expf(s - ref) : 0.f;
    float ps = p;
#pragma unroll
    for (int o = 16; o; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
    st.l = st.l * r + ps;
    st.m = nm;
#pragma unroll
    for (int c = 0; c < kAttnMaxDim / 32; ++c) st.acc[c] *= r;
    const int nb = min(32, nk - j0);
    for (int b = 0; b < nb; ++b) {
      const float w = __shfl_sync(0xffffffffu, p, b);
      const T *kp, *vp;
      if (at(j0 + b, kp, vp)) {
#pragma unroll
        for (int c = 0; c < kAttnMaxDim / 32; ++c)
          if (c * 32 + lane < dv) st.acc[c] = fmaf(w, to_f<T>(vp[c * 32 + lane]), st.acc[c]);
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void write_row(const RowState& st, T* out, float* lse, int dv,
                                          int lane) {
  const float inv = st.l == 0.f ? 0.f : 1.f / st.l;
#pragma unroll
  for (int c = 0; c < kAttnMaxDim / 32; ++c)
    if (c * 32 + lane < dv) out[c * 32 + lane] = from_f<T>(st.acc[c] * inv);
  if (lse && lane == 0) *lse = st.l == 0.f ? -INFINITY : st.m + logf(st.l);
}

template <typename T>
__device__ __forceinline__ void load_query(float* dst, const T* src, int d, float scale, int lane) {
  for (int c = lane; c < d; c += 32) dst[c] = to_f<T>(src[c]) * scale;
  __syncwarp();
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) prompt_general_kernel(PromptArgs a) {
  __shared__ float qs[kWarps][kAttnMaxDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t total = a.q_rows * a.heads;
  for (int64_t w = (int64_t)blockIdx.x * kWarps + warp; w < total; w += (int64_t)gridDim.x * kWarps) {
    const int64_t row = w / a.heads;
    const int h = (int)(w - row * a.heads), g = h / a.group;
    // The last sequence that starts at or before the row (empty ones share
    // their start with the next).
    int lo = 0, hi = a.n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int64_t)a.q_off[mid] <= row) lo = mid;
      else hi = mid;
    }
    int q0, nq, k0, nk;
    bool bad = false;
    seq_range(a.q_off, lo, a.q_rows, q0, nq, bad);
    seq_range(a.k_off, lo, a.k_rows, k0, nk, bad);
    if (bad && lane == 0) attn_report(a.status, NYS_ATTN_BAD_OFFSETS);
    if (row < q0 || row >= (int64_t)q0 + nq) continue;  // between sequences: not theirs
    const int64_t seen = (row - q0) + (int64_t)nk - nq + 1;
    const int n_seen = (int)(seen < 0 ? 0 : (seen > nk ? nk : seen));
    __syncwarp();
    load_query<T>(qs[warp], (const T*)a.q.p + row * a.q.row + h * a.q.head, a.d, a.scale, lane);
    RowState st;
    const T* kb = (const T*)a.k.p + k0 * a.k.row + g * a.k.head;
    const T* vb = (const T*)a.v.p + k0 * a.v.row + g * a.v.head;
    add_keys<T>(st, qs[warp], a.d, a.dv, n_seen, lane, [&](int j, const T*& kp, const T*& vp) {
      kp = kb + j * a.k.row;
      vp = vb + j * a.v.row;
      return true;
    });
    write_row<T>(st, (T*)a.out.p + row * a.out.row + h * a.out.head,
                 a.lse ? a.lse + row * a.heads + h : nullptr, a.dv, lane);
  }
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) shared_general_kernel(SharedArgs a) {
  __shared__ float qs[kWarps][kAttnMaxDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t total = (int64_t)a.n * a.heads;
  for (int64_t w = (int64_t)blockIdx.x * kWarps + warp; w < total; w += (int64_t)gridDim.x * kWarps) {
    const int64_t b = w / a.heads;
    const int h = (int)(w - b * a.heads), g = h / a.group;
    __syncwarp();
    load_query<T>(qs[warp], (const T*)a.q.p + b * a.q.row + h * a.q.head, a.d, a.scale, lane);
    RowState st;
    auto run = [&](const int32_t* pages, int len) {
      add_keys<T>(st, qs[warp], a.d, a.dv, len, lane, [&](int j, const T*& kp, const T*& vp) {
        const int32_t pg = pages[j / a.page];
        if (pg < 0 || pg >= a.n_pages) {
          attn_report(a.status, NYS_ATTN_BAD_PAGE);
          return false;
        }
        const int64_t r = ((int64_t)pg * a.page + j % a.page) * a.kv_heads + g;
        kp = (const T*)a.k + r * a.d;
        vp = (const T*)a.v + r * a.dv;
        return true;
      });
    };
    run(a.prefix_pages, a.prefix_len);
    const int64_t len = a.lens[b], cap = (int64_t)a.width * a.page;
    if (len < 0 || len > cap) attn_report(a.status, NYS_ATTN_BAD_LENGTH);
    run(a.table + b * a.width, (int)(len < 0 ? 0 : (len > cap ? cap : len)));
    write_row<T>(st, (T*)a.out.p + b * a.out.row + h * a.out.head,
                 a.lse ? a.lse + b * a.heads + h : nullptr, a.dv, lane);
  }
}

unsigned grid_for(int64_t warps) {
  const int64_t g = (warps + kWarps - 1) / kWarps;
  return (unsigned)(g < 152 * 64 ? g : 152 * 64);
}

}  // namespace

cudaError_t launch_prompt_general(const PromptArgs& a, cudaStream_t stream) {
  const int64_t warps = a.q_rows * a.heads;
  if (warps == 0) return cudaSuccess;
  const unsigned grid = grid_for(warps);
  if (a.dtype == NYS_F32) prompt_general_kernel<float><<<grid, kWarps * 32, 0, stream>>>(a);
  else if (a.dtype == NYS_BF16)
    prompt_general_kernel<__nv_bfloat16><<<grid, kWarps * 32, 0, stream>>>(a);
  else prompt_general_kernel<__half><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_shared_general(const SharedArgs& a, cudaStream_t stream) {
  const int64_t warps = (int64_t)a.n * a.heads;
  if (warps == 0) return cudaSuccess;
  const unsigned grid = grid_for(warps);
  if (a.dtype == NYS_F32) shared_general_kernel<float><<<grid, kWarps * 32, 0, stream>>>(a);
  else if (a.dtype == NYS_BF16)
    shared_general_kernel<__nv_bfloat16><<<grid, kWarps * 32, 0, stream>>>(a);
  else shared_general_kernel<__half><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace nys
