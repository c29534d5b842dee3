// The paged cache's bookkeeping and writes.
//
// Plan: request i holds cached_i tokens and gets fresh_i more, p tokens a
// page.  With old_i = ceil(cached_i / p), new_i = ceil((cached_i + fresh_i) / p)
// and start_i = sum_{j<i} (new_j - old_j), columns old_i .. new_i - 1 of its
// block table take free[start_i ..], and its token at position x lies in slot
// table[i][x / p] * p + x mod p.
//
// One launch and no step between CTAs: every CTA scans all lengths by itself
// (n is thousands at most, 8 bytes each, from L2) and then writes the tokens
// of its own range.  The scan carries tokens and pages as one 64-bit word, and
// its sums stop at one token more than there are slots and at the pages there
// are: lengths that sum past them, past 32 bits even, reach no other memory.
// What bounds a call is its launch: one new token for 64 requests takes 7 us,
// 1,000 prompts of up to 1,024 tokens 8 us, most of it the host's call.  A token finds its request by bisection of the chunk's offsets in shared
// memory; a page's first token also writes the page's number to the table,
// and the numbers of new pages come from the free list, so no CTA reads what
// another writes.
#include <cstdint>

#include "nys_attn.h"
#include "nys_kv.h"

namespace nys {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanEach = 4;  // requests of a thread in one chunk
constexpr int kPlanChunk = kPlanThreads * kPlanEach;
constexpr int kPlanTokens = 1024;  // tokens of a CTA, at least

__device__ __forceinline__ int ceil_div(int64_t x, int p) { return (int)((x + p - 1) / p); }

// Sum of two (pages << 32 | tokens) words, each part held at its part of `most`
// (below 2^31), which keeps it associative.
__device__ __forceinline__ uint64_t add_held(uint64_t a, uint64_t b, uint64_t most) {
  const uint32_t tokens = min((uint32_t)a + (uint32_t)b, (uint32_t)most);
  const uint32_t pages = min((uint32_t)(a >> 32) + (uint32_t)(b >> 32), (uint32_t)(most >> 32));
  return (uint64_t)pages << 32 | tokens;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a, int64_t per_cta) {
  __shared__ int s_off[kPlanChunk + 1];    // first token of each request of the chunk
  __shared__ int s_start[kPlanChunk];      // its rank in the free list
  __shared__ int s_cached[kPlanChunk];
  __shared__ uint64_t s_warp[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t0 = blockIdx.x * per_cta;
  const int64_t t1 = t0 + per_cta < a.total ? t0 + per_cta : a.total;
  const uint64_t most = (uint64_t)a.n_free << 32 | (uint32_t)(a.total + 1);
  uint64_t carry = 0;  // pages << 32 | tokens before this chunk
  for (int c0 = 0; c0 < a.n; c0 += kPlanChunk) {
    uint64_t mine[kPlanEach], sum = 0;
    int cached[kPlanEach], fresh[kPlanEach];
#pragma unroll
    for (int e = 0; e < kPlanEach; ++e) {
      const int i = c0 + tid * kPlanEach + e;
      cached[e] = i < a.n ? a.cached[i] : 0;
      fresh[e] = i < a.n ? a.fresh[i] : 0;
    }
#pragma unroll
    for (int e = 0; e < kPlanEach; ++e) {
      if (cached[e] < 0 || fresh[e] < 0 || (int64_t)cached[e] + fresh[e] > INT32_MAX) {
        if (blockIdx.x == 0) attn_report(a.status, NYS_PLAN_BAD_LENGTH);
        cached[e] = max(cached[e], 0);
        fresh[e] = 0;
      }
      const int need = ceil_div((int64_t)cached[e] + fresh[e], a.page) - ceil_div(cached[e], a.page);
      mine[e] = sum;
      sum = add_held(sum, add_held((uint64_t)(uint32_t)need << 32 | (uint32_t)fresh[e], 0, most), most);
    }
    uint64_t scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan = add_held(scan, y, most);
    }
    uint64_t lower = __shfl_up_sync(0xffffffffu, scan, 1);  // the lanes' before this one
    if (lane == 0) lower = 0;
    if (lane == 31) s_warp[warp] = scan;
    __syncthreads();
    uint64_t before = carry, all = carry;
#pragma unroll
    for (int x = 0; x < kPlanThreads / 32; ++x) {
      if (x < warp) before = add_held(before, s_warp[x], most);
      all = add_held(all, s_warp[x], most);
    }
    before = add_held(before, lower, most);
#pragma unroll
    for (int e = 0; e < kPlanEach; ++e) {
      const int x = tid * kPlanEach + e;
      const uint64_t at = add_held(before, mine[e], most);
      s_off[x] = (int)(uint32_t)at;
      s_start[x] = (int)(at >> 32);
      s_cached[x] = cached[e];
      const int i = c0 + x;
      if (i < a.n && blockIdx.x == (unsigned)(c0 / kPlanChunk) % gridDim.x) {
        a.q_off[i] = (int)(uint32_t)at;
        if (a.lens) a.lens[i] = cached[e] + fresh[e];
      }
    }
    if (tid == 0) s_off[kPlanChunk] = (int)(uint32_t)all;
    __syncthreads();
    const int first = s_off[0], end = s_off[kPlanChunk];
    const int64_t lo = t0 > first ? t0 : first, hi = t1 < end ? t1 : end;
    for (int64_t t = lo + tid; t < hi; t += kPlanThreads) {
      int x = 0;  // the last request of the chunk with off <= t
#pragma unroll
      for (int step = kPlanChunk >> 1; step; step >>= 1)
        if (s_off[x + step] <= t) x += step;
      const int i = c0 + x;
      const int pos = s_cached[x] + (int)(t - s_off[x]);
      const int col = pos / a.page, in = pos - col * a.page;
      const int old = ceil_div(s_cached[x], a.page);
      int32_t pg = -1;
      if (col < a.width) {
        int32_t* cell = a.table + (int64_t)i * a.width + col;
        if (col < old) {
          pg = *cell;
          if (pg < 0) attn_report(a.status, NYS_PLAN_NO_PAGES);
        } else {
          const int64_t rank = (int64_t)s_start[x] + (col - old);
          if (rank < a.n_free) pg = a.free_pages[rank];
          else attn_report(a.status, NYS_PLAN_NO_PAGES);
          if (in == 0) *cell = pg;
        }
      } else {
        attn_report(a.status, NYS_PLAN_TABLE_FULL);
      }
      a.slots[t] = pg < 0 ? -1 : (int64_t)pg * a.page + in;
      a.positions[t] = pos;
    }
    carry = all;
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) {
    const int64_t tokens = (uint32_t)carry, pages = (int64_t)(carry >> 32);
    a.q_off[a.n] = (int32_t)tokens;
    *a.taken = (int32_t)(pages < a.n_free ? pages : a.n_free);
    if (tokens != a.total) attn_report(a.status, NYS_PLAN_BAD_LENGTH);
  }
  // Tokens that no request has (the lengths sum to less than `total`).
  for (int64_t t = (t0 > (int64_t)(uint32_t)carry ? t0 : (int64_t)(uint32_t)carry) + tid; t < t1;
       t += kPlanThreads) {
    a.slots[t] = -1;
    a.positions[t] = -1;
  }
}

// New lengths in place of the old ones (lens is cached), after the plan's CTAs have
// all read them; bad lengths as plan_kernel takes them.
__global__ void __launch_bounds__(256) grow_kernel(int32_t* lens, const int32_t* fresh, int32_t n) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int c = lens[i], f = fresh[i];
  lens[i] = c < 0 || f < 0 || (int64_t)c + f > INT32_MAX ? max(c, 0) : c + f;
}

// Rows into pages: token t's K and V rows go to slot slots[t] of the pools; a
// slot outside the pool (-1: the plan had no page) is skipped.  Bound by HBM:
// every byte is read once and written once; 16,384 tokens of 8 heads of 128 + 128
// in bf16 (134 MB moved) take 25 us, 79% of the measured copy rate.  A thread moves kWriteEach units
// of W bytes, loaded before the first is stored, so that enough reads are in
// flight; units of a token are consecutive lanes, so reads and writes are
// whole rows.
constexpr int kWriteThreads = 256;
constexpr int kWriteEach = 4;

template <typename U>
__global__ void __launch_bounds__(kWriteThreads) write_kernel(WriteArgs a) {
  const uint32_t ku = a.k_units, per = a.k_units + a.v_units;  // units of a token
  const int64_t total = a.tokens * per;
  const int64_t stride = (int64_t)gridDim.x * kWriteThreads;
  for (int64_t u0 = (int64_t)blockIdx.x * kWriteThreads + threadIdx.x; u0 < total;
       u0 += stride * kWriteEach) {
    // All slots, then all rows, then the stores: no load waits for another
    // unit's.
    int64_t token[kWriteEach], slot[kWriteEach];
    uint32_t in[kWriteEach];
#pragma unroll
    for (int e = 0; e < kWriteEach; ++e) {
      const int64_t u = u0 + e * stride;
      const bool here = u < total;
      token[e] = total <= INT32_MAX ? (int64_t)((uint32_t)(here ? u : 0) / per) : (here ? u : 0) / per;
      in[e] = (uint32_t)((here ? u : 0) - token[e] * per);
      slot[e] = here ? a.slots[token[e]] : -1;
    }
    U x[kWriteEach];
    U* dst[kWriteEach];
#pragma unroll
    for (int e = 0; e < kWriteEach; ++e) {
      const bool is_k = in[e] < ku;
      const uint32_t at = is_k ? in[e] : in[e] - ku;
      const uint32_t hu = is_k ? a.k_head_units : a.v_head_units;
      const uint32_t h = at / hu;
      const U* src = is_k ? (const U*)a.k + token[e] * a.k_row + h * a.k_head + (at - h * hu)
                          : (const U*)a.v + token[e] * a.v_row + h * a.v_head + (at - h * hu);
      x[e] = *src;  // (a token without a slot is read too: its row exists)
      dst[e] = slot[e] < 0 || slot[e] >= a.n_slots ? nullptr
               : is_k ? (U*)a.pool_k + slot[e] * ku + at
                      : (U*)a.pool_v + slot[e] * a.v_units + at;
    }
#pragma unroll
    for (int e = 0; e < kWriteEach; ++e)
      if (dst[e]) *dst[e] = x[e];
  }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t stream) {
  int64_t ctas = (a.total + kPlanTokens - 1) / kPlanTokens;
  if (ctas < 1) ctas = 1;
  if (ctas > 2 * 152) ctas = 2 * 152;
  const int64_t per = (a.total + ctas - 1) / ctas;
  // A single CTA's threads read a length before they write it; more CTAs leave the
  // writing of lengths that they all read to a launch of its own.
  PlanArgs p = a;
  const bool later = a.n > 0 && a.lens == a.cached && ctas > 1;
  if (later) p.lens = nullptr;
  plan_kernel<<<(unsigned)ctas, kPlanThreads, 0, stream>>>(p, per < 1 ? 1 : per);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !later) return e;
  grow_kernel<<<(unsigned)((a.n + 255) / 256), 256, 0, stream>>>(a.lens, a.fresh, a.n);
  return cudaGetLastError();
}

cudaError_t launch_write(const WriteArgs& a, cudaStream_t stream) {
  const int64_t units = a.tokens * (int64_t)(a.k_units + a.v_units);
  if (units == 0) return cudaSuccess;
  int64_t ctas = (units + kWriteThreads * kWriteEach - 1) / (kWriteThreads * kWriteEach);
  if (ctas < 152 * 4) ctas = (units + kWriteThreads - 1) / kWriteThreads;  // few rows: spread them
  if (ctas > 152 * 64) ctas = 152 * 64;
  switch (a.unit) {
    case 16: write_kernel<uint4><<<(unsigned)ctas, kWriteThreads, 0, stream>>>(a); break;
    case 8: write_kernel<uint2><<<(unsigned)ctas, kWriteThreads, 0, stream>>>(a); break;
    case 4: write_kernel<uint32_t><<<(unsigned)ctas, kWriteThreads, 0, stream>>>(a); break;
    default: write_kernel<uint16_t><<<(unsigned)ctas, kWriteThreads, 0, stream>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace nys
