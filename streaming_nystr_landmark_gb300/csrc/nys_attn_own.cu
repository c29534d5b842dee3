// Single-token attention over a request's own pages, and the joining of
// partial results (flash form, nys_attn_general.cu):
//
//   for pieces x with maxima m_x, sums l_x and O_x = sum_j 2^{s_j - m_x} v_j:
//   out = sum_x 2^{m_x - m} O_x / sum_x 2^{m_x - m} l_x,  m = max_x m_x.
//
// Bound by HBM: a request's keys and values are read once for the heads of a
// group (8 of them in f32, 16 in 16-bit types; wider groups read them again), and there
// is little arithmetic a byte.  A CTA of four warps
// takes one (request, KV head, piece of its keys); each warp streams tiles of
// its own through a private ring in shared memory with cp.async, no barrier
// between warps until their results are joined; three CTAs a SM keep the reads
// in flight.  64 requests of 97 to 1025 keys over a prefix of 2,000 (8 KV heads of
// 128, f32): 43 us for 208 MB from memory, 62% of its peak, and 60 us for the whole
// call (floor 33 us).  Pieces of a request are joined by a second launch,
// or, where all CTAs run at once, in shared memory as a cluster (4 requests of 3 to
// 45 keys over a prefix of 301, bf16: 6.6 us, 8.3 us with the launch).
// Keys past the length and pages outside the pool
// are filled with zeros and never read from memory.
//
// bf16 / fp16: tiles of 16 keys, mma.sync m16n8k16 with the group's heads as
// the (padded) 16 rows -- the product is far too small for the 128-row
// tensor-memory form and memory sets the time.  f32: tiles of 8 keys, lane =
// four columns, exact f32 FMAs; the dot products of 8 keys x the heads finish in one
// interleaved butterfly.
#include <cmath>

#include "nys_attn_tc.h"

namespace nys {
namespace {

using namespace tc;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazy = 8.f;

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

// Request b's length, held inside its table.
__device__ __forceinline__ int own_len(const SharedArgs& a, int b, bool report) {
  const int len = a.lens[b], cap = a.width * a.page;
  if (report && (len < 0 || len > cap)) attn_report(a.status, NYS_ATTN_BAD_LENGTH);
  return len < 0 ? 0 : (len > cap ? cap : len);
}
// Keys of a piece of a request's `len`: even pieces, of short requests fewer, and
// more than 16 only of 256 keys and more (the join's time).
__device__ __forceinline__ int piece_keys(const OwnArgs& o, int len) {
  const int some = min(256, len / 16), even = (len + o.pieces - 1) / o.pieces;
  return (max(max(some, even), o.keys) + 31) & ~31;
}
// The piece of its keys (the prefix's first, where they are read with them) that
// this CTA reads, [lo, hi); false: there is none.
__device__ __forceinline__ bool own_range(const SharedArgs& a, const OwnArgs& o, int b, int piece,
                                          int& lo, int& hi) {
  const int len = o.lead + own_len(a, b, true);
  const int keys = piece_keys(o, len);
  lo = piece * keys;
  hi = min(len, lo + keys);
  return o.pieces == 1 || lo < hi;
}

constexpr uint32_t kNoRow = 0xffffffffu;

// Row (slot x KV heads + KV head) of key j < hi of a request in the pool, kNoRow
// past the end or where its page is not in the pool.
__device__ __forceinline__ uint32_t own_row(const SharedArgs& a, const OwnArgs& o,
                                            const int32_t* pages, int j, int hi, int kvh) {
  if (j >= hi) return kNoRow;
  if (j < o.lead) pages = a.prefix_pages;
  else j -= o.lead;
  const int pi = j / a.page;
  const int32_t pg = pages[pi];
  if (pg < 0 || pg >= a.n_pages) {
    attn_report(a.status, NYS_ATTN_BAD_PAGE);
    return kNoRow;
  }
  return ((uint32_t)pg * a.page + (j - pi * a.page)) * a.kv_heads + kvh;
}

// A warp's keys come in blocks of 32 (block i of warp w: 32 (4 i + w) ..), whose
// rows the lanes look up one block ahead.
struct RowAhead {
  uint32_t now = kNoRow, next = kNoRow;
};

template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half narrow<__half>(float x) {
  return __float2half_rn(x);
}

// The prefix's pieces of one row: how many, and the row of the first in `part`
// (those of the others follow `step` rows apart).
struct PrefixRow {
  int pieces = 0;
  int64_t first = 0, step = 0;
  __device__ __forceinline__ PrefixRow(const SharedArgs& a, const OwnArgs& o, int b, int h) {
    const Shares& s = o.shares;
    if (s.units == 0) return;
    const int kvh = h / a.group, unit = b / s.rows * a.kv_heads + kvh;
    const int pos = b % s.rows, tile = pos / s.tp;
    pieces = s.pieces(unit);
    step = (int64_t)o.per * kTileM;
    first = (unit + s.cta_of((int64_t)unit * s.nt)) * step + tile * kTileM +
            (pos - tile * s.tp) * a.group + (h - kvh * a.group);
  }
};

// Shared memory of CTA `rank` of this cluster.
__device__ __forceinline__ uint32_t cluster_at(uint32_t mine, int rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(mine), "r"(rank));
  return at;
}
__device__ __forceinline__ float cluster_read(uint32_t at) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ float4 cluster_read4(uint32_t at) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(at)
               : "memory");
  return x;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::
                   : "memory");
}

// Joins the pieces of a request where they are one cluster: each CTA's results
// (log of the sum, and the row) are in its shared memory at `lse` and `y`; a warp
// takes a head.
template <typename T>
__device__ void cluster_join(const SharedArgs& a, const OwnArgs& o, const float* lse,
                             const float* y, int b, int h0, int heads, int piece) {
  cluster_sync();
  const int lane = threadIdx.x & 31;
  const bool col = lane * 4 < a.dv;
  for (int h = piece * kWarps + (threadIdx.x >> 5); h < heads; h += o.pieces * kWarps) {
    float w = lane < o.pieces ? cluster_read(cluster_at(sptr(lse + h), lane)) * kLog2e : -INFINITY;
    float top = w;
#pragma unroll
    for (int s = 4; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    top = __shfl_sync(0xffffffffu, top, 0);
    w = ex2(w - (top == -INFINITY ? 0.f : top));
    float total = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
    for (int p = 0; p < o.pieces; ++p) {
      const float f = __shfl_sync(0xffffffffu, w, p);
      total += f;
      if (col && f != 0.f) {
        const float4 z = cluster_read4(cluster_at(sptr(y + h * a.dv + lane * 4), p));
        x[0] = fmaf(z.x, f, x[0]);
        x[1] = fmaf(z.y, f, x[1]);
        x[2] = fmaf(z.z, f, x[2]);
        x[3] = fmaf(z.w, f, x[3]);
      }
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    if (col) {
      T* out = (T*)a.out.p + b * a.out.row + (h0 + h) * a.out.head + lane * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) out[i] = narrow<T>(x[i] * inv);
    }
    if (lane == 0 && a.lse)
      a.lse[(int64_t)b * a.heads + h0 + h] =
          total == 0.f ? -INFINITY : fmaf(top, 0.6931471805599453f, logf(total));
  }
  cluster_sync();  // (no CTA leaves while its results are read)
}

// Joins the warps' results (log2 maxima m and sums l [warp][head], O
// [warp][head][dv]) and, where this CTA has all of the request's own keys, the
// prefix's pieces; thread = column.  heads: of this CTA, from h0.
template <typename T, int HB>
__device__ void join(const SharedArgs& a, const OwnArgs& o, const float* m, const float* l,
                     float* acc, int b, int h0, int heads, int piece) {
  float* cy = acc + kWarps * HB * a.dv;  // this CTA's results for its cluster
  float* cl = cy + HB * a.dv;
  for (int h = threadIdx.x >> 5; h < heads; h += kWarps) {
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)b * a.heads + h0 + h;
    const int64_t rows = (int64_t)a.n * a.heads;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m[w * HB + h]);
    // The prefix's pieces: lane = piece, log2 of their sums.
    const PrefixRow pre(a, o, b, h0 + h);
    const int np = o.pieces == 1 ? pre.pieces : 0;
    float pl[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (lane + 32 * i < np) pl[i] = o.part_lse[pre.first + (lane + 32 * i) * pre.step] * kLog2e;
    float pt = fmaxf(pl[0], pl[1]);
#pragma unroll
    for (int s = 16; s; s >>= 1) pt = fmaxf(pt, __shfl_xor_sync(0xffffffffu, pt, s));
    top = fmaxf(top, pt);
    const float ref = top == -INFINITY ? 0.f : top;
    float wf[kWarps], total = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      wf[w] = ex2(m[w * HB + h] - ref);
      total = fmaf(l[w * HB + h], wf[w], total);
    }
    // (A piece's NaN must not vanish in the maximum: its factor is NaN.)
    float pf[2] = {0.f, 0.f}, ps;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (lane + 32 * i < np) pf[i] = ex2(pl[i] - ref);
    ps = pf[0] + pf[1];
#pragma unroll
    for (int s = 16; s; s >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, s);
    total += ps;
    const float inv = total == 0.f ? 0.f : 1.f / total;
    float y[4] = {0.f, 0.f, 0.f, 0.f};  // columns lane * 4 ..
    const bool col = lane * 4 < a.dv;
    if (col) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(acc + (w * HB + h) * a.dv + lane * 4);
        y[0] = fmaf(x.x, wf[w], y[0]);
        y[1] = fmaf(x.y, wf[w], y[1]);
        y[2] = fmaf(x.z, wf[w], y[2]);
        y[3] = fmaf(x.w, wf[w], y[3]);
      }
    }
#pragma unroll 4
    for (int p = 0; p < np; ++p) {
      const float f = __shfl_sync(0xffffffffu, p < 32 ? pf[0] : pf[1], p & 31);
      if (col && f != 0.f) {
        const float4 x = *reinterpret_cast<const float4*>(o.part + (pre.first + p * pre.step) * a.dv + lane * 4);
        y[0] = fmaf(x.x, f, y[0]);
        y[1] = fmaf(x.y, f, y[1]);
        y[2] = fmaf(x.z, f, y[2]);
        y[3] = fmaf(x.w, f, y[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] *= inv;
    const float lse = total == 0.f ? -INFINITY : fmaf(top, 0.6931471805599453f, logf(total));
    if (o.pieces == 1) {
      if (col) {
        T* out = (T*)a.out.p + b * a.out.row + (h0 + h) * a.out.head + lane * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = narrow<T>(y[i]);
      }
      if (lane == 0 && a.lse) a.lse[row] = lse;
    } else if (o.cluster) {
      if (col) *reinterpret_cast<float4*>(cy + h * a.dv + lane * 4) = make_float4(y[0], y[1], y[2], y[3]);
      if (lane == 0) cl[h] = lse;
    } else {
      const int64_t at = (int64_t)piece * rows + row;
      if (col) *reinterpret_cast<float4*>(o.own + at * a.dv + lane * 4) = make_float4(y[0], y[1], y[2], y[3]);
      if (lane == 0) o.own_lse[at] = lse;
    }
  }
  if (o.cluster) cluster_join<T>(a, o, cl, cy, b, h0, heads, piece);
}

// ------------------------------------------------------------ bf16 and fp16
constexpr int kHeads16 = 16;      // MMA rows: heads of a CTA
constexpr int kKeys16 = 16;       // keys of a warp's tile
constexpr int kStages16 = 2;
constexpr int kRow16 = 272;       // bytes of a row in shared memory: 256 + 16, conflict-free
constexpr int kStage16 = 2 * kKeys16 * kRow16;
constexpr int kSmem16 = kWarps * kStages16 * kStage16;
static_assert(kSmem16 >= ((kWarps + 1) * kHeads16 * 129 + kWarps * kHeads16) * 4, "results to join");

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
  if (Type16<T>::kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Grid: x = pieces, y = KV heads x blocks of 16 heads, z-major requests in x.
template <typename T>
__global__ void __launch_bounds__(kThreads, 3) own16_kernel(SharedArgs a, OwnArgs o) {
  extern __shared__ __align__(128) unsigned char sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int piece = blockIdx.x % o.pieces, b = blockIdx.x / o.pieces;
  const int blocks = (a.group + kHeads16 - 1) / kHeads16;
  const int kvh = blockIdx.y / blocks, hb = blockIdx.y - kvh * blocks;
  const int h0 = kvh * a.group + hb * kHeads16;
  const int heads = min(kHeads16, a.group - hb * kHeads16);
  int lo, hi;
  let_next_start();
  // Pieces need nothing of the prefix's launch and leave at once, so that the
  // rest of this grid gets their places while that one runs; one CTA waits for
  // it, so that this grid does not end before it.
  const bool waits = o.pieces == 1 || (blockIdx.x == 0 && blockIdx.y == 0);
  if (!own_range(a, o, b, piece, lo, hi)) {
    if (waits) wait_for_previous();
    if (!o.cluster) return;
  }
  const int32_t* pages = a.table + (int64_t)b * a.width;
  const int dc = a.d >> 3, vc = a.dv >> 3;  // 16-byte chunks of a row
  const int ks = (a.d + 15) >> 4, ns = (a.dv + 15) >> 4;
  unsigned char* ring = sm + warp * kStages16 * kStage16;
  // Columns that pad a dim to 16 hold zeros.
  if ((a.d | a.dv) & 15) {
    for (int i = tid * 16; i < kSmem16; i += kThreads * 16)
      *reinterpret_cast<uint4*>(sm + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  // Two tiles a block of 32 keys.
  const int blocks32 = (hi - lo + 31) / 32;
  const int mine = 2 * (blocks32 > warp ? (blocks32 - warp + kWarps - 1) / kWarps : 0);
  auto key_of = [&](int t) { return lo + ((t >> 1) * kWarps + warp) * 32 + (t & 1) * kKeys16; };
  RowAhead row;
  row.next = own_row(a, o, pages, key_of(0) + lane, hi, kvh);
  const unsigned char* kb = (const unsigned char*)a.k + (lane & 15) * 16;
  const unsigned char* vb = (const unsigned char*)a.v + (lane & 15) * 16;
  const bool kcol = (lane & 15) < dc, vcol = (lane & 15) < vc;
  auto fetch = [&](int t) {
    if (t < mine) {
      if (!(t & 1)) {
        row.now = row.next;
        row.next = own_row(a, o, pages, key_of(t + 2) + lane, hi, kvh);
      }
      const uint32_t st = sptr(ring + (t % kStages16) * kStage16) + (lane >> 4) * kRow16 + (lane & 15) * 16;
#pragma unroll
      for (int i = 0; i < kKeys16; i += 2) {
        const uint32_t at = __shfl_sync(0xffffffffu, row.now, (t & 1) * kKeys16 + i + (lane >> 4));
        const bool have = at != kNoRow;
        const uint64_t r = have ? at : 0;
        if (kcol) cp16(st + i * kRow16, kb + r * (uint32_t)(a.d * 2), have);
        if (vcol) cp16(st + (kKeys16 + i) * kRow16, vb + r * (uint32_t)(a.dv * 2), have);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int t = 0; t < kStages16 - 1; ++t) fetch(t);

  // The queries, as A fragments: rows lane / 4 and + 8, zero past the heads.
  uint32_t q[8][4];
  {
    const int r = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int hh = r + (x & 1) * 8, cc = k * 16 + c + (x >> 1) * 8;
        q[k][x] = 0;
        if (hh < heads && cc < a.d)
          q[k][x] = *reinterpret_cast<const uint32_t*>((const T*)a.q.p + b * a.q.row +
                                                       (h0 + hh) * a.q.head + cc);
      }
  }
  const float sc = a.scale * kLog2e;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float acc[16][4];
#pragma unroll
  for (int n = 0; n < 16; ++n)
#pragma unroll
    for (int x = 0; x < 4; ++x) acc[n][x] = 0.f;

  for (int t = 0; t < mine; ++t) {
    cp_wait<kStages16 - 2>();
    __syncwarp();
    fetch(t + kStages16 - 1);
    const uint32_t ks_at = sptr(ring + (t % kStages16) * kStage16), vs_at = ks_at + kKeys16 * kRow16;
    float s[2][4] = {};
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < ks) {
        uint32_t r[4];
        ldsm4(r, ks_at + ((lane & 7) + (lane >> 4) * 8) * kRow16 + k * 32 + ((lane >> 3) & 1) * 16);
        mma16<T>(s[0], q[k], r[0], r[1]);
        mma16<T>(s[1], q[k], r[2], r[3]);
      }
    const int left = hi - key_of(t);  // keys of this tile
    uint32_t p[4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {  // rows lane / 4 and lane / 4 + 8
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (n * 8 + (lane & 3) * 2 + e >= left) s[n][x * 2 + e] = -INFINITY;
      float top = fmaxf(fmaxf(s[0][x * 2], s[0][x * 2 + 1]), fmaxf(s[1][x * 2], s[1][x * 2 + 1]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)) * sc;
      const bool grow = m[x] == -INFINITY ? top > m[x] : top - m[x] > kLazy;
      if (__any_sync(0xffffffffu, grow)) {
        const float nm = fmaxf(m[x], top);
        const float f = nm == m[x] ? 1.f : ex2(m[x] - nm);
        m[x] = nm;
        l[x] *= f;
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          acc[n][x * 2] *= f;
          acc[n][x * 2 + 1] *= f;
        }
      }
      const float ref = (m[x] == -INFINITY ? 0.f : m[x]) - Type16<T>::kLift;
      float w[4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          w[n * 2 + e] = ex2(fmaf(s[n][x * 2 + e], sc, -ref));
          l[x] += w[n * 2 + e];
        }
      p[x] = Type16<T>::pack(w[0], w[1]);
      p[2 + x] = Type16<T>::pack(w[2], w[3]);
    }
#pragma unroll
    for (int n = 0; n < 8; ++n)
      if (n < ns) {
        uint32_t r[4];
        ldsm4t(r, vs_at + ((lane & 7) + ((lane >> 3) & 1) * 8) * kRow16 + n * 32 + (lane >> 4) * 16);
        mma16<T>(acc[2 * n], p, r[0], r[1]);
        mma16<T>(acc[2 * n + 1], p, r[2], r[3]);
      }
  }
  cp_wait<0>();
  if (waits) wait_for_previous();  // the prefix's pieces, which this kernel ran beside
  __syncthreads();                 // the ring becomes the warps' results
  float* jm = reinterpret_cast<float*>(sm);
  float* jl = jm + kWarps * kHeads16;
  float* ja = jl + kWarps * kHeads16;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    const int h = (lane >> 2) + x * 8;
    if (h < heads) {
      if ((lane & 3) == 0) {
        jm[warp * kHeads16 + h] = m[x] - Type16<T>::kLift;  // (what the weights refer to)
        jl[warp * kHeads16 + h] = l[x];
      }
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        const int c = n * 8 + (lane & 3) * 2;
        if (c < a.dv)
          *reinterpret_cast<float2*>(ja + (warp * kHeads16 + h) * a.dv + c) =
              make_float2(acc[n][x * 2], acc[n][x * 2 + 1]);
      }
    }
  }
  __syncthreads();
  join<T, kHeads16>(a, o, jm, jl, ja, b, h0, heads, piece);
}

// --------------------------------------------------------------------- f32
constexpr int kKeys32 = 8;
constexpr int kStages32 = 2;
constexpr int kStage32 = 2 * kKeys32 * 512;
constexpr int kSmem32 = kWarps * kStages32 * kStage32;
static_assert(kSmem32 >= ((kWarps + 1) * 8 * 129 + kWarps * 8) * 4, "results to join");

// Sums each of V per-lane partials over the warp; lane gets the total of value
// value_of<V>(lane).
template <int V>
__device__ __forceinline__ float sum_multi(float (&x)[V], int lane) {
  constexpr int kSteps = V >= 32 ? 5 : V >= 16 ? 4 : V >= 8 ? 3 : 2;
#pragma unroll
  for (int st = 0; st < kSteps; ++st) {
    const int half = V >> (st + 1), off = 16 >> st;
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? x[i] : x[i + half];
      const float keep = up ? x[i + half] : x[i];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
    }
  }
  float r = x[0];
#pragma unroll
  for (int off = 16 >> kSteps; off; off >>= 1) r += __shfl_xor_sync(0xffffffffu, r, off);
  return r;
}

// HT heads at a time.  A value is (head, key) = head * KB + key: its lanes
// are the top bits of the lane number, so a head's keys are neighbours.
template <int HT>
__global__ void __launch_bounds__(kThreads, 3) own32_kernel(SharedArgs a, OwnArgs o) {
  extern __shared__ __align__(128) unsigned char sm[];
  constexpr int KB = HT == 8 ? 4 : 8;  // keys of one butterfly
  constexpr int V = HT * KB;
  constexpr int kRep = 32 / V;         // lanes that hold one value
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int piece = blockIdx.x % o.pieces, b = blockIdx.x / o.pieces;
  const int blocks = (a.group + HT - 1) / HT;
  const int kvh = blockIdx.y / blocks, hb = blockIdx.y - kvh * blocks;
  const int h0 = kvh * a.group + hb * HT;
  const int heads = min(HT, a.group - hb * HT);
  int lo, hi;
  let_next_start();
  // Pieces need nothing of the prefix's launch and leave at once, so that the
  // rest of this grid gets their places while that one runs; one CTA waits for
  // it, so that this grid does not end before it.
  const bool waits = o.pieces == 1 || (blockIdx.x == 0 && blockIdx.y == 0);
  if (!own_range(a, o, b, piece, lo, hi)) {
    if (waits) wait_for_previous();
    if (!o.cluster) return;
  }
  const int32_t* pages = a.table + (int64_t)b * a.width;
  const bool kcol = lane * 4 < a.d, vcol = lane * 4 < a.dv;
  unsigned char* ring = sm + warp * kStages32 * kStage32 + lane * 16;  // this lane's columns
  // Four tiles a block of 32 keys.
  const int blocks32 = (hi - lo + 31) / 32;
  const int mine = 4 * (blocks32 > warp ? (blocks32 - warp + kWarps - 1) / kWarps : 0);
  auto key_of = [&](int t) { return lo + ((t >> 2) * kWarps + warp) * 32 + (t & 3) * kKeys32; };
  RowAhead row;
  row.next = own_row(a, o, pages, key_of(0) + lane, hi, kvh);
  const float4* kb = (const float4*)a.k + (kcol ? lane : 0);
  const float4* vb = (const float4*)a.v + (vcol ? lane : 0);
  auto fetch = [&](int t) {
    if (t < mine) {
      if (!(t & 3)) {
        row.now = row.next;
        row.next = own_row(a, o, pages, key_of(t + 4) + lane, hi, kvh);
      }
      const uint32_t st = sptr(ring + (t % kStages32) * kStage32);
#pragma unroll
      for (int i = 0; i < kKeys32; ++i) {
        const uint32_t at = __shfl_sync(0xffffffffu, row.now, (t & 3) * kKeys32 + i);
        const bool have = at != kNoRow;
        const uint64_t r = have ? at : 0;
        if (kcol) cp16(st + i * 512, kb + r * (uint32_t)(a.d >> 2), have);
        if (vcol) cp16(st + (kKeys32 + i) * 512, vb + r * (uint32_t)(a.dv >> 2), have);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int t = 0; t < kStages32 - 1; ++t) fetch(t);

  const float sc = a.scale * kLog2e;
  uint64_t q[HT][2], acc[HT][2];  // four columns as two pairs
#pragma unroll
  for (int h = 0; h < HT; ++h) {
    q[h][0] = q[h][1] = acc[h][0] = acc[h][1] = pair(0.f, 0.f);
    if (h < heads && kcol) {
      const float* p = (const float*)a.q.p + b * a.q.row + (h0 + h) * a.q.head + lane * 4;
      q[h][0] = pair(p[0] * sc, p[1] * sc);
      q[h][1] = pair(p[2] * sc, p[3] * sc);
    }
  }
  const int my_key = lane / kRep % KB;  // of this lane's (head, key) pair
  float m = -INFINITY, l = 0.f;                    // of this lane's head
  for (int t = 0; t < mine; ++t) {
    cp_wait<kStages32 - 2>();  // (each lane reads back what it copied itself)
    fetch(t + kStages32 - 1);
    const unsigned char* st = ring + (t % kStages32) * kStage32;
#pragma unroll
    for (int g = 0; g < kKeys32; g += KB) {
      const int left = hi - key_of(t) - g;
      float x[V];
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        const float4 k = kcol ? *reinterpret_cast<const float4*>(st + (g + i) * 512)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int h = 0; h < HT; ++h) {
          float x0, x1;
          unpair(fma2(q[h][0], pair(k.x, k.y), mul2(q[h][1], pair(k.z, k.w))), x0, x1);
          x[h * KB + i] = x0 + x1;
        }
      }
      float s = sum_multi<V>(x, lane);
      if (my_key >= left) s = -INFINITY;
      float top = s;
#pragma unroll
      for (int off = kRep * KB / 2; off >= kRep; off >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const bool grow = m == -INFINITY ? top > m : top - m > kLazy;
      if (__any_sync(0xffffffffu, grow)) {
        const float nm = fmaxf(m, top);
        const float f = nm == m ? 1.f : ex2(m - nm);
        m = nm;
        l *= f;
#pragma unroll
        for (int h = 0; h < HT; ++h) {
          const float fh = __shfl_sync(0xffffffffu, f, h * KB * kRep);
          acc[h][0] = mul2(acc[h][0], pair(fh, fh));
          acc[h][1] = mul2(acc[h][1], pair(fh, fh));
        }
      }
      const float p = ex2(s - (m == -INFINITY ? 0.f : m));
      l += p;
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        const float4 v = vcol ? *reinterpret_cast<const float4*>(st + (kKeys32 + g + i) * 512)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int h = 0; h < HT; ++h) {
          const float w = __shfl_sync(0xffffffffu, p, (h * KB + i) * kRep);
          acc[h][0] = fma2(pair(w, w), pair(v.x, v.y), acc[h][0]);
          acc[h][1] = fma2(pair(w, w), pair(v.z, v.w), acc[h][1]);
        }
      }
    }
  }
  // l: the sum over a head's keys (lanes kRep apart).
#pragma unroll
  for (int off = kRep * KB / 2; off >= kRep; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  cp_wait<0>();
  if (waits) wait_for_previous();
  __syncthreads();
  float* jm = reinterpret_cast<float*>(sm);
  float* jl = jm + kWarps * HT;
  float* ja = jl + kWarps * HT;
#pragma unroll
  for (int h = 0; h < HT; ++h) {
    if (lane == h * KB * kRep) {
      jm[warp * HT + h] = m;
      jl[warp * HT + h] = l;
    }
    if (vcol)
      *reinterpret_cast<ulonglong2*>(ja + (warp * HT + h) * a.dv + lane * 4) =
          make_ulonglong2(acc[h][0], acc[h][1]);
  }
  __syncthreads();
  join<float, HT>(a, o, jm, jl, ja, b, h0, heads, piece);
}

// Joins the prefix's and the own pieces of each row; one warp a row.
template <typename T>
__global__ void __launch_bounds__(kThreads) join_kernel(SharedArgs a, OwnArgs o) {
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.n * a.heads;
  for (int64_t r = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); r < rows;
       r += (int64_t)gridDim.x * kWarps) {
    const int b = (int)(r / a.heads), h = (int)(r - (int64_t)b * a.heads);
    const PrefixRow pre(a, o, b, h);
    const int len = o.lead + own_len(a, b, false), keys = piece_keys(o, len);
    const int np = pre.pieces, own = (len + keys - 1) / keys, all = np + own;
    auto lse_of = [&](int p) {
      return p < np ? o.part_lse[pre.first + p * pre.step] : o.own_lse[(p - np) * rows + r];
    };
    auto row_of = [&](int p) {
      return (p < np ? o.part + (pre.first + p * pre.step) * a.dv : o.own + ((p - np) * rows + r) * a.dv) +
             lane * 4;
    };
    // Lane = piece (at most 128): its weight against the largest.
    float w[4], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = lane + 32 * i < all ? lse_of(lane + 32 * i) * kLog2e : -INFINITY;
      top = fmaxf(top, w[i]);
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    const float ref = top == -INFINITY ? 0.f : top;
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = ex2(w[i] - ref);
      total += w[i];
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) total += __shfl_xor_sync(0xffffffffu, total, s);
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    const bool col = lane * 4 < a.dv;
#pragma unroll 8
    for (int p = 0; p < all; ++p) {
      const float f = __shfl_sync(0xffffffffu, p < 32 ? w[0] : p < 64 ? w[1] : p < 96 ? w[2] : w[3], p & 31);
      if (col && f != 0.f) {
        const float4 x = *reinterpret_cast<const float4*>(row_of(p));
        y[0] = fmaf(x.x, f, y[0]);
        y[1] = fmaf(x.y, f, y[1]);
        y[2] = fmaf(x.z, f, y[2]);
        y[3] = fmaf(x.w, f, y[3]);
      }
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    if (col) {
      T* out = (T*)a.out.p + b * a.out.row + h * a.out.head + lane * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) out[i] = narrow<T>(y[i] * inv);
    }
    if (lane == 0 && a.lse)
      a.lse[r] = total == 0.f ? -INFINITY : fmaf(top, 0.6931471805599453f, logf(total));
  }
}

// Joins the pieces of a prompt's cut units: blockIdx.x is the unit, a warp takes a
// row (16 CTAs a unit: a row is a chain of a few dependent reads, so rows have to
// be many at once).
template <typename T>
__global__ void __launch_bounds__(256) tail_join_kernel(const __grid_constant__ TileArgs a, int ctas) {
  __shared__ Unit su;
  __shared__ Tail st;
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp == 0) {
    Tail t;
    t.find(a, ctas, lane);
    Unit u;
    u.valid = 0;
    if ((int)blockIdx.x < t.units) {
      UnitWalk w;
      w.load(a, lane);
      w.get(a, t.full + blockIdx.x, lane, u);
    }
    if (lane == 0) {
      su = u;
      st = t;
    }
  }
  __syncthreads();
  if (!su.valid) return;
  const int64_t step = (int64_t)a.per * kTileM;
  const int cut = cut_pieces(su, st.cut);
  for (int row = blockIdx.y * 8 + warp; row < (su.np1 > 0 ? 2 : 1) * kTileM; row += 8 * gridDim.y) {
    const int tile = row / kTileM, r = row - tile * kTileM, pos = r / a.group;
    if (pos >= (tile ? su.np1 : su.np0)) continue;
    const int h = su.kvh * a.group + (r - pos * a.group);
    const int64_t orow = (int64_t)su.q_row + tile * a.tp + pos;
    const int64_t first = blockIdx.x * (int64_t)st.cut * step + row;
    float top = -INFINITY, w[5];  // lane = piece (at most 152)
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      w[i] = lane + 32 * i < cut ? a.part_lse[first + (lane + 32 * i) * step] * kLog2e : -INFINITY;
      top = fmaxf(top, w[i]);
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    const float ref = top == -INFINITY ? 0.f : top;
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      w[i] = ex2(w[i] - ref);
      total += w[i];
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) total += __shfl_xor_sync(0xffffffffu, total, s);
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    const bool col = lane * 4 < a.dv;
#pragma unroll 8
    for (int p = 0; p < cut; ++p) {
      const float f = __shfl_sync(0xffffffffu, p < 32 ? w[0] : p < 64 ? w[1] : p < 96 ? w[2] : p < 128 ? w[3] : w[4], p & 31);
      if (col && f != 0.f) {
        const float4 x = *reinterpret_cast<const float4*>(a.part + (first + p * step) * a.dv + lane * 4);
        y[0] = fmaf(x.x, f, y[0]);
        y[1] = fmaf(x.y, f, y[1]);
        y[2] = fmaf(x.z, f, y[2]);
        y[3] = fmaf(x.w, f, y[3]);
      }
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    if (col) {
      T* out = (T*)a.out.p + orow * a.out.row + h * a.out.head + lane * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) out[i] = narrow<T>(y[i] * inv);
    }
    if (lane == 0 && a.lse)
      a.lse[orow * a.heads + h] = total == 0.f ? -INFINITY : fmaf(top, 0.6931471805599453f, logf(total));
  }
}

// Beside the prefix's launch where there is one; with a request's pieces as
// clusters where they join themselves.
cudaError_t launch_own_kernel(void (*kernel)(SharedArgs, OwnArgs), dim3 grid, size_t smem,
                              cudaStream_t stream, const SharedArgs& a, const OwnArgs& o) {
  if (o.shares.units > 0) return launch_dependent(kernel, grid, kThreads, smem, stream, a, o);
  if (o.cluster) {
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)o.pieces;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, a, o);
  }
  kernel<<<grid, kThreads, smem, stream>>>(a, o);
  return cudaGetLastError();
}

template <int HT>
cudaError_t launch32(const SharedArgs& a, const OwnArgs& o, cudaStream_t stream) {
  const cudaError_t ready = ensure_smem<own32_kernel<HT>>(kSmem32);
  if (ready != cudaSuccess) return ready;
  const dim3 grid((unsigned)(a.n * o.pieces), (unsigned)(a.kv_heads * ((a.group + HT - 1) / HT)));
  return launch_own_kernel(own32_kernel<HT>, grid, kSmem32, stream, a, o);
}
template <typename T>
cudaError_t launch16(const SharedArgs& a, const OwnArgs& o, cudaStream_t stream) {
  const cudaError_t ready = ensure_smem<own16_kernel<T>>(kSmem16);
  if (ready != cudaSuccess) return ready;
  const dim3 grid((unsigned)(a.n * o.pieces),
                  (unsigned)(a.kv_heads * ((a.group + kHeads16 - 1) / kHeads16)));
  return launch_own_kernel(own16_kernel<T>, grid, kSmem16, stream, a, o);
}

}  // namespace

cudaError_t launch_own(const SharedArgs& a, const OwnArgs& o, cudaStream_t stream) {
  if (a.dtype == NYS_BF16) return launch16<__nv_bfloat16>(a, o, stream);
  if (a.dtype == NYS_F16) return launch16<__half>(a, o, stream);
  return a.group == 1   ? launch32<1>(a, o, stream)
         : a.group == 2 ? launch32<2>(a, o, stream)
         : a.group <= 4 ? launch32<4>(a, o, stream)
                        : launch32<8>(a, o, stream);
}

cudaError_t launch_join(const SharedArgs& a, const OwnArgs& o, cudaStream_t stream) {
  const int64_t want = ((int64_t)a.n * a.heads + kWarps - 1) / kWarps;
  const unsigned grid = (unsigned)(want < 152 * 16 ? want : 152 * 16);
  void (*kernel)(SharedArgs, OwnArgs) = a.dtype == NYS_F32    ? join_kernel<float>
                                        : a.dtype == NYS_BF16 ? join_kernel<__nv_bfloat16>
                                                              : join_kernel<__half>;
  return launch_dependent(kernel, grid, kThreads, 0, stream, a, o);
}

cudaError_t launch_tail_join(const TileArgs& a, int dtype, unsigned ctas, cudaStream_t stream) {
  void (*kernel)(TileArgs, int) = dtype == NYS_F32    ? tail_join_kernel<float>
                                  : dtype == NYS_BF16 ? tail_join_kernel<__nv_bfloat16>
                                                      : tail_join_kernel<__half>;
  return launch_dependent(kernel, dim3(ctas / 2, 16), 256, 0, stream, a, (int)ctas);
}

}  // namespace nys
