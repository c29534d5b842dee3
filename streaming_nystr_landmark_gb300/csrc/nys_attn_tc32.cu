// Exact attention on the tensor cores, f32.
//
// The formulas are those of nys_attn_tc.cu.  An f32 operand x is taken as a
// pair of fp16 pieces of x' = x 2^-e: hi = x' cut to 11 bits, lo = x' - hi
// rounded to 11 bits, so that x' = hi + lo to 2^-22; a product takes three
// tcgen05 products, lo hi + hi lo + hi hi (the dropped lo lo is below 2^-20 of
// |x y| at worst, 2^-23 in the mean), summed in f32 in tensor memory, small
// ones first.  The exponent e is common to 16 rows (those that one warp
// converts) and puts their largest value at 2^13, where fp16 keeps 22 bits of
// everything down to 2^-27 of it.
//
//   S' = Q' K'^T gives s_ij = S' 2^(eq + ek) scale log2(e), one multiplier a
//   group of 16 keys.  The value's exponent goes into the weight:
//   P_ij = 2^(s_ij + ev_j - m_i + 6), m_i the running maximum of s + ev, so
//   that P V' is the plain sum at scale 2^(6 - m_i); l_i += P_ij 2^-ev_j.
//   P is split into two pieces as the operands are; the 6 keeps small weights
//   above fp16's smallest numbers (P stays below 2^14).
//
// The tensor cores cut sums towards zero, so O is taken out after each tile of
// 128 keys (24 sums) and added to f32 accumulators in registers; a long row
// gathers no drift.
//
// One CTA of 512 threads a SM works on one query tile of 128 rows (positions x
// heads of the group): warps 0-3 softmax and accumulation (thread = row, 128
// accumulators), 4-11 load f32 rows and convert them into the swizzled tiles
// (16 rows a warp, the next tile's loads in flight while this one is
// converted), 12 products, 13 units of work.  Registers move from the others
// to the softmax.  Shared memory: Q, K and V, each a hi and a lo tile of 32 KB.
// Products of tile j + 1's scores run during tile j's softmax, and K (V) is
// converted while the value (score) products run, so single buffers suffice.
// Tensor memory: two S and two O of 128 columns; P hi and lo take S's place, 8
// columns each for 16 keys.
//
// Rows that are not in the sequence are zeros and never read.  Values that are
// not finite where some row of the tile does not see their key are replaced
// by 0 and added in the epilogue to the rows that see them.
//
// Every wait is bounded (2 s), as in nys_attn_tc.cu.
#include <cmath>

#include "nys_attn_tc.h"

namespace nys {
namespace {

using namespace tc;

constexpr int kThreads = 512;
constexpr int kConv = 8;        // converting warps
constexpr int kConvRows = 16;   // rows of one of them
constexpr uint32_t kPiece = 32768;
constexpr uint32_t kOffK = 2 * kPiece, kOffV = 4 * kPiece, kTiles = 6 * kPiece;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.f;
constexpr float kLift = 6.f;
constexpr int kTop = 13;        // the largest value's power of two after scaling

struct Shared {
  uint64_t q_full, q_empty, k_full, k_empty, v_full, v_empty;
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2], x_full[2];
  uint64_t u_full[kUnitRing], u_empty[kUnitRing];
  uint64_t drain;
  Unit unit[kUnitRing];
  float q_mul[2][kConv];             // 2^eq, [unit & 1][16 rows]
  float k_mul[4][kConv];             // 2^ek, [tile & 3][16 keys]
  float v_exp[4][kConv], v_inv[4][kConv];  // ev, 2^-ev
  uint32_t tmem;
  int abort;
};
constexpr uint32_t kSmem = kTiles + sizeof(Shared);
static_assert(kSmem <= 227 * 1024, "one CTA's shared memory");

enum { kJobQ = 0, kJobK = 1, kJobV = 2 };

// Step e of a unit's conversions: Q K0 V0 K1 K2 V1 K3 V2 .. (K of the tile
// after next, once its scores' predecessor is done, before the next V).
__device__ __forceinline__ void job_of(int e, int nt, int& what, int& j) {
  if (e == 0) {
    what = kJobQ;
    j = 0;
  } else if (e == 2 * nt) {
    what = kJobV;
    j = nt - 1;
  } else if (e < 4) {
    what = e == 2 ? kJobV : kJobK;
    j = e == 3 ? 1 : 0;
  } else {
    what = (e & 1) ? kJobV : kJobK;
    j = (e & 1) ? (e - 3) >> 1 : e >> 1;
  }
}

// Offset (elements) of row r of a job's tile in its tensor, -1: zeros.
template <bool PAGED>
__device__ __forceinline__ int64_t job_row(const TileArgs& a, const Unit& u, int what, int j,
                                           int r) {
  if (what == kJobQ) {
    const int pos = r / a.group, hd = r - pos * a.group;
    if (pos >= u.np0) return -1;
    return (u.q_row + (int64_t)pos) * a.q.row + (int64_t)(u.kvh * a.group + hd) * a.q.head;
  }
  const int key = u.kb + j * kTileN + r;
  if (key >= u.nkl) return -1;
  int64_t row = (int64_t)u.k_row + key;
  if (PAGED) {
    const int32_t pg = a.pages[key / a.page];
    if (pg < 0 || pg >= a.n_pages) {
      attn_report(a.status, NYS_ATTN_BAD_PAGE);
      return -1;
    }
    row = (int64_t)pg * a.page + key % a.page;
  }
  return what == kJobK ? row * a.k_row + u.kvh * a.k_head : row * a.v_row + u.kvh * a.v_head;
}

__device__ __forceinline__ float4 load4(const float* p) {
  return __ldg(reinterpret_cast<const float4*>(p));
}
__device__ __forceinline__ bool finite_bits(float x) {
  return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
}

// ---- conversion (eight warps; cw = 0 .. 7)
template <bool PAGED>
__device__ void convert_role(const TileArgs& a, Shared& sh, unsigned char* sm, int cw, int lane) {
  volatile int* ab = &sh.abort;
  uint32_t nu = 0, nq = 0, tile0 = 0, done_k = 0, done_v = 0;
  Unit u;
  // The next job: unit u, step e.  Skips units without keys.
  int e = 0;
  uint32_t held = 0;  // ring place of u
  auto next_unit = [&]() {
    for (;;) {
      if (!bar_wait_warp(&sh.u_full[nu % kUnitRing], (nu / kUnitRing) & 1, ab)) return false;
      held = nu % kUnitRing;
      u = sh.unit[held];
      ++nu;
      if (!u.valid) return false;
      if (u.nt > 0) return true;
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.u_empty[held]);
    }
  };
  const bool kcol = lane * 4 < a.d, vcol = lane * 4 < a.dv;
  const int r0 = cw * kConvRows;
  const float* base[3] = {(const float*)a.q.p + lane * 4, (const float*)a.k_raw + lane * 4,
                          (const float*)a.v_raw + lane * 4};
  float4 x[kConvRows];
  bool have = next_unit();
  if (!have) return;
  {
    const int64_t off = lane < kConvRows ? job_row<PAGED>(a, u, kJobQ, 0, r0 + lane) : -1;
#pragma unroll
    for (int r = 0; r < kConvRows; ++r) {
      const int64_t o = __shfl_sync(0xffffffffu, off, r);
      x[r] = o >= 0 && kcol ? load4(base[0] + o) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  // Where this lane's four columns lie in row r of a tile: 64-column block,
  // then 16-byte units exchanged by the row's low bits (128-byte swizzle).
  const uint32_t col_at = (uint32_t)(lane >> 4) * 16384u + (uint32_t)(lane & 1) * 8u;
  const uint32_t unit16 = (uint32_t)(lane & 15) >> 1;
  while (have) {
    int what, j;
    job_of(e, u.nt, what, j);
    const uint32_t tile = tile0 + (uint32_t)j;
    const Unit cur = u;
    const uint32_t cur_held = held, cur_nq = nq;
    // What comes after it.
    bool last = false;
    if (++e > 2 * u.nt) {
      last = true;
      tile0 += (uint32_t)u.nt;
      ++nq;
      e = 0;
      have = next_unit();
    }
    int nwhat = kJobQ, nj = 0;
    int64_t off = -1;
    if (have) {
      job_of(e, u.nt, nwhat, nj);
      if (lane < kConvRows) off = job_row<PAGED>(a, u, nwhat, nj, r0 + lane);
    }
    const float* nbase = base[nwhat];
    const bool ncol = have && (nwhat == kJobV ? vcol : kcol);

    // The rows' common exponent.
    float t0 = 0.f, t1 = 0.f;
#pragma unroll
    for (int r = 0; r < kConvRows; ++r) {
      t0 = max3(t0, fabsf(x[r].x), fabsf(x[r].y));
      t1 = max3(t1, fabsf(x[r].z), fabsf(x[r].w));
    }
    uint32_t top = __float_as_uint(fmaxf(t0, t1));
    bool odd = false;  // (fmaxf passes NaN by: sums keep it)
    {
      float z = 0.f;
#pragma unroll
      for (int r = 0; r < kConvRows; ++r)
        z += (x[r].x * 0.f + x[r].y * 0.f) + (x[r].z * 0.f + x[r].w * 0.f);
      odd = __any_sync(0xffffffffu, z != 0.f);  // NaN: some value is not finite
    }
    if (odd) {
      float f = 0.f;
#pragma unroll
      for (int r = 0; r < kConvRows; ++r) {
        const float y[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (finite_bits(y[i])) f = fmaxf(f, fabsf(y[i]));
      }
      top = __float_as_uint(f);
      // Values that some row does not see: out, and added in the epilogue.
      if (what == kJobV && j >= cur.edge) {
#pragma unroll
        for (int r = 0; r < kConvRows; ++r) {
          if (!finite_bits(x[r].x)) x[r].x = 0.f;
          if (!finite_bits(x[r].y)) x[r].y = 0.f;
          if (!finite_bits(x[r].z)) x[r].z = 0.f;
          if (!finite_bits(x[r].w)) x[r].w = 0.f;
        }
        if (lane == 0) *(volatile int*)&sh.unit[cur_held].patch = 1;
        odd = false;
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    int ex = (int)(top >> 23);          // biased
    if (ex == 0) ex = 127;              // all zero: any scale
    if (ex < 40) ex = 40;
    const float scale = __uint_as_float((uint32_t)(254 + kTop - ex) << 23);  // 2^(13 - (ex - 127))
    const float back = __uint_as_float((uint32_t)(ex - kTop) << 23);
    if (lane == 0) {
      if (what == kJobQ) {
        sh.q_mul[cur_nq & 1][cw] = back;
      } else if (what == kJobK) {
        sh.k_mul[tile & 3][cw] = back;
      } else {
        sh.v_exp[tile & 3][cw] = (float)(ex - 127 - kTop);
        sh.v_inv[tile & 3][cw] = scale;
        bar_arrive(&sh.x_full[tile & 1]);
      }
    }
    bool ok;
    if (what == kJobQ) ok = bar_wait_warp(&sh.q_empty, (cur_nq & 1) ^ 1, ab);
    else if (what == kJobK) ok = bar_wait_warp(&sh.k_empty, (done_k++ & 1) ^ 1, ab);
    else ok = bar_wait_warp(&sh.v_empty, (done_v++ & 1) ^ 1, ab);
    if (!ok) return;
    unsigned char* t = sm + what * 2 * kPiece + col_at;
    const int cols = what == kJobV ? a.dv : a.d;
    const bool put = lane * 4 < ((cols + 15) & ~15);
#pragma unroll
    for (int r = 0; r < kConvRows; ++r) {
      const int row = r0 + r;
      const uint32_t at = (uint32_t)row * 128u + ((unit16 ^ (uint32_t)(row & 7)) << 4);
      float y[4] = {x[r].x * scale, x[r].y * scale, x[r].z * scale, x[r].w * scale};
      float h[4], l[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[i] = __uint_as_float(__float_as_uint(y[i]) & 0xFFFFE000u);
        l[i] = y[i] - h[i];
      }
      if (odd) {  // infinities and NaN stay what they are, alone in hi
        const float z[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!finite_bits(z[i])) {
            h[i] = z[i];
            l[i] = 0.f;
          }
      }
      using H = Type16<__half>;
      if (put) {
        *reinterpret_cast<uint2*>(t + at) = make_uint2(H::pack(h[0], h[1]), H::pack(h[2], h[3]));
        *reinterpret_cast<uint2*>(t + kPiece + at) =
            make_uint2(H::pack(l[0], l[1]), H::pack(l[2], l[3]));
      }
      // The next job's row takes these registers.
      const int64_t o = __shfl_sync(0xffffffffu, off, r);
      x[r] = o >= 0 && ncol ? load4(nbase + o) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    proxy_fence();
    __syncwarp();
    if (lane == 0) {
      bar_arrive(what == kJobQ ? &sh.q_full : what == kJobK ? &sh.k_full : &sh.v_full);
      if (last) bar_arrive(&sh.u_empty[cur_held]);
    }
  }
}

// ---- products (one thread)
__device__ void mma_role(const TileArgs& a, Shared& sh, unsigned char* sm, uint32_t tmem) {
  volatile int* ab = &sh.abort;
  const int ks = (a.d + 15) / 16;
  const int nv = (a.dv + 15) & ~15;
  const uint32_t id_s = idesc(kTileM, kTileN, false, false);
  const uint32_t id_o = idesc(kTileM, nv, false, true);
  const uint32_t q0 = sptr(sm), k0 = sptr(sm + kOffK), v0 = sptr(sm + kOffV);
  uint32_t nu = 0, nq = 0, n_s = 0, n_o = 0;  // units, query tiles, score and value tiles begun
  bool ok = true;
  for (; ok; ++nu) {
    if (!bar_wait(&sh.u_full[nu % kUnitRing], (nu / kUnitRing) & 1, ab)) break;
    const int valid = sh.unit[nu % kUnitRing].valid, nt = sh.unit[nu % kUnitRing].nt;
    bar_arrive(&sh.u_empty[nu % kUnitRing]);
    if (!valid) break;
    if (nt == 0) continue;
    if (!bar_wait(&sh.q_full, nq & 1, ab)) break;
    ++nq;
    auto scores = [&](bool last) {
      if (!bar_wait(&sh.k_full, n_s & 1, ab)) return false;
      fence_after();
      const uint32_t d = tmem + (n_s & 1) * 128;
#pragma unroll 1
      for (int p = 0; p < 3; ++p) {  // lo hi, hi lo, hi hi
        const uint32_t q = q0 + (p == 0 ? kPiece : 0), k = k0 + (p == 1 ? kPiece : 0);
        for (int i = 0; i < ks; ++i) {
          const uint32_t off = (i >> 2) * 16384 + (i & 3) * 32;
          mma_ss(d, desc128(q + off, 16, 1024), desc128(k + off, 16, 1024), id_s, p + i > 0);
        }
      }
      commit(&sh.k_empty);
      commit(&sh.s_full[n_s & 1]);
      if (last) commit(&sh.q_empty);
      ++n_s;
      return true;
    };
    ok = scores(nt == 1);
    if (ok && nt > 1) ok = scores(nt == 2);
    for (int j = 0; j < nt && ok; ++j) {
      const uint32_t b = n_o & 1, ph = (n_o >> 1) & 1;
      ok = bar_wait(&sh.v_full, n_o & 1, ab) && bar_wait(&sh.p_full[b], ph, ab) &&
           bar_wait(&sh.o_empty[b], ph ^ 1, ab);
      if (!ok) break;
      fence_after();
      const uint32_t s = tmem + b * 128, o = tmem + 256 + b * 128;
#pragma unroll 1
      for (int p = 0; p < 3; ++p) {
        const uint32_t v = v0 + (p == 1 ? kPiece : 0), w = s + (p == 0 ? 8 : 0);
        for (int i = 0; i < kTileN / 16; ++i)
          mma_ts(o, w + i * 16, desc128(v + i * 2048, 16384, 1024), id_o,
                 p + i > 0);
      }
      commit(&sh.v_empty);
      commit(&sh.o_full[b]);
      ++n_o;
      if (j + 2 < nt) ok = scores(j + 3 == nt);
    }
  }
  int none = 0;
  commit(&sh.drain);
  bar_wait(&sh.drain, 0, &none);
}

__device__ void unit_role(const TileArgs& a, Shared& sh, int lane) {
  volatile int* ab = &sh.abort;
  UnitWalk walk;
  walk.load(a, lane);
  for (uint32_t nu = 0;; ++nu) {
    const int64_t w = (int64_t)nu * gridDim.x +
                      ((nu & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    Unit u;
    walk.get(a, w, lane, u);
    if (!bar_wait_warp(&sh.u_empty[nu % kUnitRing], ((nu / kUnitRing) & 1) ^ 1, ab)) return;
    if (lane == 0) {
      sh.unit[nu % kUnitRing] = u;
      bar_arrive(&sh.u_full[nu % kUnitRing]);
    }
    __syncwarp();
    if (!u.valid) return;
  }
}

template <bool PAGED>
__device__ __forceinline__ const float* value_row(const TileArgs& a, const Unit& u, int j) {
  int64_t row = (int64_t)u.k_row + j;
  if (PAGED) {
    const int32_t pg = a.pages[j / a.page];
    if (pg < 0 || pg >= a.n_pages) return nullptr;
    row = (int64_t)pg * a.page + j % a.page;
  }
  return (const float*)a.v_raw + row * a.v_row + u.kvh * a.v_head;
}

// ---- softmax, accumulation and results (one warpgroup, thread = row)
template <bool PAGED>
__device__ void row_role(const TileArgs& a, Shared& sh, uint32_t tmem, int row, int lane) {
  volatile int* ab = &sh.abort;
  const float sc = a.scale * kLog2e;
  const int pos = row / a.group, hd = row - pos * a.group;
  const uint32_t at = tmem + ((uint32_t)(row & ~31) << 16);
  uint32_t n = 0, nq = 0;  // tiles, query tiles
  for (uint32_t nu = 0;; ++nu) {
    if (!bar_wait_warp(&sh.u_full[nu % kUnitRing], (nu / kUnitRing) & 1, ab)) return;
    const Unit& u = sh.unit[nu % kUnitRing];  // (kept in shared memory: registers are short)
    if (!u.valid) return;
    const int nt = u.nt;
    const int lim0 = min(u.lim, u.nkl) - u.kb;
    const int lim = min(a.causal ? u.lim + pos : u.lim, u.nkl) - u.kb;
    float m = -INFINITY, l = 0.f, qm = 0.f;
    float acc[128];
#pragma unroll
    for (int c = 0; c < 128; ++c) acc[c] = 0.f;
    // acc += O of the last tile.
    auto fold = [&](uint32_t t) {
      if (!bar_wait_warp(&sh.o_full[t & 1], (t >> 1) & 1, ab)) return false;
      fence_after();
#pragma unroll
      for (int c = 0; c < 128; c += 32)
        if (c < a.dv) {
          uint32_t o[32];
          ld32(at + 256 + (t & 1) * 128 + c, o);
          wait_ld();
          pin32(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[c + i] += __uint_as_float(o[i]);
        }
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.o_empty[t & 1]);
      return true;
    };
    for (int j = 0; j < nt; ++j, ++n) {
      const uint32_t b = n & 1, ph = (n >> 1) & 1;
      if (!bar_wait_warp(&sh.s_full[b], ph, ab)) return;
      if (!bar_wait_warp(&sh.x_full[b], ph, ab)) return;
      fence_after();
      if (j == 0) qm = sh.q_mul[nq & 1][row >> 4] * sc;
      const uint32_t s_at = at + b * 128;
      const float* km = sh.k_mul[n & 3];
      const float* ve = sh.v_exp[n & 3];
      const float* vi = sh.v_inv[n & 3];
      const bool cut = lim0 < (j + 1) * kTileN;
      const int vis = lim - j * kTileN;
      float top = m;
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        uint32_t x[32];
        ld32(s_at + c, x);
        wait_ld();
        pin32(x);
        if (cut) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i >= vis) x[i] = 0xff800000u;
        }
#pragma unroll
        for (int g = 0; g < 32; g += 16) {
          float t0 = __uint_as_float(x[g]), t1 = __uint_as_float(x[g + 1]);
#pragma unroll
          for (int i = 2; i < 16; i += 2) {
            t0 = fmaxf(t0, __uint_as_float(x[g + i]));
            t1 = fmaxf(t1, __uint_as_float(x[g + i + 1]));
          }
          const float f = fmaxf(km[(c + g) >> 4] * qm, 1e-36f);
          top = fmaxf(top, fmaf(fmaxf(t0, t1), f, ve[(c + g) >> 4]));
        }
      }
      float alpha = 1.f;
      const bool grow = m == -INFINITY ? top > m : top - m > kLazy;
      if (__any_sync(0xffffffffu, grow)) {
        alpha = top == m ? 1.f : ex2(m - top);
        m = top;
        l *= alpha;
      }
      const float ref = (m == -INFINITY ? 0.f : m) - kLift;
      // A group of 16 keys at a time, the next one's scores on their way: P's
      // pieces take the group's own 16 columns.
      uint32_t x[2][16];
      ld16(s_at, x[0]);
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        wait_ld();
        pin16(x[g & 1]);
        if (g < 7) ld16(s_at + (g + 1) * 16, x[(g + 1) & 1]);
        const float f = fmaxf(km[g] * qm, 1e-36f), z = ve[g] - ref;
        uint32_t p[16];
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          float y0 = fmaf(__uint_as_float(x[g & 1][i]), f, z);
          float y1 = fmaf(__uint_as_float(x[g & 1][i + 1]), f, z);
          if (cut) {
            if (g * 16 + i >= vis) y0 = -INFINITY;
            if (g * 16 + i + 1 >= vis) y1 = -INFINITY;
          }
          const float p0 = ex2(y0), p1 = ex2(y1);
          l0 += p0;
          l1 += p1;
          const float h0 = __uint_as_float(__float_as_uint(p0) & 0xFFFFE000u);
          const float h1 = __uint_as_float(__float_as_uint(p1) & 0xFFFFE000u);
          p[i / 2] = Type16<__half>::pack(h0, h1);
          p[8 + i / 2] = Type16<__half>::pack(p0 - h0, p1 - h1);
        }
        l = fmaf(l0 + l1, vi[g], l);
        st16(s_at + g * 16, p);
      }
      wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.p_full[b]);
      if (j > 0) {
        if (!fold(n - 1)) return;
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
          for (int c = 0; c < 128; ++c) acc[c] *= alpha;
        }
      }
    }
    if (nt > 0) {
      ++nq;
      if (!fold(n - 1)) return;
    }
    if (pos < u.np0) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int64_t orow = (int64_t)u.q_row + pos;
      const int head = u.kvh * a.group + hd;
      const int64_t prow = ((int64_t)u.split * a.q_rows + orow) * a.heads + head;
      float* out = a.splits ? a.part + prow * a.dv
                            : (float*)a.out.p + orow * a.out.row + head * a.out.head;
      const bool patch = *(volatile int*)&sh.unit[nu % kUnitRing].patch != 0;
      if (patch) {
#pragma unroll
        for (int c = 0; c < 128; c += 4)
          if (c < a.dv)
#pragma unroll 1
            for (int k = u.edge * kTileN; k < lim; ++k) {
              const float* v = value_row<PAGED>(a, u, u.kb + k);
              if (!v) continue;
              const float4 z = load4(v + c);
              if (!finite_bits(z.x)) acc[c] += z.x;
              if (!finite_bits(z.y)) acc[c + 1] += z.y;
              if (!finite_bits(z.z)) acc[c + 2] += z.z;
              if (!finite_bits(z.w)) acc[c + 3] += z.w;
            }
      }
#pragma unroll
      for (int c = 0; c < 128; c += 4)
        if (c < a.dv)
          *reinterpret_cast<float4*>(out + c) =
              make_float4(acc[c] * inv, acc[c + 1] * inv, acc[c + 2] * inv, acc[c + 3] * inv);
      const float v = l == 0.f ? -INFINITY : fmaf(m - kLift, kLn2, logf(l));
      if (a.splits) a.part_lse[prow] = v;
      else if (a.lse) a.lse[orow * a.heads + head] = v;
    }
    __syncwarp();
    if (lane == 0) bar_arrive(&sh.u_empty[nu % kUnitRing]);
  }
}

template <int N>
__device__ __forceinline__ void more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// The launch holds 512 x 128 registers; the shares are 128 x 232 + 256 x 104 +
// 128 x 72 = those 65,536.
constexpr int kRegsRow = 232, kRegsConvert = 104, kRegsRest = 72;
static_assert(128 * kRegsRow + 256 * kRegsConvert + 128 * kRegsRest <= 512 * 128, "registers");

template <bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) attn_tc32_kernel(const __grid_constant__ TileArgs a) {
  extern __shared__ __align__(1024) unsigned char sm[];
  Shared& sh = *reinterpret_cast<Shared*>(sm + kTiles);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    bar_init(&sh.q_full, kConv);
    bar_init(&sh.q_empty, 1);
    bar_init(&sh.k_full, kConv);
    bar_init(&sh.k_empty, 1);
    bar_init(&sh.v_full, kConv);
    bar_init(&sh.v_empty, 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(&sh.s_full[i], 1);
      bar_init(&sh.p_full[i], 4);
      bar_init(&sh.o_full[i], 1);
      bar_init(&sh.o_empty[i], 4);
      bar_init(&sh.x_full[i], kConv);
    }
    for (int i = 0; i < kUnitRing; ++i) {
      bar_init(&sh.u_full[i], 1);
      bar_init(&sh.u_empty[i], 4 + kConv + 1);  // softmax, converting and product warps
    }
    bar_init(&sh.drain, 1);
    bar_init_fence();
    sh.abort = 0;
  }
  if (warp == 12) tmem_alloc(&sh.tmem, 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sh.tmem;
  if (warp < 4) {
    more_regs<kRegsRow>();
    row_role<PAGED>(a, sh, tmem, tid, lane);
  } else if (warp < 12) {
    fewer_regs<kRegsConvert>();
    convert_role<PAGED>(a, sh, sm, warp - 4, lane);
  } else {
    fewer_regs<kRegsRest>();
    if (warp == 12) {
      if (lane == 0) mma_role(a, sh, sm, tmem);
    } else if (warp == 13) {
      unit_role(a, sh, lane);
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (tid == 0 && sh.abort) attn_report(a.status, NYS_ATTN_GAVE_UP);
  if (warp == 12) {
    fence_after();
    tmem_free(tmem, 512);
  }
}

template <bool PAGED>
cudaError_t launch_t(const TileArgs& a, unsigned grid, cudaStream_t stream) {
  static const cudaError_t ready = cudaFuncSetAttribute(
      attn_tc32_kernel<PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (ready != cudaSuccess) return ready;
  attn_tc32_kernel<PAGED><<<grid, kThreads, kSmem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_tc32(const TileArgs& a, unsigned grid, cudaStream_t stream) {
  return a.pages ? launch_t<true>(a, grid, stream) : launch_t<false>(a, grid, stream);
}

}  // namespace nys
