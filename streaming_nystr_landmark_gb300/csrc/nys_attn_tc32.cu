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

// Where row r of a job's tile begins in its tensor, in units of 16 bytes.  Rows
// past the sequence stand for its last one: their scores are masked, their
// weights 0, their results not stored.  A page outside the pool: 0, and `bad`.
template <bool PAGED>
__device__ __forceinline__ uint32_t job_row(const TileArgs& a, const Unit& u, int what, int j,
                                            int r, bool& bad) {
  if (what == kJobQ) {
    const int pos = r / a.group, hd = r - pos * a.group;
    return (uint32_t)(((u.q_row + (int64_t)min(pos, u.np0 - 1)) * a.q.row +
                       (int64_t)(u.kvh * a.group + hd) * a.q.head) >> 2);
  }
  const int key = min(u.kb + j * kTileN + r, u.nkl - 1);
  int64_t row = (int64_t)u.k_row + key;
  if (PAGED) {
    const int32_t pg = a.pages[key / a.page];
    if (pg < 0 || pg >= a.n_pages) {
      attn_report(a.status, NYS_ATTN_BAD_PAGE);
      bad = true;
      return 0;
    }
    row = (int64_t)pg * a.page + key % a.page;
  }
  return (uint32_t)((what == kJobK ? row * a.k_row + u.kvh * a.k_head
                                   : row * a.v_row + u.kvh * a.v_head) >> 2);
}

__device__ __forceinline__ bool finite_bits(float x) {
  return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
}

// ---- conversion (eight warps; cw = 0 .. 7)
template <bool PAGED>
__device__ void convert_role(const TileArgs& a, Shared& sh, unsigned char* sm, int cw, int lane) {
  volatile int* ab = &sh.abort;
  uint32_t nu = 0, nq = 0, tile0 = 0, done_k = 0, done_v = 0;
  // The next job: unit u, step e.  Skips units without keys.
  int e = 0;
  uint32_t held = 0;  // the unit's place in the ring (it is read there: registers are short)
  int nt = 0;
  auto next_unit = [&]() {
    for (;;) {
      if (!bar_wait_warp(&sh.u_full[nu % kUnitRing], (nu / kUnitRing) & 1, ab)) return false;
      held = nu % kUnitRing;
      ++nu;
      if (!sh.unit[held].valid) return false;
      nt = sh.unit[held].nt;
      if (nt > 0) return true;
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.u_empty[held]);
    }
  };
  const bool kcol = lane * 4 < a.d, vcol = lane * 4 < a.dv;
  const int r0 = cw * kConvRows;
  float4 x[kConvRows];
  bool have = next_unit();
  if (!have) return;
  // Rows of the next job, its first column for this lane, and its bad rows.
  uint32_t off;
  const float4* src;
  uint32_t bad_rows = 0;
  auto aim = [&](int what, int j) {
    bool bad = false;
    off = job_row<PAGED>(a, sh.unit[held], what, j, r0 + (lane & (kConvRows - 1)), bad);
    bad_rows = PAGED ? __ballot_sync(0xffffffffu, bad) & 0xffffu : 0;
    const float* p = (const float*)(what == kJobQ ? a.q.p : what == kJobK ? a.k_raw : a.v_raw);
    src = reinterpret_cast<const float4*>(p) + ((what == kJobV ? vcol : kcol) ? lane : 0);
  };
  aim(kJobQ, 0);
#pragma unroll
  for (int r = 0; r < kConvRows; ++r) x[r] = __ldg(src + __shfl_sync(0xffffffffu, off, r));
  // Where this lane's four columns lie in a row of a tile: 64-column block,
  // then 16-byte units exchanged by the row's low bits (128-byte swizzle).
  const uint32_t col_at = (uint32_t)(lane >> 4) * 16384u + (uint32_t)(lane & 1) * 8u +
                          (uint32_t)r0 * 128u;
  const uint32_t unit16 = ((uint32_t)(lane & 15) >> 1) << 4;
  while (have) {
    int what, j;
    job_of(e, nt, what, j);
    const uint32_t tile = tile0 + (uint32_t)j;
    const bool edge = what == kJobV && j >= sh.unit[held].edge;
    const uint32_t cur_held = held, cur_nq = nq;
    const uint32_t cur_bad = bad_rows;
    // What comes after it.
    bool last = false;
    if (++e > 2 * nt) {
      last = true;
      tile0 += (uint32_t)nt;
      ++nq;
      e = 0;
      have = next_unit();
    }
    if (have) {  // (otherwise the last rows are read once more)
      int nwhat, nj;
      job_of(e, nt, nwhat, nj);
      aim(nwhat, nj);
    }
    const int cols = what == kJobV ? a.dv : a.d;
    if (cur_bad || ((cols & 15) && lane * 4 >= cols)) {  // zeros
#pragma unroll
      for (int r = 0; r < kConvRows; ++r)
        if (((cur_bad >> r) & 1) || lane * 4 >= cols) x[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }

    // The rows' common exponent.
    float t0 = 0.f, t1 = 0.f;
#pragma unroll
    for (int r = 0; r < kConvRows; ++r) {
      t0 = max3_abs_nan(t0, x[r].x, x[r].y);
      t1 = max3_abs_nan(t1, x[r].z, x[r].w);
    }
    uint32_t top = __reduce_max_sync(
        0xffffffffu, max(__float_as_uint(t0) & 0x7FFFFFFFu, __float_as_uint(t1) & 0x7FFFFFFFu));
    bool odd = top >= 0x7F800000u;  // some value is not finite
    if (odd) {
      float f = 0.f;
#pragma unroll
      for (int r = 0; r < kConvRows; ++r) {
        const float y[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (finite_bits(y[i])) f = fmaxf(f, fabsf(y[i]));
      }
      top = __reduce_max_sync(0xffffffffu, __float_as_uint(f));
      // Values that some row does not see: out, and added in the epilogue.
      if (edge) {
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
    const bool put = lane * 4 < ((cols + 15) & ~15);
    const uint64_t scale2 = pair(scale, scale), minus2 = pair(-1.f, -1.f);
    using H = Type16<__half>;
    auto store_row = [&](int r, bool keep) {
      float y[4];
      const uint64_t ya = mul2(pair(x[r].x, x[r].y), scale2), yb = mul2(pair(x[r].z, x[r].w), scale2);
      unpair(ya, y[0], y[1]);
      unpair(yb, y[2], y[3]);
      float h[4], l[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = cut11(y[i]);
      unpair(fma2(pair(h[0], h[1]), minus2, ya), l[0], l[1]);
      unpair(fma2(pair(h[2], h[3]), minus2, yb), l[2], l[3]);
      if (keep) {  // infinities and NaN stay what they are, alone in hi
        const float z[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!finite_bits(z[i])) {
            h[i] = z[i];
            l[i] = 0.f;
          }
      }
      if (put) {
        unsigned char* to = t + r * 128 + (unit16 ^ (uint32_t)((r & 7) << 4));
        *reinterpret_cast<uint2*>(to) = make_uint2(H::pack(h[0], h[1]), H::pack(h[2], h[3]));
        *reinterpret_cast<uint2*>(to + kPiece) = make_uint2(H::pack(l[0], l[1]), H::pack(l[2], l[3]));
      }
      // The next job's row takes these registers.
      x[r] = __ldg(src + __shfl_sync(0xffffffffu, off, r));
    };
    if (odd) {
#pragma unroll
      for (int r = 0; r < kConvRows; ++r) store_row(r, true);
    } else {
#pragma unroll
      for (int r = 0; r < kConvRows; ++r) store_row(r, false);
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
          for (int i = 0; i < 32; i += 2)
            unpair(add2(pair(acc[c + i], acc[c + i + 1]),
                        pair(__uint_as_float(o[i]), __uint_as_float(o[i + 1]))),
                   acc[c + i], acc[c + i + 1]);
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
      if (lim0 < (j + 1) * kTileN) {  // some row does not see some key: mask S in place
        const int vis = lim - j * kTileN;
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          uint32_t x[32];
          ld32(s_at + c, x);
          wait_ld();
          pin32(x);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i >= vis) x[i] = 0xff800000u;
          st32(s_at + c, x);
        }
        wait_st();
      }
      float top = m;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t x[32];
        ld32(s_at + c, x);
        wait_ld();
        pin32(x);
#pragma unroll
        for (int g = 0; g < 32; g += 16) {
          float t0 = max3(__uint_as_float(x[g]), __uint_as_float(x[g + 1]), __uint_as_float(x[g + 2]));
          float t1 = max3(__uint_as_float(x[g + 3]), __uint_as_float(x[g + 4]), __uint_as_float(x[g + 5]));
#pragma unroll
          for (int i = 6; i < 14; i += 4) {
            t0 = max3(t0, __uint_as_float(x[g + i]), __uint_as_float(x[g + i + 1]));
            t1 = max3(t1, __uint_as_float(x[g + i + 2]), __uint_as_float(x[g + i + 3]));
          }
          t0 = max3(t0, __uint_as_float(x[g + 14]), __uint_as_float(x[g + 15]));
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
      uint32_t xa[16], xb[16];
      auto weights = [&](uint32_t* x, int g) {
        const float f = fmaxf(km[g] * qm, 1e-36f), z = ve[g] - ref;
        uint32_t p[16];
        const uint64_t f2 = pair(f, f), z2 = pair(z, z), minus2 = pair(-1.f, -1.f);
        uint64_t sum = pair(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          float y0, y1, r0, r1;
          unpair(fma2(pair(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), f2, z2), y0, y1);
          const float p0 = ex2(y0), p1 = ex2(y1);
          const uint64_t w = pair(p0, p1);
          sum = add2(sum, w);
          const float h0 = cut11(p0), h1 = cut11(p1);
          unpair(fma2(pair(h0, h1), minus2, w), r0, r1);
          p[i / 2] = Type16<__half>::pack(h0, h1);
          p[8 + i / 2] = Type16<__half>::pack(r0, r1);
        }
        float l0, l1;
        unpair(sum, l0, l1);
        l = fmaf(l0 + l1, vi[g], l);
        st16(s_at + g * 16, p);
      };
      ld16(s_at, xa);
#pragma unroll 1
      for (int g = 0; g < 8; g += 2) {
        wait_ld();
        pin16(xa);
        ld16(s_at + g * 16 + 16, xb);
        weights(xa, g);
        wait_ld();
        pin16(xb);
        if (g < 6) ld16(s_at + g * 16 + 32, xa);
        weights(xb, g + 1);
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
              const float4 z = *reinterpret_cast<const float4*>(v + c);
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
// The launch holds 512 x 128 registers; the shares are 128 x 208 + 256 x 120 +
// 128 x 64 = those 65,536.
constexpr int kRegsRow = 208, kRegsConvert = 120, kRegsRest = 64;
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
      if (elect_one()) mma_role(a, sh, sm, tmem);
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
