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
// accumulators), 4-11 convert, 12 products, 13 units of work, 14 TMA loads.
// Registers move from the others to the softmax.  TMA brings f32 rows into a
// ring of three 32 KB stages (64 rows each); converting warps turn 16 rows each
// into the swizzled hi and lo tiles of K and V (32 KB a piece), and the query
// tile, thread = row, straight into tensor memory, because a product with A
// there takes 74 clocks and one with A in shared memory 107.  Products of tile
// j + 1's scores run during tile j's softmax, and K (V) is converted while the
// value (score) products run, so single buffers suffice.  Tensor memory: Q hi
// and lo (64 columns each), two S and one O of 128 columns; P hi and lo take S's
// place, 8 columns each for 16 keys.
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
constexpr int kStages = 3;
constexpr int kStageRows = 64;
constexpr uint32_t kStageBytes = kStageRows * 512;
constexpr uint32_t kOffV = 2 * kPiece, kOffStage = 4 * kPiece;
constexpr uint32_t kTiles = kOffStage + kStages * kStageBytes;
constexpr uint32_t kColQ = 0, kColS = 128, kColO = 384;  // tensor memory
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.f;
constexpr float kLift = 6.f;
constexpr int kTop = 13;        // the largest value's power of two after scaling

struct Shared {
  uint64_t q_full, q_empty, k_full, k_empty, v_full, v_empty;
  uint64_t s_full[2], p_full[2], x_full[2], o_full, o_empty;
  uint64_t st_full[kStages], st_empty[kStages];
  uint64_t u_full[kUnitRing], u_empty[kUnitRing];
  uint64_t drain;
  Unit unit[kUnitRing];
  float q_mul[2][kTileM];            // 2^eq, [unit & 1][row]
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

__device__ __forceinline__ bool finite_bits(float x) {
  return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
}

// ---- TMA loads (one thread): every tile as two stages of 64 rows.  A stage
// past the sequence's end is passed on empty.
template <bool PAGED>
__device__ void load_role(const TileArgs& a, const CUtensorMap* mk, const CUtensorMap* mv,
                          Shared& sh, unsigned char* sm) {
  volatile int* ab = &sh.abort;
  uint32_t cnt = 0, filled = 0;
  bool ok = true;
  for (uint32_t nu = 0; ok; ++nu) {
    if (!bar_wait(&sh.u_full[nu % kUnitRing], (nu / kUnitRing) & 1, ab)) break;
    const Unit u = sh.unit[nu % kUnitRing];
    bar_arrive(&sh.u_empty[nu % kUnitRing]);
    if (!u.valid) break;
    const int y = a.kv_y ? u.kvh : 0;
    for (int e = 1; e <= 2 * u.nt && ok; ++e) {
      int what, j;
      job_of(e, u.nt, what, j);
      const CUtensorMap* m = what == kJobK ? mk : mv;
      for (int h = 0; h < 2; ++h) {
        const uint32_t slot = cnt % kStages;
        ok = bar_wait(&sh.st_empty[slot], ((cnt / kStages) & 1) ^ 1, ab);
        if (!ok) break;
        ++cnt;
        const int key = u.kb + j * kTileN + h * kStageRows;
        if (key >= u.nkl) {
          filled &= ~(1u << slot);
          bar_arrive(&sh.st_full[slot]);
          continue;
        }
        filled |= 1u << slot;
        unsigned char* dst = sm + kOffStage + slot * kStageBytes;
        bar_expect(&sh.st_full[slot], kStageBytes);
        if (!PAGED) {
          tma_load3(dst, m, 0, y, u.k_row + key, &sh.st_full[slot]);
        } else {
          for (int b = 0; b < kStageRows; b += a.box) {
            // Past the prefix or outside the pool: a row past the tensor's
            // end, which reads as zeros.
            int64_t row = a.n_pages * a.page;
            if (key + b < u.nkl) {
              const int32_t pg = a.pages[(key + b) / a.page];
              if (pg >= 0 && pg < a.n_pages) row = (int64_t)pg * a.page + (key + b) % a.page;
              else attn_report(a.status, NYS_ATTN_BAD_PAGE);
            }
            tma_load3(dst + b * 512, m, 0, y, (int)row, &sh.st_full[slot]);
          }
        }
      }
    }
  }
  // Copies in flight land before the CTA may leave.
  if (*ab) {
    int none = 0;
    for (uint32_t c = cnt > kStages ? cnt - kStages : 0; c < cnt; ++c)
      if ((filled >> (c % kStages)) & 1)
        bar_wait(&sh.st_full[c % kStages], (c / kStages) & 1, &none);
  }
}

// ---- conversion (eight warps)
// The power of two that puts a value with these upper bits at 2^13, and back.
__device__ __forceinline__ int top_exponent(uint32_t top) {
  const int ex = (int)(top >> 23);         // biased
  return ex == 0 ? 127 : (ex < 40 ? 40 : ex);  // all zero: any scale
}
__device__ __forceinline__ float scale_of(int ex) {  // 2^(13 - (ex - 127))
  return __uint_as_float((uint32_t)(254 + kTop - ex) << 23);
}
__device__ __forceinline__ float back_of(int ex) {
  return __uint_as_float((uint32_t)(ex - kTop) << 23);
}
// Four scaled values as hi and lo words.  keep: infinities and NaN stay what
// they are, alone in hi.
__device__ __forceinline__ void split4(float4 x, uint64_t scale2, bool keep, uint32_t (&hi)[2],
                                       uint32_t (&lo)[2]) {
  const uint64_t ya = mul2(pair(x.x, x.y), scale2), yb = mul2(pair(x.z, x.w), scale2);
  const uint64_t minus2 = pair(-1.f, -1.f);
  float y[4], h[4], l[4];
  unpair(ya, y[0], y[1]);
  unpair(yb, y[2], y[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = cut11(y[i]);
  unpair(fma2(pair(h[0], h[1]), minus2, ya), l[0], l[1]);
  unpair(fma2(pair(h[2], h[3]), minus2, yb), l[2], l[3]);
  if (keep) {
    const float z[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!finite_bits(z[i])) {
        h[i] = z[i];
        l[i] = 0.f;
      }
  }
  using H = Type16<__half>;
  hi[0] = H::pack(h[0], h[1]);
  hi[1] = H::pack(h[2], h[3]);
  lo[0] = H::pack(l[0], l[1]);
  lo[1] = H::pack(l[2], l[3]);
}
__device__ __forceinline__ float finite_max(float4 x) {
  float f = 0.f;
  if (finite_bits(x.x)) f = fmaxf(f, fabsf(x.x));
  if (finite_bits(x.y)) f = fmaxf(f, fabsf(x.y));
  if (finite_bits(x.z)) f = fmaxf(f, fabsf(x.z));
  if (finite_bits(x.w)) f = fmaxf(f, fabsf(x.w));
  return f;
}

// The query tile into tensor memory: thread = row of the warp's 32, columns
// 64 * half .. (the other half is read for the row's exponent alone).  Rows past
// the tile's positions stand for its last one.
__device__ __forceinline__ void convert_q(const TileArgs& a, const Unit& u, float* q_mul,
                                          uint32_t tmem, int warp, int lane, bool& waited,
                                          uint64_t* q_empty, uint32_t parity, volatile int* ab) {
  const int row = (warp & 3) * 32 + lane, half = warp >= 8;
  const int pos = row / a.group, hd = row - pos * a.group;
  const float* src = (const float*)a.q.p + (u.q_row + (int64_t)min(pos, u.np0 - 1)) * a.q.row +
                     (int64_t)(u.kvh * a.group + hd) * a.q.head;
  float4 x[16];
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = half * 64 + i * 4;
    x[i] = c < a.d ? __ldg(reinterpret_cast<const float4*>(src + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = (1 - half) * 64 + i * 4;
    if (c < a.d) {
      const float4 z = __ldg(reinterpret_cast<const float4*>(src + c));
      t = max3_abs_nan(t, z.x, z.y);
      t = max3_abs_nan(t, z.z, z.w);
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    t = max3_abs_nan(t, x[i].x, x[i].y);
    t = max3_abs_nan(t, x[i].z, x[i].w);
  }
  uint32_t top = __float_as_uint(t) & 0x7FFFFFFFu;
  const bool odd = __any_sync(0xffffffffu, top >= 0x7F800000u);
  if (odd && top >= 0x7F800000u) {
    float f = 0.f;
    for (int c = 0; c < a.d; c += 4) f = fmaxf(f, finite_max(*reinterpret_cast<const float4*>(src + c)));
    top = __float_as_uint(f);
  }
  const int ex = top_exponent(top);
  if (half == 0) q_mul[row] = back_of(ex);
  const float scale = scale_of(ex);
  const uint64_t scale2 = pair(scale, scale);
  waited = bar_wait_warp(q_empty, parity, ab);
  if (!waited) return;
  fence_after();
  const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kColQ + half * 32;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t h2[2], l2[2];
      split4(x[b * 8 + i], scale2, odd, h2, l2);
      hi[2 * i] = h2[0];
      hi[2 * i + 1] = h2[1];
      lo[2 * i] = l2[0];
      lo[2 * i + 1] = l2[1];
    }
    st16(at + b * 16, hi);
    st16(at + 64 + b * 16, lo);
  }
  wait_st();
  fence_before();
}

__device__ void convert_role(const TileArgs& a, Shared& sh, unsigned char* sm, uint32_t tmem,
                             int warp, int lane) {
  volatile int* ab = &sh.abort;
  const int cw = warp - 4, half = cw >> 2;
  const int r0 = cw * kConvRows;  // first row in the tile
  uint32_t tile0 = 0, n_q = 0, n_job = 0;
  // Where this lane's four columns lie in a row of a tile: 64-column block,
  // then 16-byte units exchanged by the row's low bits (128-byte swizzle).
  const uint32_t col_at = (uint32_t)(lane >> 4) * 16384u + (uint32_t)(lane & 1) * 8u +
                          (uint32_t)r0 * 128u;
  const uint32_t unit16 = ((uint32_t)(lane & 15) >> 1) << 4;
  const uint32_t stage_at = kOffStage + (uint32_t)(cw & 3) * kConvRows * 512u + (uint32_t)lane * 16u;
  for (uint32_t nu = 0;; ++nu) {
    if (!bar_wait_warp(&sh.u_full[nu % kUnitRing], (nu / kUnitRing) & 1, ab)) return;
    const Unit& u = sh.unit[nu % kUnitRing];  // (read in place: registers are short)
    if (!u.valid) return;
    const int nt = u.nt, keys = u.nkl - u.kb, edge = u.edge;
    if (nt > 0) {
      bool ok;
      convert_q(a, u, sh.q_mul[n_q & 1], tmem, warp, lane, ok, &sh.q_empty, (n_q & 1) ^ 1, ab);
      if (!ok) return;
      ++n_q;
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.q_full);
    }
    for (int e = 1; e <= 2 * nt; ++e, ++n_job) {
      int what, j;
      job_of(e, nt, what, j);
      const uint32_t tile = tile0 + (uint32_t)j;
      const uint32_t n_st = 2 * n_job + half, slot = n_st % kStages;
      if (!bar_wait_warp(&sh.st_full[slot], (n_st / kStages) & 1, ab)) return;
      float4 x[kConvRows];
      const unsigned char* from = sm + stage_at + slot * kStageBytes;
#pragma unroll
      for (int r = 0; r < kConvRows; ++r) x[r] = *reinterpret_cast<const float4*>(from + r * 512);
      const int rows = keys - j * kTileN - r0;  // of them, those in the sequence
      if (rows < kConvRows) {
#pragma unroll
        for (int r = 0; r < kConvRows; ++r)
          if (r >= rows) x[r] = make_float4(0.f, 0.f, 0.f, 0.f);
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
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.st_empty[slot]);
      bool odd = top >= 0x7F800000u;  // some value is not finite
      if (odd) {
        float f = 0.f;
#pragma unroll
        for (int r = 0; r < kConvRows; ++r) f = fmaxf(f, finite_max(x[r]));
        top = __reduce_max_sync(0xffffffffu, __float_as_uint(f));
        // Values that some row does not see: out, and added in the epilogue.
        if (what == kJobV && j >= edge) {
#pragma unroll
          for (int r = 0; r < kConvRows; ++r) {
            if (!finite_bits(x[r].x)) x[r].x = 0.f;
            if (!finite_bits(x[r].y)) x[r].y = 0.f;
            if (!finite_bits(x[r].z)) x[r].z = 0.f;
            if (!finite_bits(x[r].w)) x[r].w = 0.f;
          }
          if (lane == 0) *(volatile int*)&sh.unit[nu % kUnitRing].patch = 1;
          odd = false;
        }
      }
      const int ex = top_exponent(top);
      const float scale = scale_of(ex);
      if (lane == 0) {
        if (what == kJobK) {
          sh.k_mul[tile & 3][cw] = back_of(ex);
        } else {
          sh.v_exp[tile & 3][cw] = (float)(ex - 127 - kTop);
          sh.v_inv[tile & 3][cw] = scale;
          bar_arrive(&sh.x_full[tile & 1]);
        }
      }
      uint64_t* empty = what == kJobK ? &sh.k_empty : &sh.v_empty;
      if (!bar_wait_warp(empty, (tile & 1) ^ 1, ab)) return;
      unsigned char* t = sm + (what == kJobK ? 0u : kOffV) + col_at;
      const bool put = lane * 4 < (((what == kJobV ? a.dv : a.d) + 15) & ~15);
      const uint64_t scale2 = pair(scale, scale);
      auto store_row = [&](int r, bool keep) {
        uint32_t hi[2], lo[2];
        split4(x[r], scale2, keep, hi, lo);
        if (put) {
          unsigned char* to = t + r * 128 + (unit16 ^ (uint32_t)((r & 7) << 4));
          *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(to + kPiece) = make_uint2(lo[0], lo[1]);
        }
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
      if (lane == 0) bar_arrive(what == kJobK ? &sh.k_full : &sh.v_full);
    }
    tile0 += (uint32_t)nt;
    __syncwarp();
    if (lane == 0) bar_arrive(&sh.u_empty[nu % kUnitRing]);
  }
}

// ---- products (one thread)
__device__ void mma_role(const TileArgs& a, Shared& sh, unsigned char* sm, uint32_t tmem) {
  volatile int* ab = &sh.abort;
  const int ks = (a.d + 15) / 16;
  const int nv = (a.dv + 15) & ~15;
  const uint32_t id_s = idesc(kTileM, kTileN, false, false);
  const uint32_t id_o = idesc(kTileM, nv, false, true);
  // Descriptors of the hi tiles; the lo tiles lie kPiece further.
  const uint64_t k0 = desc128(sptr(sm), 16, 1024), v0 = desc128(sptr(sm + kOffV), 16384, 1024);
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
      const uint32_t d = tmem + kColS + (n_s & 1) * 128;
#pragma unroll 1
      for (int p = 0; p < 3; ++p) {  // lo hi, hi lo, hi hi
        const uint32_t q = tmem + kColQ + (p == 0 ? 64 : 0);
        const uint64_t k = k0 + (p == 1 ? kPiece >> 4 : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < ks)
            mma_ts(d, q + i * 8, k + (uint64_t)((i >> 2) * 1024 + (i & 3) * 2), id_s, p + i > 0);
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
           bar_wait(&sh.o_empty, (n_o & 1) ^ 1, ab);
      if (!ok) break;
      fence_after();
      const uint32_t w0 = tmem + kColS + b * 128, o = tmem + kColO;
#pragma unroll 1
      for (int p = 0; p < 3; ++p) {
        const uint64_t v = v0 + (p == 1 ? kPiece >> 4 : 0);
        const uint32_t w = w0 + (p == 0 ? 8 : 0);
#pragma unroll
        for (int i = 0; i < kTileN / 16; ++i)
          mma_ts(o, w + i * 16, v + (uint64_t)(i * 128), id_o, p + i > 0);
      }
      commit(&sh.v_empty);
      commit(&sh.o_full);
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
      if (!bar_wait_warp(&sh.o_full, t & 1, ab)) return false;
      fence_after();
#pragma unroll
      for (int c = 0; c < 128; c += 32)
        if (c < a.dv) {
          uint32_t o[32];
          ld32(at + kColO + c, o);
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
      if (lane == 0) bar_arrive(&sh.o_empty);
      return true;
    };
    for (int j = 0; j < nt; ++j, ++n) {
      const uint32_t b = n & 1, ph = (n >> 1) & 1;
      if (!bar_wait_warp(&sh.s_full[b], ph, ab)) return;
      if (!bar_wait_warp(&sh.x_full[b], ph, ab)) return;
      fence_after();
      if (j == 0) qm = sh.q_mul[nq & 1][row] * sc;
      const uint32_t s_at = at + kColS + b * 128;
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
// The launch holds 512 x 128 registers; the shares are 128 x 208 + 256 x 112 +
// 128 x 80 = those 65,536.
constexpr int kRegsRow = 208, kRegsConvert = 112, kRegsRest = 80;
static_assert(128 * kRegsRow + 256 * kRegsConvert + 128 * kRegsRest <= 512 * 128, "registers");

template <bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) 
attn_tc32_kernel(const __grid_constant__ TileArgs a, const __grid_constant__ CUtensorMap mk,
                 const __grid_constant__ CUtensorMap mv) {
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
      bar_init(&sh.x_full[i], kConv);
    }
    bar_init(&sh.o_full, 1);
    bar_init(&sh.o_empty, 4);
    for (int i = 0; i < kStages; ++i) {
      bar_init(&sh.st_full[i], 1);
      bar_init(&sh.st_empty[i], kConv / 2);
    }
    for (int i = 0; i < kUnitRing; ++i) {
      bar_init(&sh.u_full[i], 1);
      bar_init(&sh.u_empty[i], 4 + kConv + 2);  // softmax, converting, product, load warps
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
    convert_role(a, sh, sm, tmem, warp, lane);
  } else {
    fewer_regs<kRegsRest>();
    if (warp == 12) {
      if (elect_one()) mma_role(a, sh, sm, tmem);
    } else if (warp == 13) {
      unit_role(a, sh, lane);
    } else if (warp == 14) {
      if (elect_one()) load_role<PAGED>(a, &mk, &mv, sh, sm);
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
cudaError_t launch_t(const TileArgs& a, const TileMaps& m, unsigned grid, cudaStream_t stream) {
  static const cudaError_t ready = cudaFuncSetAttribute(
      attn_tc32_kernel<PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (ready != cudaSuccess) return ready;
  attn_tc32_kernel<PAGED><<<grid, kThreads, kSmem, stream>>>(a, m.k, m.v);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_tc32(const TileArgs& a, const TileMaps& m, unsigned grid,
                             cudaStream_t stream) {
  return a.pages ? launch_t<true>(a, m, grid, stream) : launch_t<false>(a, m, grid, stream);
}

}  // namespace nys
