// Exact attention on the tensor cores, f32.
//
// The formulas are those of nys_attn_tc.cu.  An f32 operand x is taken as a
// pair of fp16 pieces of x' = x 2^-e: hi = x' to 11 bits, lo = x' - hi rounded to
// 11 bits, so that x' = hi + lo to 2^-22; a product takes three tcgen05 products,
// lo hi + hi lo + hi hi (the dropped lo lo is below 2^-21 of |x y| at worst, about
// 2^-24 in the mean and of either sign), summed in f32 in tensor memory, small
// ones first.  The exponent e is common to 16 rows (those that one warp
// converts) and puts their largest value at 2^13.  fp16's smallest step is 2^-24, so
// 22 bits are kept down to 2^-15 of the largest, and 2^-38 of it below.  Groups and
// units with a wider range than that takes are computed in f32 (below).
//
//   S' = Q' K'^T gives s_ij = S' 2^(eq + ek) scale log2(e), one multiplier a
//   group of 16 keys.  The value's exponent goes into the weight:
//   P_ij = 2^15 2^(s_ij + ev_j - m_i), m_i the running maximum of s + ev, so that P V'
//   is the plain sum at scale 2^(15 - m_i); l_i += P_ij 2^-ev_j.
//   P is split into two pieces as the operands are; 2^15 is the most that fp16
//   takes, so that keys by the thousand far below the largest still count (they are
//   held down to 2^-40 of it, in 22 bits to 2^-18).  That takes the maximum itself: one
//   that was followed only after a growth by 2^8 cost 8 of those bits and saved nothing
//   here, where a new one rescales registers.  (Added to the exponent instead, the 15
//   would round it: error of 64 prompts of 256 3.0e-7 -> 3.5e-7.)
//
// The tensor cores cut sums towards zero, so O is taken out after each tile of
// 128 keys (24 sums) and added to f32 accumulators in registers; a long row
// gathers no drift.
//
// Two kernels.  split_kernel turns K and V into pieces once a call: a tile of 128
// keys of one KV head becomes the image that shared memory is to hold (hi, then
// lo, each 64-column blocks of 128-byte-swizzled rows; rows past the sequence
// zero), with its eight groups' exponents beside it.  Done inside the attention
// kernel instead, each query tile converting what it reads, the conversion took
// longer than the products (a tile of keys 6,400 clocks against 3,600).  It runs
// at the memory's rate: 64 prompts of 256 tokens, 8 KV heads of 128: 42 us, 134 MB
// read and as much written (76 MB of it during the kernel, the rest stays in L2).
//
// attn_tc32_kernel: one CTA of 512 threads a SM works on one query tile of 128
// rows (positions x heads of the group): warps 0-7 softmax and accumulation (two
// threads a row: each takes half the tile's keys for the weights and half the
// value columns for the sums), 8-11 the query tile's pieces and the results'
// stores, 12 products, 13 units of work, 14 copies.  The products bound it where
// prompts are long (2 prompts continued over 5,003 tokens: 224 us, tensor pipe 80%
// busy), each unit's chain of steps where they are short (64 prompts of 256: 163 us
// with the split).  Q goes straight into tensor memory, because a
// product with A there takes 74 clocks and one with A in shared memory 107; K and
// V images stream through three 64 KB slots as plain bulk copies.  Scores of
// tile j + 1 run during tile j's softmax.  Tensor memory: Q hi and lo (64 columns
// each), two S and one O of 128 columns; P hi and lo take S's place, 8 columns
// each for 16 keys.
//
// Keys and values that are not finite are 0 in the images, and their group is flagged
// (odd), as are groups whose numbers are too far apart for a common exponent: units
// that read a flagged tile, and warps with such a query row, leave their results to the
// query warps, which compute them in f32 from the tensors (exact_rows).  So a key
// that a row does not see costs the row no more than roundings at f32's level, and one
// that it sees none but its own.  (A product of pieces with an infinity has the sign
// of either piece: lo x inf + hi x inf would be NaN for a key of weight 0.)
//
// Every wait is bounded (2 s), as in nys_attn_tc.cu.
#include <cmath>

#include "nys_attn_tc.h"

namespace nys {
namespace {

using namespace tc;

constexpr int kThreads = 512;
constexpr int kUnitRing = 3;  // units a CTA has taken: the last, the current and the next
constexpr int kLongUnit = 8;  // key tiles from which a unit is long
constexpr int kGroup = 16;      // keys of one exponent
constexpr int kGroups = kTileN / kGroup;
constexpr int kSlots = 3;
constexpr uint32_t kPiece = 32768;
constexpr uint32_t kSlotBytes = 2 * kPiece;
// The query warps move their 32 rows between global memory (whole sectors, 16
// columns of 8 rows an instruction) and "thread = row" through a buffer of 16
// columns each; 16-byte units are exchanged by the row so that neither side
// meets bank conflicts.
constexpr uint32_t kTurn = 32 * 64;
constexpr uint32_t kOffTurn = kSlots * kSlotBytes;
constexpr uint32_t kTiles = kOffTurn + 4 * kTurn;
__device__ __forceinline__ uint32_t turn_at(int row, int unit) {
  return (uint32_t)(row * 64 + ((unit ^ ((row >> 1) & 3)) << 4));
}
constexpr uint32_t kColQ = 0, kColS = 128, kColO = 384;  // tensor memory
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kLift = 15;
constexpr int kTop = 13;        // the largest value's power of two after scaling
// A group of values that are all 0 has no exponent of its own.  It takes one that is
// below those of values above 2^-47, so that its keys do not raise the reference above
// other keys' weights, and high enough that their weights, which l still counts, stay
// f32 numbers beside values up to 2^43; units with values outside that are flagged.
constexpr int kZeroExp = -60, kZeroLow = kZeroExp, kZeroHigh = 30;
// What a group of values says to its units: 0, all are 0; kOdd, computed in f32; else
// the biased exponent of the largest.
constexpr uint32_t kOdd = 255;
// fp16 holds a piece lo of a number at 2^-38 of its group's largest at best, so a key
// beside a far larger one, and a column beside a far larger one, would be rounded to what
// the larger one leaves.  A group is odd where rows, columns or most numbers lie that
// far below its largest, kSpan powers of two (is_odd); single numbers do in any group,
// and in some the half of them, and do no harm among others of their row and column.
// (Without that, one value row or column 2^10 above the rest leaves the other columns
// where they were, 2^12 five times, 2^14 forty times, 2^16 a hundred times further off.
// Keys and queries are a sum's operands: 2^18 there leaves results where they were.)
// Weights are rounded at 2^-40 of the largest contribution (weight and value), so a unit
// is odd where its groups' largest values are more than kSpanUnit apart and f32's last
// bits would go.  Products of exponents stay below f32's range.
constexpr int kSpanV = 13, kSpanMostV = 16, kSpanK = 17, kSpanUnit = 16;
constexpr int kLeastK = 40, kMostK = 187, kLeastV = 60;  // biased exponents

struct Shared {
  uint64_t q_full, q_empty;
  uint64_t kv_full[kSlots], kv_empty[kSlots];
  uint64_t s_full[2], p_full[2], o_full, o_empty, r_full;  // r: O holds the results
  uint64_t mx_full[4];               // both halves of a quarter's rows have their maxima
  uint64_t u_full[kUnitRing], u_empty[kUnitRing], patch_full[kUnitRing];
  uint64_t drain;
  Unit unit[kUnitRing];
  int patch[kUnitRing];  // results are computed in f32 by the query warps (exact_rows)
  alignas(16) TileExps exps[4];      // of tile & 3
  int8_t q_exp[4][kTileM];           // eq, [unit & 3][row]: the query warps run up to three units ahead
  float mx[2][2][kTileM];            // halves' maxima [exchange & 1][half][row], also of l
  uint32_t tmem;
  Beats beats;
};
constexpr uint32_t kSmem = kTiles + sizeof(Shared);
static_assert(kSmem <= 227 * 1024, "one CTA's shared memory");

// Place of K tile j and V tile j in the order in which a unit's tiles are
// copied: K0 K1 V0 K2 V1 ..
__device__ __forceinline__ uint32_t k_at(int j) { return j < 2 ? j : 2 * j - 1; }
__device__ __forceinline__ uint32_t v_at(int j, int nt) { return min(2 * j + 2, 2 * nt - 1); }

__device__ __forceinline__ float4 shared_load4(uint32_t at) {
  float4 x;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(at));
  return x;
}
__device__ __forceinline__ void shared_store4(uint32_t at, float4 x) {
  asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(at), "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w)
               : "memory");
}
__device__ __forceinline__ bool finite_bits(float x) {
  return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
}

// ---- copies (one thread)
__device__ void load_role(const TileArgs& a, Shared& sh, unsigned char* sm) {
  volatile Beats* ab = &sh.beats;
  uint32_t cnt = 0, tile = 0;
  const uint32_t kb = (uint32_t)((a.d + 63) / 64) * 16384u, vb = (uint32_t)((a.dv + 63) / 64) * 16384u;
  bool ok = true;
  for (uint32_t nu = 0; ok; ++nu) {
    if (!bar_wait(&sh.u_full[nu % kUnitRing], (nu / kUnitRing) & 1, ab)) break;
    const int valid = sh.unit[nu % kUnitRing].valid, nt = sh.unit[nu % kUnitRing].nt;
    const int64_t im = (int64_t)sh.unit[nu % kUnitRing].tile * a.kv_heads + sh.unit[nu % kUnitRing].kvh;
    bar_arrive(&sh.u_empty[nu % kUnitRing]);
    if (!valid || (a.stall == kStallCopies && blockIdx.x == 0)) break;
    if (nu == 0) wait_for_previous();  // the images
    for (int e = 0; e < 2 * nt; ++e) {
      bool is_k;
      int j;
      if (e < 2 && e < nt) {
        is_k = true;
        j = e;
      } else if (e == 2 * nt - 1) {
        is_k = false;
        j = nt - 1;
      } else {
        is_k = e & 1;
        j = is_k ? (e + 1) >> 1 : (e - 2) >> 1;
      }
      const uint32_t slot = cnt % kSlots;
      ok = bar_wait(&sh.kv_empty[slot], ((cnt / kSlots) & 1) ^ 1, ab);
      if (!ok) break;
      ++cnt;
      const int64_t at = im + (int64_t)j * a.kv_heads;
      const uint32_t bytes = is_k ? kb : vb;
      const unsigned char* src = (is_k ? a.k_image : a.v_image) + at * 2 * bytes;
      unsigned char* dst = sm + slot * kSlotBytes;
      uint64_t* full = &sh.kv_full[slot];
      bar_expect(full, 2 * bytes + (is_k ? (uint32_t)sizeof(TileExps) : 0u));
      if (is_k) bulk_copy(&sh.exps[(tile + j) & 3], a.exps + at, (uint32_t)sizeof(TileExps), full);
      bulk_copy(dst, src, bytes, full);
      bulk_copy(dst + kPiece, src + bytes, bytes, full);
    }
    tile += (uint32_t)nt;
  }
  // Copies in flight land before the CTA may leave.
  if (ab->abort) {
    Beats none{};
    for (uint32_t c = cnt > kSlots ? cnt - kSlots : 0; c < cnt; ++c)
      bar_wait(&sh.kv_full[c % kSlots], (c / kSlots) & 1, &none);
  }
}

// ---- conversion
// The power of two that puts a value with these upper bits at 2^13, and back.
__device__ __forceinline__ int top_exponent(uint32_t top) {
  const int ex = (int)(top >> 23);         // biased
  return ex == 0 ? 127 : (ex < 40 ? 40 : ex);  // all zero: any scale
}
__device__ __forceinline__ float scale_of(int ex) {  // 2^(13 - (ex - 127))
  return __uint_as_float((uint32_t)(254 + kTop - ex) << 23);
}
__device__ __forceinline__ float exp_of(int e) {  // 2^e, -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
__device__ __forceinline__ float back_of(int ex) {
  return __uint_as_float((uint32_t)(ex - kTop) << 23);
}
// The largest magnitude of four columns, NaN if one is.
__device__ __forceinline__ float cell_of(float4 x) {
  return max3_abs_nan(max3_abs_nan(0.f, x.x, x.y), x.z, x.w);
}
// Magnitudes below this are small against a largest one of biased exponent ex; zeros,
// which any scale holds, are not.
__device__ __forceinline__ float small_below(int ex, int span) {
  return __uint_as_float(ex > span ? (uint32_t)(ex - span) << 23 : 0u);
}
__device__ __forceinline__ int is_small(float x, float below) { return x != 0.f && fabsf(x) < below; }
__device__ __forceinline__ int count_small(float4 x, float below) {
  return is_small(x.x, below) + is_small(x.y, below) + is_small(x.z, below) + is_small(x.w, below);
}
// From how many small ones of `numbers` on they are most.
__device__ __forceinline__ int most_of(int numbers) { return max(3, numbers / 8); }
// Four scaled values as hi and lo words; DROP: 0 for infinities and NaN, which
// else do not occur.
template <bool DROP>
__device__ __forceinline__ void split4(float4 x, uint64_t scale2, uint32_t (&hi)[2],
                                       uint32_t (&lo)[2]) {
  const uint64_t ya = mul2(pair(x.x, x.y), scale2), yb = mul2(pair(x.z, x.w), scale2);
  const uint64_t minus2 = pair(-1.f, -1.f);
  // hi is the value with about half a step of hi added, then cut (4/3 2^-12 of the
  // value is 0.33 to 0.67 steps): lo has either sign, so that the dropped lo lo
  // does not add up.  Against plain cutting the error of 64 prompts of 256 falls
  // from 4.6e-7 to 3.0e-7, for 1% of the time.
  const uint64_t half = pair(3.2552083e-4f, 3.2552083e-4f);
  float y[4], h[4], l[4];
  unpair(fma2(ya, half, ya), y[0], y[1]);
  unpair(fma2(yb, half, yb), y[2], y[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = cut11(y[i]);
  unpair(fma2(pair(h[0], h[1]), minus2, ya), l[0], l[1]);
  unpair(fma2(pair(h[2], h[3]), minus2, yb), l[2], l[3]);
  if (DROP) {
    const float z[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!finite_bits(z[i])) h[i] = l[i] = 0.f;
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

// Results of this warp's 32 rows of a unit in f32 throughout, from the tensors
// themselves: for units that hold what the fp16 pieces do not.  Every row reads the
// keys that it sees and no others.  Eight rows at a time, two keys a step, which come
// through shared memory (`turn`) and are asked for a step ahead: four lanes have a
// row, each a quarter of its columns.  Right for everything and fast for nothing: 64
// prompts of 256 with a flag each take 2.9 ms (162 us without), 4 of 4,096 49 ms (0.56
// ms).  Its beats tell the waiting warps that it goes on.  (A call: inlined, its code costs the
// tiles 1%, 64 prompts of 256 158.8 -> 160.5 us.)
template <bool PAGED>
__device__ __noinline__ void exact_rows(const TileArgs& a, const Unit& u, unsigned char* turn,
                                        int warp, int lane, volatile Beats* beats) {
  constexpr int kKeys = 2, kCols = 8;  // keys of a step; pieces of four columns of a lane
  static_assert(kTurn == kKeys * 2 * 512, "the keys and values of a step");
  const float sc = a.scale * kLog2e;
  const int d = a.d, dv = a.dv, page = a.page, kb = u.kb, c0 = (lane & 3) * 4;
  const int64_t k_step = a.k_row, v_step = a.v_row, first = u.k_row, n_pages = a.n_pages;
  const int32_t* pages = a.pages;
  const float* k_lane = (const float*)a.k_raw + u.kvh * a.k_head + lane * 4;
  const float* v_lane = (const float*)a.v_raw + u.kvh * a.v_head + lane * 4;
  const bool k_col = lane * 4 < d, v_col = lane * 4 < dv;
  const uint32_t mine = sptr(turn) + lane * 16;  // [key or value][512 bytes]
  const uint32_t quarter = sptr(turn) + (lane & 3) * 16;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  // Row of key j of the piece; -1 where its page is not in the pool.
  auto key_row = [&](int j) {
    j += kb;
    if (!PAGED) return first + j;
    const int32_t pg = pages[j / page];
    return pg < 0 || pg >= n_pages ? (int64_t)-1 : (int64_t)pg * page + j % page;
  };
#pragma unroll 1
  for (int r0 = warp * 32; r0 < warp * 32 + 32; r0 += 8) {
    if (r0 / a.group >= u.np0) return;
    const int row = r0 + (lane >> 2), pos = row / a.group, h = u.kvh * a.group + (row - pos * a.group);
    const bool here = pos < u.np0;
    const int lim = here ? min(a.causal ? u.lim + pos : u.lim, u.nkl) - kb : 0;
    const int most = __reduce_max_sync(0xffffffffu, lim);
    uint64_t q[2 * kCols], acc[2 * kCols];
    const float* src = (const float*)a.q.p + (u.q_row + (int64_t)pos) * a.q.row + h * a.q.head + c0;
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (here && c * 16 + c0 < d) x = __ldg(reinterpret_cast<const float4*>(src + c * 16));
      q[2 * c] = pair(x.x * sc, x.y * sc);
      q[2 * c + 1] = pair(x.z * sc, x.w * sc);
      acc[2 * c] = acc[2 * c + 1] = pair(0.f, 0.f);
    }
    float m = -INFINITY, l = 0.f;
    float4 kx[kKeys], vx[kKeys];
    auto ask = [&](int k0) {
#pragma unroll
      for (int j = 0; j < kKeys; ++j) {
        const int64_t o = k0 + j < most ? key_row(k0 + j) : -1;
        kx[j] = o >= 0 && k_col ? __ldg(reinterpret_cast<const float4*>(k_lane + o * k_step)) : zero;
        vx[j] = o >= 0 && v_col ? __ldg(reinterpret_cast<const float4*>(v_lane + o * v_step)) : zero;
      }
    };
    ask(0);
#pragma unroll 1
    for (int k0 = 0; k0 < most; k0 += kKeys) {
      if (lane == 0 && !(k0 & 2047)) beats->beat = now_ns();
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kKeys; ++j) {
        shared_store4(mine + j * 512, kx[j]);
        shared_store4(mine + (kKeys + j) * 512, vx[j]);
      }
      __syncwarp();
      ask(k0 + kKeys);
      uint64_t sum[kKeys];
#pragma unroll
      for (int j = 0; j < kKeys; ++j) sum[j] = pair(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < kCols; c += 2) {
        float4 x[2 * kKeys];
#pragma unroll
        for (int j = 0; j < 2 * kKeys; ++j) x[j] = shared_load4(quarter + (j >> 1) * 512 + (c + (j & 1)) * 64);
#pragma unroll
        for (int j = 0; j < 2 * kKeys; ++j) {
          sum[j >> 1] = fma2(q[2 * (c + (j & 1))], pair(x[j].x, x[j].y), sum[j >> 1]);
          sum[j >> 1] = fma2(q[2 * (c + (j & 1)) + 1], pair(x[j].z, x[j].w), sum[j >> 1]);
        }
      }
      float y[kKeys], top = m;
#pragma unroll
      for (int j = 0; j < kKeys; ++j) {
        float y0, y1;
        unpair(sum[j], y0, y1);
        y0 += y1;
        y0 += __shfl_xor_sync(0xffffffffu, y0, 1);
        y0 += __shfl_xor_sync(0xffffffffu, y0, 2);
        y[j] = k0 + j < lim ? y0 : -INFINITY;
        top = fmaxf(top, y[j]);
      }
      const float f = top == m ? 1.f : ex2(m - top);
      m = top;
      l *= f;
#pragma unroll
      for (int j = 0; j < kKeys; ++j) {
        y[j] = ex2(y[j] - (m == -INFINITY ? 0.f : m));
        l += y[j];
      }
      if (__any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
        for (int c = 0; c < 2 * kCols; ++c) acc[c] = mul2(acc[c], pair(f, f));
      }
#pragma unroll
      for (int j = 0; j < kKeys; ++j)
        if (k0 + j < lim) {  // (0 x NaN is NaN)
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {
            float4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = shared_load4(quarter + (kKeys + j) * 512 + (c + i) * 64);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              acc[2 * (c + i)] = fma2(pair(y[j], y[j]), pair(x[i].x, x[i].y), acc[2 * (c + i)]);
              acc[2 * (c + i) + 1] = fma2(pair(y[j], y[j]), pair(x[i].z, x[i].w), acc[2 * (c + i) + 1]);
            }
          }
        }
    }
    if (!here) continue;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t part_row = (int64_t)u.slot * kTileM + row, orow = u.q_row + (int64_t)pos;
    float* out = (u.slot >= 0 ? a.part + part_row * dv : (float*)a.out.p + orow * a.out.row + h * a.out.head) + c0;
#pragma unroll
    for (int c = 0; c < kCols; ++c)
      if (c * 16 + c0 < dv) {
        float4 y;
        unpair(acc[2 * c], y.x, y.y);
        unpair(acc[2 * c + 1], y.z, y.w);
        *reinterpret_cast<float4*>(out + c * 16) = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
      }
    const float lse = l == 0.f ? -INFINITY : fmaf(m, kLn2, logf(l));
    if ((lane & 3) == 0) {
      if (u.slot >= 0) a.part_lse[part_row] = lse;
      else if (a.lse) a.lse[orow * a.heads + h] = lse;
    }
  }
}

// The query tile into tensor memory, and the results out of it (four warps, 32
// rows each; towards global memory a lane has 16 bytes of rows lane / 4 + 8 i,
// towards tensor memory row `lane`).  Rows past the tile's positions stand for
// its last one; their results are not stored.  While one unit is worked on, the
// next one's query is fetched and the last one's results leave.
template <bool PAGED>
__device__ void query_role(const TileArgs& a, Shared& sh, unsigned char* turn, uint32_t tmem,
                           int warp, int lane) {
  volatile Beats* ab = &sh.beats;
  const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
  const int sub = lane & 3;  // 4 columns of a chunk of 16
  int pos[4], hd[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = warp * 32 + i * 8 + (lane >> 2);
    pos[i] = r / a.group;
    hd[i] = r - pos[i] * a.group;
  }
  uint32_t n_q = 0, n_r = 0;
  bool odd_now = false, odd_last = false;  // the warp's rows of this unit and the last

  // Results of unit nu.
  auto results = [&](uint32_t nu) {
    const uint32_t at = nu % kUnitRing;
    const Unit& u = sh.unit[at];
    if (!bar_wait_warp(&sh.patch_full[at], (nu / kUnitRing) & 1, ab)) return false;
    const int64_t part_row = (int64_t)u.slot * kTileM + warp * 32;
    if (u.nt > 0) {
      if (!bar_wait_warp(&sh.r_full, n_r & 1, ab)) return false;
      ++n_r;
      fence_after();
    }
    if (sh.patch[at] || odd_last) {  // (a unit with tiles: nobody reads its O, whose next use may begin)
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.o_empty, 2);
      exact_rows<PAGED>(a, u, turn, warp, lane, ab);
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.u_empty[at]);
      return true;
    }
    float* to[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int h = u.kvh * a.group + hd[i];
      to[i] = pos[i] >= u.np0 ? nullptr
              : u.slot >= 0   ? a.part + (part_row + i * 8 + (lane >> 2)) * a.dv + sub * 4
                              : (float*)a.out.p + (u.q_row + (int64_t)pos[i]) * a.out.row +
                                    h * a.out.head + sub * 4;
    }
#pragma unroll 1
    for (int c = 0; c < a.dv; c += 32) {
      uint32_t o[32];
      if (u.nt > 0) {
        ld32(lanes + kColO + c, o);
        wait_ld();
        pin32(o);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0;
      }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(turn + turn_at(lane, i)) =
              make_uint4(o[g * 16 + i * 4], o[g * 16 + i * 4 + 1], o[g * 16 + i * 4 + 2], o[g * 16 + i * 4 + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(turn + turn_at(i * 8 + (lane >> 2), sub));
          if (to[i] && c + g * 16 + sub * 4 < a.dv) *reinterpret_cast<float4*>(to[i] + c + g * 16) = v;
        }
      }
    }
    fence_before();
    __syncwarp();
    if (lane == 0) {
      if (u.nt > 0) bar_arrive(&sh.o_empty, 2);  // eight arrivals free O
      bar_arrive(&sh.u_empty[at]);
    }
    return true;
  };

  for (uint32_t nu = 0;; ++nu) {
    if (!bar_wait_warp(&sh.u_full[nu % kUnitRing], (nu / kUnitRing) & 1, ab)) return;
    const Unit& u = sh.unit[nu % kUnitRing];
    const bool valid = u.valid;
    odd_now = false;
    if (valid && u.nt > 0) {
      // The whole tile at once, 32 loads a lane.
      float4 x[32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* src = (const float*)a.q.p + (u.q_row + (int64_t)min(pos[i], u.np0 - 1)) * a.q.row +
                           (int64_t)(u.kvh * a.group + hd[i]) * a.q.head + sub * 4;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          x[c * 4 + i] = c * 16 + sub * 4 < a.d ? __ldg(reinterpret_cast<const float4*>(src + c * 16))
                                                : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      // The rows' exponents.
      bool odd = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float t = 0.f, least = INFINITY;  // (zeros count: the check itself is rare enough)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float4 y = x[c * 4 + i];
          t = max3_abs_nan(t, y.x, y.y);
          t = max3_abs_nan(t, y.z, y.w);
          least = min3_abs(least, y.x, y.y);
          least = min3_abs(least, y.z, y.w);
        }
        uint32_t top = __float_as_uint(t) & 0x7FFFFFFFu;
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = (int)(top >> 23);
        const float below = small_below(e, kSpanK);
        if (__any_sync(0xffffffffu, least < below)) {
          int small = 0;  // a row's columns are on four lanes
#pragma unroll
          for (int c = 0; c < 8; ++c) small += count_small(x[c * 4 + i], below);
          small += __shfl_xor_sync(0xffffffffu, small, 1);
          small += __shfl_xor_sync(0xffffffffu, small, 2);
          odd |= small >= most_of(a.d);
        }
        odd |= (top != 0 && e < kLeastK) || e > kMostK;  // (infinities, NaN too)
        // (127 marks a query with a value that is not finite, whatever S then holds)
        if (sub == 0) sh.q_exp[n_q & 3][warp * 32 + i * 8 + (lane >> 2)] =
            (int8_t)(top >= 0x7F800000u ? 127 : top_exponent(top) - 127 - kTop);
      }
      odd = __any_sync(0xffffffffu, odd);
      odd_now = odd;
      __syncwarp();
      const int qe = sh.q_exp[n_q & 3][warp * 32 + lane];
      const float scale = qe == 127 ? NAN : exp_of(-qe);
      const uint64_t scale2 = pair(scale, scale);
      if (!bar_wait_warp(&sh.q_empty, (n_q & 1) ^ 1, ab)) return;
      fence_after();
#pragma unroll
      for (int b = 0; b < 8; ++b) {  // 16 columns
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(turn + turn_at(i * 8 + (lane >> 2), sub)) = x[b * 4 + i];
        __syncwarp();
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(turn + turn_at(lane, i));
          uint32_t h2[2], l2[2];
          split4<false>(v, scale2, h2, l2);
          w[2 * i] = h2[0];
          w[2 * i + 1] = h2[1];
          w[8 + 2 * i] = l2[0];
          w[9 + 2 * i] = l2[1];
        }
        st8(lanes + kColQ + b * 8, w);
        st8(lanes + kColQ + 64 + b * 8, w + 8);
      }
      wait_st();
      fence_before();
      ++n_q;
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.q_full);
    }
    if (nu > 0 && !results(nu - 1)) return;
    if (!valid) return;
    odd_last = odd_now;
  }
}

// Whether rows, columns or most numbers of a group are small (a warp; x: four columns of
// each row, `columns` their largest).  A row is small where half of it is, four columns
// at a time, below `below`: of normal numbers four are once in 10^13, in a group with
// columns 2^10 above the rest once in 100.  In fewer rows than 16 a column may be small
// by chance.  Most: an eighth, below `far`; what the others miss, large numbers in every
// row and every column, and short and narrow groups.  Zeros let the first checks through
// to the counting, which leaves them out.
__device__ __forceinline__ bool is_odd(const float4 (&x)[kGroup], float4 columns, int rows, int dim,
                                       float below, float far, bool col) {
  float cell = INFINITY, number = INFINITY;
#pragma unroll
  for (int r = 0; r < kGroup; r += 2) cell = min3_abs(cell, cell_of(x[r]), cell_of(x[r + 1]));
#pragma unroll
  for (int r = 0; r < kGroup; ++r) {
    number = min3_abs(number, x[r].x, x[r].y);
    number = min3_abs(number, x[r].z, x[r].w);
  }
  bool odd = rows == kGroup && __any_sync(0xffffffffu, count_small(columns, below) > 0);
  if (__any_sync(0xffffffffu, col && cell < below)) {
    int small = 0;
#pragma unroll
    for (int r = 0; r < kGroup; ++r) small += is_small(cell_of(x[r]), below);
    odd |= (int)__reduce_add_sync(0xffffffffu, small) >= max(1, dim / 8);
  }
  if (__any_sync(0xffffffffu, col && number < far)) {
    int small = 0;
#pragma unroll
    for (int r = 0; r < kGroup; ++r) small += count_small(x[r], far);
    odd |= (int)__reduce_add_sync(0xffffffffu, small) >= most_of(max(min(rows, kGroup), 0) * dim);
  }
  return odd;
}

// K and V as tile images.  Grid: tiles x KV heads, K and V; a warp takes 16 rows.  Three
// CTAs a SM: with the two that 105 registers would leave 64 prompts of 256 take 1.8 us
// longer.
template <bool PAGED>
__global__ void __launch_bounds__(256, 3) split_kernel(const __grid_constant__ TileArgs a) {
  let_next_start();
  if (a.counter && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.counter = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool is_v = blockIdx.y != 0;
  const int64_t at = blockIdx.x;  // tile * kv_heads + KV head
  const int tile = (int)(at / a.kv_heads), kvh = (int)(at - (int64_t)tile * a.kv_heads);
  // The sequence whose tiles begin at or before this one (seq_tile ascends).
  int k0 = 0, nk = (int)a.k_rows, j = tile;
  if (a.k_off) {
    int lo = 0, hi = a.n;
    bool bad = false;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      int s0, sn;
      seq_range(a.k_off, mid, a.k_rows, s0, sn, bad);
      if (seq_tile(s0, mid) <= tile) lo = mid;
      else hi = mid;
    }
    seq_range(a.k_off, lo, a.k_rows, k0, nk, bad);
    j = tile - seq_tile(k0, lo);
  }
  const int key0 = j * kTileN;
  if (j < 0 || key0 >= nk) return;  // between two sequences' tiles
  const int dim = is_v ? a.dv : a.d;
  const int r0 = warp * kGroup, rows = min(kGroup, nk - key0 - r0);  // rows <= 0: zeros
  const bool col = lane * 4 < dim;
  const float* src = (const float*)(is_v ? a.v_raw : a.k_raw) + kvh * (is_v ? a.v_head : a.k_head) +
                     (col ? lane * 4 : 0);
  const int64_t stride = is_v ? a.v_row : a.k_row;
  int64_t row = -1;
  if (lane < rows) {
    const int key = key0 + r0 + lane;
    row = (int64_t)k0 + key;
    if (PAGED) {
      const int32_t pg = a.pages[key / a.page];
      row = -1;
      if (pg >= 0 && pg < a.n_pages) row = (int64_t)pg * a.page + key % a.page;
      else attn_report(a.status, NYS_ATTN_BAD_PAGE);
    }
  }
  float4 x[kGroup];
#pragma unroll
  for (int r = 0; r < kGroup; ++r) {
    const int64_t o = __shfl_sync(0xffffffffu, row, r);
    x[r] = o >= 0 && col ? __ldcs(reinterpret_cast<const float4*>(src + o * stride))
                         : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float column[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int r = 0; r < kGroup; r += 2) {
    column[0] = max3_abs_nan(column[0], x[r].x, x[r + 1].x);
    column[1] = max3_abs_nan(column[1], x[r].y, x[r + 1].y);
    column[2] = max3_abs_nan(column[2], x[r].z, x[r + 1].z);
    column[3] = max3_abs_nan(column[3], x[r].w, x[r + 1].w);
  }
  const float4 columns = make_float4(column[0], column[1], column[2], column[3]);
  uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(cell_of(columns)) & 0x7FFFFFFFu);
  const bool bad = top >= 0x7F800000u;
  bool odd = bad;
  if (bad) {
    float f = 0.f;
#pragma unroll
    for (int r = 0; r < kGroup; ++r) f = fmaxf(f, finite_max(x[r]));
    top = __reduce_max_sync(0xffffffffu, __float_as_uint(f));
  } else {
    const int e = (int)(top >> 23);
    odd = is_odd(x, columns, rows, dim, small_below(e, is_v ? kSpanV : kSpanK),
                 small_below(e, is_v ? kSpanMostV : kSpanK), col);
    odd |= is_v ? top != 0 && e < kLeastV : (top != 0 && e < kLeastK) || e > kMostK;
  }
  const int ex = top_exponent(top);
  if (lane == 0) {
    const bool none = top >> 23 == 0;
    if (is_v) a.exps[at].v_exp[warp] = none ? kZeroExp : ex - 127 - kTop;
    else a.exps[at].k_mul[warp] = back_of(ex);
    a.odd[(at * 2 + is_v) * kGroups + warp] = (uint8_t)(odd ? kOdd : is_v && !none ? (uint32_t)ex : 0u);
  }
  const float scale = scale_of(ex);
  const uint64_t scale2 = pair(scale, scale);
  const uint32_t piece = (uint32_t)((dim + 63) / 64) * 16384u;
  // This lane's four columns: 64-column block, then 16-byte units exchanged by
  // the row's low bits (128-byte swizzle).
  unsigned char* t = (is_v ? a.v_image : a.k_image) + at * 2 * piece + (uint32_t)(lane >> 4) * 16384u +
                     (uint32_t)(lane & 1) * 8u + (uint32_t)r0 * 128u;
  const uint32_t unit16 = ((uint32_t)(lane & 15) >> 1) << 4;
  if (lane * 4 >= ((dim + 15) & ~15)) return;
#pragma unroll
  for (int r = 0; r < kGroup; ++r) {
    uint32_t hi[2], lo[2];
    if (!bad) split4<false>(x[r], scale2, hi, lo);
    else split4<true>(x[r], scale2, hi, lo);
    unsigned char* to = t + r * 128 + (unit16 ^ (uint32_t)((r & 7) << 4));
    *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
    *reinterpret_cast<uint2*>(to + piece) = make_uint2(lo[0], lo[1]);
  }
}

// ---- products (one thread)
__device__ void mma_role(const TileArgs& a, Shared& sh, unsigned char* sm, uint32_t tmem) {
  volatile Beats* ab = &sh.beats;
  const int ks = (a.d + 15) / 16;
  const int nv = (a.dv + 15) & ~15;
  const uint32_t id_s = idesc(kTileM, kTileN, false, false);
  const uint32_t id_o = idesc(kTileM, nv, false, true);
  uint32_t nu = 0, nq = 0, base = 0, n_s = 0, n_o = 0;  // units, query tiles, score and value tiles
  bool ok = true;
  for (; ok; ++nu) {
    if (!bar_wait(&sh.u_full[nu % kUnitRing], (nu / kUnitRing) & 1, ab)) break;
    const int valid = sh.unit[nu % kUnitRing].valid, nt = sh.unit[nu % kUnitRing].nt;
    bar_arrive(&sh.u_empty[nu % kUnitRing]);
    if (!valid || (a.stall == kStallProducts && blockIdx.x == 0)) break;
    if (nt == 0) continue;
    if (!bar_wait(&sh.q_full, nq & 1, ab)) break;
    ++nq;
    auto scores = [&](int j) {
      const uint32_t at = base + k_at(j), slot = at % kSlots;
      if (!bar_wait(&sh.kv_full[slot], (at / kSlots) & 1, ab)) return false;
      fence_after();
      const uint32_t d = tmem + kColS + (n_s & 1) * 128;
      const uint64_t k0 = desc128(sptr(sm + slot * kSlotBytes), 16, 1024);
#pragma unroll 1
      for (int p = 0; p < 3; ++p) {  // lo hi, hi lo, hi hi
        const uint32_t q = tmem + kColQ + (p == 0 ? 64 : 0);
        const uint64_t k = k0 + (p == 1 ? kPiece >> 4 : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < ks)
            mma_ts(d, q + i * 8, k + (uint64_t)((i >> 2) * 1024 + (i & 3) * 2), id_s, p + i > 0);
      }
      commit(&sh.s_full[n_s & 1]);
      commit(&sh.kv_empty[slot]);
      if (j == nt - 1) commit(&sh.q_empty);
      ++n_s;
      return true;
    };
    ok = scores(0);
    if (ok && nt > 1) ok = scores(1);
    for (int j = 0; j < nt && ok; ++j) {
      const uint32_t b = n_o & 1, ph = (n_o >> 1) & 1;
      const uint32_t at = base + v_at(j, nt), slot = at % kSlots;
      ok = bar_wait(&sh.kv_full[slot], (at / kSlots) & 1, ab) && bar_wait(&sh.p_full[b], ph, ab) &&
           bar_wait(&sh.o_empty, (n_o & 1) ^ 1, ab);
      if (!ok) break;
      fence_after();
      const uint32_t w0 = tmem + kColS + b * 128, o = tmem + kColO;
      const uint64_t v0 = desc128(sptr(sm + slot * kSlotBytes), 16384, 1024);
#pragma unroll 1
      for (int p = 0; p < 3; ++p) {
        const uint64_t v = v0 + (p == 1 ? kPiece >> 4 : 0);
        const uint32_t w = w0 + (p == 0 ? 8 : 0);
#pragma unroll
        for (int i = 0; i < kTileN / 16; ++i)
          mma_ts(o, w + i * 16, v + (uint64_t)(i * 128), id_o, p + i > 0);
      }
      commit(&sh.o_full);
      commit(&sh.kv_empty[slot]);
      ++n_o;
      if (j + 2 < nt) ok = scores(j + 2);
    }
    base += 2 * (uint32_t)nt;
  }
  Beats none{};
  commit(&sh.drain);
  bar_wait(&sh.drain, 0, &none);
}

__device__ void unit_role(const TileArgs& a, Shared& sh, UnitSource& source, int lane) {
  volatile Beats* ab = &sh.beats;
  int last_nt = 0;
  for (uint32_t nu = 0;; ++nu) {
    if (!bar_wait_warp(&sh.u_empty[nu % kUnitRing], ((nu / kUnitRing) & 1) ^ 1, ab)) return;
    // Long units are taken one at a time, when the one before the last is done:
    // others may be free for them sooner (2 prompts continued, 320 units of 45
    // tiles: 272 us, 307 without).  Short ones two ahead, so that the next
    // query is on its way (64 prompts of 256: 150 us, 159 one ahead).
    if (last_nt >= kLongUnit && nu >= 2 &&
        !bar_wait_warp(&sh.u_empty[(nu - 2) % kUnitRing], ((nu - 2) / kUnitRing) & 1, ab))
      return;
    Unit u;
    source.next(a, nu, lane, u);
    if (lane == 0) {
      sh.unit[nu % kUnitRing] = u;
      bar_arrive(&sh.u_full[nu % kUnitRing]);
    }
    __syncwarp();
    if (!u.valid) {
      // (A launch without units does not end before the split, which the next launch
      // on this workspace would then overtake.)
      if (nu == 0) wait_for_previous();
      return;
    }
    last_nt = u.nt;
    // (The flags, and the counter from here on, are the split's.)
    if (nu == 0) wait_for_previous();
    // Is a tile flagged?  Nobody asks before the results, so nobody waits for the
    // answer's way from memory.
    uint32_t keys = 0, low = ~0u, high = 0, zero = 0;  // of values: four groups at a time
#pragma unroll 4
    for (int i = lane; i < u.nt; i += 32) {
      const uint4 x = reinterpret_cast<const uint4*>(a.odd)[(int64_t)(u.tile + i) * a.kv_heads + u.kvh];
      keys |= x.x | x.y;
      high = __vmaxu4(high, __vmaxu4(x.z, x.w));
      low = __vminu4(low, __vminu4(__vsub4(x.z, 0x01010101u), __vsub4(x.w, 0x01010101u)));  // (0: 255)
      zero |= __vcmpeq4(x.z, 0u) | __vcmpeq4(x.w, 0u);
    }
    auto most = [](uint32_t x) {  // of a word's bytes and the warp
      x = __vmaxu4(x, x >> 16);
      return __reduce_max_sync(0xffffffffu, max(x & 255u, x >> 8 & 255u));
    };
    const int top = (int)most(high), bottom = 256 - (int)most(~low);  // 256: all are zero
    const bool mixed = zero != 0 && bottom < 256 &&
                       (bottom - 127 - kTop < kZeroLow || top - 127 - kTop > kZeroHigh);
    const bool apart = bottom < 256 && top - bottom > kSpanUnit;
    const bool odd = __any_sync(0xffffffffu, keys != 0 || mixed) || apart || top == (int)kOdd;
    if (lane == 0) {
      sh.patch[nu % kUnitRing] = odd;
      bar_arrive(&sh.patch_full[nu % kUnitRing]);
    }
  }
}

// Log of a row's sum l 2^(m - kLift).  m and l each hold the values' exponents, one up
// and one down: whole powers of two meet m first, so that what is left has the size of the
// result and is rounded there.  (This is what pieces are joined by: error of 100 requests
// over a prefix of 8,000 8.7e-7 -> 5.4e-7.)
__device__ __forceinline__ float log_sum(float m, float l) {
  const uint32_t bits = __float_as_uint(l);
  const int e = (int)(bits >> 23) - 127;
  if (l == 0.f) return -INFINITY;
  if (!finite_bits(l)) return l;
  return ((m + (float)(e - kLift)) + lg2(__uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u))) * kLn2;
}

// ---- softmax and accumulation (two warpgroups, two threads a row:
// `half` takes keys 64 * half .. of each tile and value columns 64 * half ..)
__device__ void row_role(const TileArgs& a, Shared& sh, uint32_t tmem, int row, int half,
                         int lane) {
  volatile Beats* ab = &sh.beats;
  const float sc = a.scale * kLog2e;
  const int pos = row / a.group, hd = row - pos * a.group;
  const uint32_t at = tmem + ((uint32_t)(row & ~31) << 16);
  uint64_t* mx_full = &sh.mx_full[row >> 5];
  uint32_t n = 0, nq = 0, n_mx = 0;  // tiles, query tiles, exchanges
  // Both halves' values of this row, through shared memory.
  auto exchange = [&](float mine, float& other) {
    sh.mx[n_mx & 1][half][row] = mine;
    __syncwarp();
    if (lane == 0) bar_arrive(mx_full);
    if (!bar_wait_warp(mx_full, n_mx & 1, ab)) return false;
    other = sh.mx[n_mx & 1][1 - half][row];
    ++n_mx;
    return true;
  };
  for (uint32_t nu = 0;; ++nu) {
    if (!bar_wait_warp(&sh.u_full[nu % kUnitRing], (nu / kUnitRing) & 1, ab)) return;
    const Unit& u = sh.unit[nu % kUnitRing];  // (kept in shared memory: registers are short)
    if (!u.valid) return;
    const int nt = u.nt;
    const int lim0 = min(u.lim, u.nkl) - u.kb;
    const int lim = min(a.causal ? u.lim + pos : u.lim, u.nkl) - u.kb;
    float m = -INFINITY, l = 0.f, qm = 0.f;
    float acc[64];
#pragma unroll
    for (int c = 0; c < 64; ++c) acc[c] = 0.f;
    // acc += O of the last tile.
    auto fold = [&](uint32_t t, bool last) {
      if (!bar_wait_warp(&sh.o_full, t & 1, ab)) return false;
      fence_after();
#pragma unroll
      for (int c = 0; c < 64; c += 32)
        if (half * 64 + c < a.dv) {
          uint32_t o[32];
          ld32(at + kColO + half * 64 + c, o);
          wait_ld();
          pin32(o);
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            unpair(add2(pair(acc[c + i], acc[c + i + 1]),
                        pair(__uint_as_float(o[i]), __uint_as_float(o[i + 1]))),
                   acc[c + i], acc[c + i + 1]);
        }
      if (last) return true;  // (the results take O's place)
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.o_empty);
      return true;
    };
    for (int j = 0; j < nt; ++j, ++n) {
      const uint32_t b = n & 1, ph = (n >> 1) & 1;
      if (!bar_wait_warp(&sh.s_full[b], ph, ab)) return;
      fence_after();
      if (j == 0) qm = exp_of(sh.q_exp[nq & 3][row]) * sc;
      const uint32_t s_at = at + kColS + b * 128 + half * 64;
      const float* km = sh.exps[n & 3].k_mul + half * 4;
      const int32_t* ve = sh.exps[n & 3].v_exp + half * 4;
      const bool cut = lim0 < (j + 1) * kTileN;  // some row does not see some key
      const int vis = lim - j * kTileN - half * 64;
      float top = m;
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        uint32_t x[32];
        ld32(s_at + c, x);
        wait_ld();
        pin32(x);
        if (cut) {  // mask S in place
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i >= vis) x[i] = 0xff800000u;
          st32(s_at + c, x);
        }
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
          top = fmaxf(top, fmaf(fmaxf(t0, t1), f, (float)ve[(c + g) >> 4]));
        }
      }
      {
        float other;
        if (!exchange(top, other)) return;
        top = fmaxf(top, other);
      }
      float alpha = 1.f;
      if (top > m) {
        alpha = ex2(m - top);
        m = top;
        l *= alpha;
      }
      const float ref = m == -INFINITY ? 0.f : m;
      // A group of 16 keys at a time, the next one's scores on their way: P's
      // pieces take the group's own 16 columns.
      uint32_t xa[16], xb[16];
      auto weights = [&](uint32_t* x, int g) {
        const int ev = ve[g];
        const float f = fmaxf(km[g] * qm, 1e-36f), z = (float)ev - ref;
        uint32_t p[16];
        const uint64_t f2 = pair(f, f), z2 = pair(z, z), minus2 = pair(-1.f, -1.f);
        const uint64_t lift2 = pair((float)(1 << kLift), (float)(1 << kLift));
        uint64_t sum = pair(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          float y0, y1, r0, r1;
          unpair(fma2(pair(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), f2, z2), y0, y1);
          const uint64_t w = mul2(pair(ex2(y0), ex2(y1)), lift2);
          sum = add2(sum, w);
          float p0, p1;
          unpair(w, p0, p1);
          const float h0 = cut11(p0), h1 = cut11(p1);
          unpair(fma2(pair(h0, h1), minus2, w), r0, r1);
          p[i / 2] = Type16<__half>::pack(h0, h1);
          p[8 + i / 2] = Type16<__half>::pack(r0, r1);
        }
        float l0, l1;
        unpair(sum, l0, l1);
        l = fmaf(l0 + l1, exp_of(-ev), l);
        st16(s_at + g * 16, p);
      };
      if (cut) wait_st();
      ld16(s_at, xa);
#pragma unroll 1
      for (int g = 0; g < 4; g += 2) {
        wait_ld();
        pin16(xa);
        ld16(s_at + g * 16 + 16, xb);
        weights(xa, g);
        wait_ld();
        pin16(xb);
        if (g < 2) ld16(s_at + g * 16 + 32, xa);
        weights(xb, g + 1);
      }
      wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.p_full[b]);
      if (j > 0) {
        if (!fold(n - 1, false)) return;
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
          for (int c = 0; c < 64; ++c) acc[c] *= alpha;
        }
      }
    }
    // The log-sum, before r_full: where the query warps compute the row themselves they
    // put theirs in its place afterwards.
    auto write_lse = [&](float v) {
      if (half != 0 || pos >= u.np0) return;
      const int64_t orow = (int64_t)u.q_row + pos;
      if (u.slot >= 0) a.part_lse[(int64_t)u.slot * kTileM + row] = v;
      else if (a.lse) a.lse[orow * a.heads + u.kvh * a.group + hd] = v;
    };
    if (nt == 0) write_lse(-INFINITY);
    if (nt > 0) {
      ++nq;
      float other;
      if (!exchange(l, other)) return;
      l = half == 0 ? l + other : other + l;
      const float inv = l == 0.f ? 0.f : reciprocal(l);
      if (!fold(n - 1, true)) return;
      // Results to tensor memory, for the query warps to store.
#pragma unroll
      for (int c = 0; c < 64; c += 16)
        if (half * 64 + c < a.dv) {
          uint32_t o[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(acc[c + i] * inv);
          st16(at + kColO + half * 64 + c, o);
        }
      write_lse(log_sum(m, l));
      wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.r_full);
    }
    __syncwarp();
    if (lane == 0) bar_arrive(&sh.u_empty[nu % kUnitRing]);
  }
}

// The launch holds 512 x 128 registers = 65,536; the shares are 256 x 136 +
// 128 x 168 + 128 x 72 of them.
constexpr int kRegsRow = 136, kRegsQuery = 168, kRegsRest = 72;
static_assert(256 * kRegsRow + 128 * kRegsQuery + 128 * kRegsRest <= 512 * 128, "registers");

template <bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) 
attn_tc32_kernel(const __grid_constant__ TileArgs a) {
  extern __shared__ __align__(1024) unsigned char sm[];
  Shared& sh = *reinterpret_cast<Shared*>(sm + kTiles);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    bar_init(&sh.q_full, 4);
    bar_init(&sh.q_empty, 1);
    for (int i = 0; i < kSlots; ++i) {
      bar_init(&sh.kv_full[i], 1);
      bar_init(&sh.kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&sh.s_full[i], 1);
      bar_init(&sh.p_full[i], 8);
    }
    bar_init(&sh.o_full, 1);
    bar_init(&sh.o_empty, 8);
    bar_init(&sh.r_full, 8);
    for (int i = 0; i < 4; ++i) bar_init(&sh.mx_full[i], 2);
    for (int i = 0; i < kUnitRing; ++i) {
      bar_init(&sh.u_full[i], 1);
      bar_init(&sh.patch_full[i], 1);
      bar_init(&sh.u_empty[i], 8 + 4 + 2);  // softmax, query, product, copying warps
    }
    bar_init(&sh.drain, 1);
    bar_init_fence();
    sh.beats = Beats{};
  }
  UnitSource source;
  if (warp == 12) tmem_alloc(&sh.tmem, 512);
  else if (warp == 13) source.begin(a, lane);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sh.tmem;
  let_next_start();
  if (warp < 8) {
    more_regs<kRegsRow>();
    row_role(a, sh, tmem, tid & 127, warp >> 2, lane);
  } else if (warp < 12) {
    more_regs<kRegsQuery>();
    query_role<PAGED>(a, sh, sm + kOffTurn + (warp & 3) * kTurn, tmem, warp & 3, lane);
  } else {
    fewer_regs<kRegsRest>();
    if (warp == 12) {
      if (elect_one()) mma_role(a, sh, sm, tmem);
    } else if (warp == 13) {
      unit_role(a, sh, source, lane);
    } else if (warp == 14) {
      if (elect_one()) load_role(a, sh, sm);
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (tid == 0 && sh.beats.abort) attn_report(a.status, NYS_ATTN_GAVE_UP);
  if (warp == 12) {
    fence_after();
    tmem_free(tmem, 512);
  }
}

template <bool PAGED>
cudaError_t launch_t(const TileArgs& a, unsigned grid, cudaStream_t stream) {
  const cudaError_t ready = ensure_smem<attn_tc32_kernel<PAGED>>(kSmem);
  if (ready != cudaSuccess) return ready;
  const dim3 images((unsigned)(key_tiles(a.k_rows, a.k_off ? a.n : 1) * a.kv_heads), 2);
  split_kernel<PAGED><<<images, 256, 0, stream>>>(a);
  return launch_dependent(attn_tc32_kernel<PAGED>, grid, kThreads, kSmem, stream, a);
}

}  // namespace

cudaError_t launch_attn_tc32(const TileArgs& a, unsigned grid, cudaStream_t stream) {
  return a.pages ? launch_t<true>(a, grid, stream) : launch_t<false>(a, grid, stream);
}

}  // namespace nys
