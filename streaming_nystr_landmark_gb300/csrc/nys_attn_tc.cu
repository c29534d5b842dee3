// Exact attention on the tensor cores, bf16 and fp16.
//
// For each query row i (one position and head) over the keys j that it sees,
// in one pass:   s_ij = q_i . k_j,  m_i = running maximum,
//   P_ij = 2^{c (s_ij - m_i)},  c = scale log2(e),   l_i += sum_j P_ij,
//   O_i += sum_j P_ij v_j,   result O_i / l_i,   lse_i = scale m_i + ln l_i
// (fp16: P 2^7 times that, Type16::kLift).
// A tile of 128 keys is one step: S = Q K^T and O += P V are tcgen05 products
// with f32 accumulators in tensor memory.  Both maxima and sums are f32; P is
// rounded once to the inputs' type, which the second product needs (half a
// step relative, independent from key to key), while l sums the unrounded
// weights.
//
// Rows: the heads of a group are packed into the query tile, so one tile of
// 128 rows is 128 / group positions times the group's heads, and a key tile
// is read once for all of them.  A CTA runs two streams, each with its own S
// and O in tensor memory and its own warpgroup of softmax (thread = row): two
// query tiles over the same keys where there are two ("pair": while one
// stream's softmax runs, the other's products do), or one query tile whose
// even and odd key tiles the two streams take, joined at the end by their
// maxima.
//
// What bounds it: the products of long prompts (one of 16,384 tokens, 32 heads on
// 4 KV heads of 128: 1.45 ms, 1.52 PFLOP/s of the causal half's operations, 77% of
// the measured dense rate in a burst and 88% of the sustained one), where S = Q K^T,
// with A in shared memory, takes 107 clocks an instruction and P V, with A in
// tensor memory, 74.  Short prompts are bound by each unit's chain of loads,
// products and softmax (33 prompts of 1 to 2,047 tokens, 16 heads on 8: 67 us).  Two query tiles at once, one
// softmax hidden behind the other's products, is why a tile is 128 rows and not
// 256: tensor memory holds no third S.
//
// Warps: 0-3 and 4-7 softmax of the two streams, 8 TMA loads, 9 products,
// 10 finds the units of work, 11 cleans value tiles.  One persistent CTA a
// SM; every role runs ahead into the next unit as far as its buffers allow.
// Shared memory: two query tiles (64 KB) and a ring of five 32 KB slots that
// K and V tiles take in turn, all 128-byte swizzled as TMA writes them.
// Tensor memory: S0 S1 O0 O1, 128 columns each; P overwrites the first half of
// its S as it is formed.
//
// The maximum is followed lazily: O is rescaled only where a row's maximum
// grew by more than 8 powers of two (P then stays below 2^8), which after the
// first tiles is rare; l and O always share one reference, so the result is
// the same formula.
//
// Values that a row does not see must not reach it, even NaN: P is 0 there,
// but 0 x NaN is NaN.  In tiles where some row does not see some key (those at
// the diagonal and at a sequence's end) warp 11 replaces values that are not
// finite by 0 in shared memory, and if there were any the epilogue adds them
// to the rows that do see them.
//
// Every wait is bounded (2 s); one that runs out sets the status word and ends
// the CTA after its copies and products in flight.
#include <cmath>

#include "nys_attn_tc.h"

namespace nys {
namespace {

using namespace tc;

constexpr int kThreads = 384;
constexpr int kUnitRing = 2;  // units that a CTA has taken: the current one and the next
constexpr int kSlots = 5;
constexpr uint32_t kSlotBytes = 32768;
constexpr uint32_t kQBytes = 65536;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazy = 8.f;  // powers of two that a row may outgrow its reference by

struct Shared {
  uint64_t q_full, q_empty;
  uint64_t kv_full[kSlots], kv_empty[kSlots];
  uint64_t v_raw[kSlots];  // a value tile landed that is to be cleaned first
  // A barrier's phases have to be seen one by one by whoever waits on it, so O's
  // completion has a pair of barriers for units whose streams are read each by
  // its own warpgroup, and one for units that both read.
  uint64_t s_full[2], p_full[2], o_full[2], both_full[2], o_empty[2], ml_full[2];
  uint64_t u_full[kUnitRing], u_empty[kUnitRing];
  uint64_t drain;
  Unit unit[kUnitRing];
  float ml[2][kTileM][2];  // [stream][row] {m, l}
  uint32_t tmem;
  int abort;
};

constexpr uint32_t kSmem = kQBytes + kSlots * kSlotBytes + sizeof(Shared);
static_assert(kSmem <= 227 * 1024, "one CTA's shared memory");

// Position of K tile j and V tile j in the order in which a unit's tiles are
// loaded.  Pair: K0 V0 K1 V1 ..; one tile: K0 K1 V0 K2 V1 ..
__device__ __forceinline__ uint32_t k_at(int j, bool pair) {
  return pair ? 2 * j : (j < 2 ? j : 2 * j - 1);
}
__device__ __forceinline__ uint32_t v_at(int j, int nt, bool pair) {
  return pair ? 2 * j + 1 : min(2 * j + 2, 2 * nt - 1);
}

// Which tile has place e in the order that k_at and v_at give.
__device__ __forceinline__ void tile_at(int e, int nt, bool pair, bool& is_k, int& j) {
  if (pair) {
    is_k = !(e & 1);
    j = e >> 1;
  } else if (e < 2 && e < nt) {
    is_k = true;
    j = e;
  } else if (e == 2 * nt - 1) {
    is_k = false;
    j = nt - 1;
  } else {
    is_k = e & 1;
    j = is_k ? (e + 1) >> 1 : (e - 2) >> 1;
  }
}

// ---- TMA loads (one warp; one lane issues, and with pages every lane looks up
// a box of the next tile, so that no load waits for its page's number)
template <bool PAGED>
__device__ void load_role(const TileArgs& a, const CUtensorMap* mq, const CUtensorMap* mk,
                          const CUtensorMap* mv, Shared& sh, unsigned char* sm, int lane) {
  volatile int* ab = &sh.abort;
  uint32_t cnt = 0, nu = 0, nq = 0;
  uint32_t raw_phase = 0, raw_last = 0;  // per slot: v_raw's phase; whether its last tile went there
  const int chunks_d = (a.d + 63) / 64, chunks_v = (a.dv + 63) / 64;
  const uint32_t q_tile = (uint32_t)(chunks_d * 128 * a.group * a.tp);
  // One 64-column block of a box, or all of them where the box is a full tile
  // (make_map's boxes).
  auto copy = [&](unsigned char* dst, const CUtensorMap* m, int dim, int rows, int y, int z,
                  uint64_t* bar) {
    const bool whole = dim % 64 == 0;
    const int n = whole && rows == kTileM ? 1 : (dim + 63) / 64;
    for (int c = 0; c < n; ++c)
      tma_load4(dst + c * 16384, m, whole ? 0 : c * 64, y, z, whole ? c : 0, bar);
  };
  const int boxes = PAGED ? kTileN / a.box : 1;
  const int none = PAGED ? (int)(a.n_pages * a.page) : 0;  // past the tensor's end: reads as zeros
  // The page of this lane's box of the tile at `key` and the box's place in it;
  // the number is not touched before the next tile's turn.
  int next_page = -1, next_in = 0;
  auto look = [&](int key) {
    key += lane * a.box;
    next_page = -1;
    next_in = -1;
    if (lane < boxes && key < a.k_rows) {
      const int pi = key / a.page;
      next_in = key - pi * a.page;
      next_page = a.pages[pi];
    }
  };
  // Its row: outside the prefix or the pool the one past the end.
  auto row_of = [&](int page, int in) {
    if (in < 0) return none;
    if (page >= 0 && page < a.n_pages) return page * a.page + in;
    attn_report(a.status, NYS_ATTN_BAD_PAGE);
    return none;
  };
  for (;; ++nu) {
    if (!bar_wait_warp(&sh.u_full[nu % kUnitRing], (nu / kUnitRing) & 1, ab)) break;
    const Unit u = sh.unit[nu % kUnitRing];
    __syncwarp();
    if (lane == 0) bar_arrive(&sh.u_empty[nu % kUnitRing]);
    if (!u.valid) break;
    if (u.nt == 0) continue;
    const bool pair = u.np1 > 0;
    if (!bar_wait_warp(&sh.q_empty, (nq & 1) ^ 1, ab)) break;
    ++nq;
    if (elect_one()) {
      bar_expect(&sh.q_full, q_tile * (pair ? 2 : 1));
      for (int s = 0; s <= (pair ? 1 : 0); ++s)
        copy(sm + s * 32768, mq, a.d, a.group * a.tp, u.kvh * a.group, u.q_row + s * a.tp, &sh.q_full);
    }
    if (a.stall == kStallCopies && blockIdx.x == 0) break;
    const int y = a.kv_y ? u.kvh : 0;
    if (PAGED) look(u.kb);
    bool ok = true;
    for (int e = 0; e < 2 * u.nt; ++e) {
      bool is_k;
      int j;
      tile_at(e, u.nt, pair, is_k, j);
      const int my_page = next_page, my_in = next_in;
      if (PAGED && e + 1 < 2 * u.nt) {
        bool k1;
        int j1;
        tile_at(e + 1, u.nt, pair, k1, j1);
        look(u.kb + j1 * kTileN);
      }
      const uint32_t slot = cnt % kSlots;
      ok = bar_wait_warp(&sh.kv_empty[slot], ((cnt / kSlots) & 1) ^ 1, ab);
      if (!ok) break;
      ++cnt;
      unsigned char* dst = sm + kQBytes + slot * kSlotBytes;
      const CUtensorMap* m = is_k ? mk : mv;
      const int chunks = is_k ? chunks_d : chunks_v;
      // Tiles to be cleaned land on v_raw; the cleaner then completes kv_full.
      const bool edge = !is_k && j >= u.edge;
      uint64_t* full = edge ? &sh.v_raw[slot] : &sh.kv_full[slot];
      raw_last = (raw_last & ~(1u << slot)) | ((uint32_t)edge << slot);
      raw_phase ^= (uint32_t)edge << slot;
      if (!PAGED) {
        if (elect_one()) {
          bar_expect(full, (uint32_t)chunks * 16384u);
          copy(dst, m, is_k ? a.d : a.dv, kTileN, y, u.k_row + u.kb + j * kTileN, full);
        }
      } else {
        const int my_row = row_of(my_page, my_in);
        if (elect_one()) bar_expect(full, (uint32_t)chunks * 16384u);
        __syncwarp();
        const int dim = is_k ? a.d : a.dv;
        const bool whole = dim % 64 == 0;
        const int each = whole && a.box == kTileM ? 1 : chunks;  // copies of a box
        for (int x0 = 0; x0 < boxes * each; x0 += 32) {
          const int x = x0 + lane, b = x / each, c = x - b * each;
          const int row = __shfl_sync(0xffffffffu, my_row, b & 31);
          if (x < boxes * each)
            tma_load4(dst + c * 16384 + b * a.box * 128, m, whole ? 0 : c * 64, y, row, whole ? c : 0,
                      full);
        }
      }
      __syncwarp();
    }
    if (!ok) break;
  }
  // Copies in flight land before the CTA may leave.
  if (*ab) {
    int never = 0;
    for (uint32_t c = cnt > kSlots ? cnt - kSlots : 0; c < cnt; ++c) {
      const uint32_t slot = c % kSlots;
      if ((raw_last >> slot) & 1) bar_wait(&sh.v_raw[slot], ((raw_phase >> slot) & 1) ^ 1, &never);
      else bar_wait(&sh.kv_full[slot], (c / kSlots) & 1, &never);
    }
    if (nq) bar_wait(&sh.q_full, (nq - 1) & 1, &never);
  }
}

// ---- products (one thread)
template <typename T>
__device__ void mma_role(const TileArgs& a, Shared& sh, unsigned char* sm, uint32_t tmem) {
  volatile int* ab = &sh.abort;
  const int ks = (a.d + 15) / 16;
  const int nv = (a.dv + 15) & ~15;
  const uint32_t id_s = idesc(kTileM, kTileN, Type16<T>::kBf16, false);
  const uint32_t id_o = idesc(kTileM, nv, Type16<T>::kBf16, true);
  const uint32_t q0 = sptr(sm), kv0 = sptr(sm + kQBytes);
  uint32_t base = 0, nu = 0, nq = 0;
  uint32_t n_p[2] = {0, 0}, n_o[2] = {0, 0};  // P tiles of each stream; units that used its O
  bool ok = true;
  for (; ok; ++nu) {
    if (!bar_wait(&sh.u_full[nu % kUnitRing], (nu / kUnitRing) & 1, ab)) break;
    const Unit u = sh.unit[nu % kUnitRing];
    bar_arrive(&sh.u_empty[nu % kUnitRing]);
    if (!u.valid || (a.stall == kStallProducts && blockIdx.x == 0)) break;
    const bool pair = u.np1 > 0;
    const int n_of[2] = {pair ? u.nt0 : (u.nt + 1) / 2, pair ? u.nt : u.nt / 2};
    if (u.nt > 0) {
      if (!bar_wait(&sh.q_full, nq & 1, ab)) break;
      ++nq;
    }
    // The i-th product S of stream s, with K in its slot.
    auto scores = [&](int s, int j) {
      const uint32_t at = base + k_at(j, pair), slot = at % kSlots;
      if (!bar_wait(&sh.kv_full[slot], (at / kSlots) & 1, ab)) return false;
      fence_after();
      const uint64_t q = desc128(q0 + (pair ? s : 0) * 32768, 16, 1024);
      const uint64_t k = desc128(kv0 + slot * kSlotBytes, 16, 1024);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < ks) {
          const uint64_t off = (i >> 2) * 1024 + (i & 3) * 2;
          mma_ss(tmem + s * 128, q + off, k + off, id_s, i > 0);
        }
      commit(&sh.s_full[s]);
      if (j == u.nt - 1 && (!pair || s == 1)) commit(&sh.q_empty);  // the unit's last
      return true;
    };
    auto values = [&](int s, int j, bool first) {
      const uint32_t at = base + v_at(j, u.nt, pair), slot = at % kSlots;
      if (!bar_wait(&sh.kv_full[slot], (at / kSlots) & 1, ab)) return false;
      if (!bar_wait(&sh.p_full[s], n_p[s] & 1, ab)) return false;
      ++n_p[s];
      if (first) {
        if (!bar_wait(&sh.o_empty[s], (n_o[s] & 1) ^ 1, ab)) return false;
        ++n_o[s];
      }
      fence_after();
      const uint64_t v = desc128(kv0 + slot * kSlotBytes, 16384, 1024);
#pragma unroll
      for (int i = 0; i < kTileN / 16; ++i)
        mma_ts(tmem + 256 + s * 128, tmem + s * 128 + i * 8, v + (uint64_t)(i * 128), id_o,
               !(first && i == 0));
      return true;
    };
    auto free_slot = [&](uint32_t at) { commit(&sh.kv_empty[(base + at) % kSlots]); };
    if (pair) {
      for (int j = -1; j < u.nt && ok; ++j) {
        for (int s = 0; s < 2 && ok; ++s) {
          if (j >= 0 && j < n_of[s]) {
            ok = values(s, j, j == 0);
            if (ok && j == n_of[s] - 1) commit(&sh.o_full[s]);
            if (ok && s == 1) free_slot(v_at(j, u.nt, true));
          }
          if (ok && j + 1 < n_of[s]) ok = scores(s, j + 1);
        }
        if (!ok) break;
        if (j + 1 < u.nt) free_slot(k_at(j + 1, true));
      }
    } else {
      for (int j = 0; j < u.nt && j < 2 && ok; ++j) {
        ok = scores(j, j);
        if (ok) free_slot(k_at(j, false));
      }
      for (int j = 0; j < u.nt && ok; ++j) {
        const int s = j & 1;
        ok = values(s, j, j < 2);
        if (!ok) break;
        free_slot(v_at(j, u.nt, false));
        if (j + 2 >= u.nt) commit(&sh.both_full[s]);
        if (j + 2 < u.nt) {
          ok = scores(s, j + 2);
          if (ok) free_slot(k_at(j + 2, false));
        }
      }
    }
    if (!ok) break;
    base += 2 * (uint32_t)u.nt;
  }
  // Every product and arrival in flight ends before the CTA may leave.
  int none = 0;
  commit(&sh.drain);
  bar_wait(&sh.drain, 0, &none);
}

// ---- units of work (one warp)
__device__ void unit_role(const TileArgs& a, Shared& sh, UnitSource& source, int lane) {
  volatile int* ab = &sh.abort;
  for (uint32_t nu = 0;; ++nu) {
    if (!bar_wait_warp(&sh.u_empty[nu % kUnitRing], ((nu / kUnitRing) & 1) ^ 1, ab)) return;
    Unit u;
    source.next(a, nu, lane, u);
    if (lane == 0) {
      sh.unit[nu % kUnitRing] = u;
      bar_arrive(&sh.u_full[nu % kUnitRing]);
    }
    __syncwarp();
    if (!u.valid) return;
  }
}

// ---- value tiles in which some row does not see some key (one warp)
template <typename T>
__device__ void clean_role(const TileArgs& a, Shared& sh, unsigned char* sm, int lane) {
  volatile int* ab = &sh.abort;
  uint32_t base = 0, phase = 0;
  const int chunks = (a.dv + 63) / 64;
  for (uint32_t nu = 0;; ++nu) {
    if (!bar_wait_warp(&sh.u_full[nu % kUnitRing], (nu / kUnitRing) & 1, ab)) return;
    const Unit u = sh.unit[nu % kUnitRing];
    if (!u.valid) return;
    const bool pair = u.np1 > 0;
    for (int j = u.edge; j < u.nt; ++j) {
      const uint32_t at = base + v_at(j, u.nt, pair), slot = at % kSlots;
      if (!bar_wait_warp(&sh.v_raw[slot], (phase >> slot) & 1, ab)) return;
      phase ^= 1u << slot;
      const int rows = u.nkl - u.kb - j * kTileN;  // keys of the sequence in this tile
      unsigned char* tile = sm + kQBytes + slot * kSlotBytes + lane * 16;
      // Usually all are finite: one operation for two values finds out.
      uint32_t m0 = 0, m1 = 0, m2 = 0, m3 = 0;
      for (int c = 0; c < chunks; ++c)
#pragma unroll 16
        for (int i = 0; i < 32; ++i) {
          const uint4 x = *reinterpret_cast<const uint4*>(tile + c * 16384 + i * 512);
          m0 = Type16<T>::max_abs(m0, x.x);
          m1 = Type16<T>::max_abs(m1, x.y);
          m2 = Type16<T>::max_abs(m2, x.z);
          m3 = Type16<T>::max_abs(m3, x.w);
        }
      const uint32_t found = not_finite<T>(m0) | not_finite<T>(m1) | not_finite<T>(m2) | not_finite<T>(m3);
      if (__any_sync(0xffffffffu, found != 0)) {
        uint32_t seen = 0;
#pragma unroll 1
        for (int i = 0; i < 32 * chunks; ++i) {  // a warp covers four rows of 128 bytes
          uint4* p = reinterpret_cast<uint4*>(tile + i * 512);
          uint4 x = *p;
          const uint32_t b0 = not_finite<T>(x.x), b1 = not_finite<T>(x.y);
          const uint32_t b2 = not_finite<T>(x.z), b3 = not_finite<T>(x.w);
          if (b0 | b1 | b2 | b3) {
            if ((i & 31) * 4 + (lane >> 3) < rows) seen = 1;
            auto keep = [](uint32_t w, uint32_t b) {
              return w & ~(((b >> 15) & 1u) * 0xFFFFu | (b >> 31) * 0xFFFF0000u);
            };
            x.x = keep(x.x, b0);
            x.y = keep(x.y, b1);
            x.z = keep(x.z, b2);
            x.w = keep(x.w, b3);
            *p = x;
          }
        }
        if (__any_sync(0xffffffffu, seen) && lane == 0)
          *(volatile int*)&sh.unit[nu % kUnitRing].patch = 1;
      }
      proxy_fence();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.kv_full[slot]);
    }
    base += 2 * (uint32_t)u.nt;
    __syncwarp();
    if (lane == 0) bar_arrive(&sh.u_empty[nu % kUnitRing]);
  }
}

// Row j of the values of KV head kvh of a unit's sequence; null where the page
// is not in the pool.
template <typename T, bool PAGED>
__device__ __forceinline__ const T* value_row(const TileArgs& a, const Unit& u, int j) {
  int64_t row = (int64_t)u.k_row + j;
  if (PAGED) {
    const int32_t pg = a.pages[j / a.page];
    if (pg < 0 || pg >= a.n_pages) return nullptr;
    row = (int64_t)pg * a.page + j % a.page;
  }
  return (const T*)a.v_raw + row * a.v_row + u.kvh * a.v_head;
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  using K = Type16<__nv_bfloat16>;
  *reinterpret_cast<uint4*>(p) = make_uint4(K::pack(x[0], x[1]), K::pack(x[2], x[3]),
                                            K::pack(x[4], x[5]), K::pack(x[6], x[7]));
}
__device__ __forceinline__ void store8(__half* p, const float* x) {
  using K = Type16<__half>;
  *reinterpret_cast<uint4*>(p) = make_uint4(K::pack(x[0], x[1]), K::pack(x[2], x[3]),
                                            K::pack(x[4], x[5]), K::pack(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// ---- softmax and results of stream s (one warpgroup, thread = row)
template <typename T, bool PAGED>
__device__ void row_role(const TileArgs& a, Shared& sh, uint32_t tmem, int s, int row, int lane) {
  volatile int* ab = &sh.abort;
  const float sc = a.scale * kLog2e;
  const int pos = row / a.group, hd = row - pos * a.group;
  const uint32_t lane_at = (uint32_t)(row & ~31) << 16;
  const uint32_t s_at = tmem + lane_at + s * 128, o_at = tmem + lane_at + 256;
  uint32_t n_s = 0, n_own = 0, n_both[2] = {0, 0}, n_merge = 0;
  for (uint32_t nu = 0;; ++nu) {
    if (!bar_wait_warp(&sh.u_full[nu % kUnitRing], (nu / kUnitRing) & 1, ab)) return;
    const Unit u = sh.unit[nu % kUnitRing];
    if (!u.valid) return;
    const bool pair = u.np1 > 0;
    const int first = pair ? 0 : s, step = pair ? 1 : 2;
    const int end = pair && s == 0 ? u.nt0 : u.nt;
    const int shift = pair ? s * a.tp : 0;  // positions before this stream's tile
    // Keys that this row sees, and that every row of the tile sees.
    const int lim0 = min(a.causal ? u.lim + shift : u.lim, u.nkl) - u.kb;
    const int lim = min(a.causal ? u.lim + shift + pos : u.lim, u.nkl) - u.kb;
    const bool mine = pos < (pair && s == 1 ? u.np1 : u.np0);
    float m = -INFINITY, l = 0.f;
    for (int j = first; j < end; j += step) {
      if (!bar_wait_warp(&sh.s_full[s], n_s & 1, ab)) return;
      ++n_s;
      fence_after();
      uint32_t x[128];
      ld32(s_at, x);
      ld32(s_at + 32, x + 32);
      ld32(s_at + 64, x + 64);
      ld32(s_at + 96, x + 96);
      wait_ld();
      pin32(x);
      pin32(x + 32);
      pin32(x + 64);
      pin32(x + 96);
      if (lim0 < (j + 1) * kTileN) {
        const int vis = lim - j * kTileN;
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= vis) x[c] = 0xff800000u;  // -inf
      }
      float t0 = -INFINITY, t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
#pragma unroll
      for (int c = 0; c < 128; c += 8) {
        t0 = max3(t0, __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
        t1 = max3(t1, __uint_as_float(x[c + 2]), __uint_as_float(x[c + 3]));
        t2 = max3(t2, __uint_as_float(x[c + 4]), __uint_as_float(x[c + 5]));
        t3 = max3(t3, __uint_as_float(x[c + 6]), __uint_as_float(x[c + 7]));
      }
      const float top = fmaxf(fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)), m);
      // (Rows that are not stored hold anything: they have no say in it.)
      const bool grow = mine && (m == -INFINITY ? top > m : (top - m) * sc > kLazy);
      if (__any_sync(0xffffffffu, grow)) {
        const float alpha = top == m ? 1.f : ex2((m - top) * sc);
        m = top;
        if (j != first) {
          // The stream's last O += P V is complete: S was issued after it.
          l *= alpha;
          const int nv = (a.dv + 15) & ~15;
          for (int c = 0; c < nv; c += 16) {
            uint32_t o[16];
            ld16(o_at + s * 128 + c, o);
            wait_ld();
            pin16(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            st16(o_at + s * 128 + c, o);
          }
          wait_st();
        }
      }
      const float ref = (m == -INFINITY ? 0.f : m * sc) - Type16<T>::kLift;
      float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float p0 = ex2(fmaf(__uint_as_float(x[c + i]), sc, -ref));
          const float p1 = ex2(fmaf(__uint_as_float(x[c + i + 1]), sc, -ref));
          const float p2 = ex2(fmaf(__uint_as_float(x[c + i + 2]), sc, -ref));
          const float p3 = ex2(fmaf(__uint_as_float(x[c + i + 3]), sc, -ref));
          l0 += p0;
          l1 += p1;
          l2 += p2;
          l3 += p3;
          p[i / 2] = Type16<T>::pack(p0, p1);
          p[i / 2 + 1] = Type16<T>::pack(p2, p3);
        }
        st16(s_at + c / 2, p);
      }
      l += (l0 + l1) + (l2 + l3);
      wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.p_full[s]);
    }

    // Results.  Pair: this stream's O alone.  One tile: both streams' O under
    // their common maximum, each warpgroup every other 16 columns.
    const int n0 = pair ? u.nt0 : (u.nt + 1) / 2, n1 = pair ? u.nt : u.nt / 2;
    const bool has0 = n0 > 0, has1 = n1 > 0;
    const bool use0 = has0 && (!pair || s == 0), use1 = has1 && (!pair || s == 1);
    if (pair) {
      if (use0 || use1) {
        if (!bar_wait_warp(&sh.o_full[s], n_own & 1, ab)) return;
        ++n_own;
      }
    } else {
      if (has0) {
        if (!bar_wait_warp(&sh.both_full[0], n_both[0] & 1, ab)) return;
        ++n_both[0];
      }
      if (has1) {
        if (!bar_wait_warp(&sh.both_full[1], n_both[1] & 1, ab)) return;
        ++n_both[1];
      }
    }
    float a0, a1, total, top = m;
    if (pair) {
      total = l;
      a0 = s == 0 ? 1.f : 0.f;
      a1 = 1.f - a0;
    } else {
      // A stream that had tiles writes its (m, l) only now, after its O is
      // complete: that O was begun after both warpgroups left the last unit,
      // so nobody still reads the last values.
      if (end > first) {
        sh.ml[s][row][0] = m;
        sh.ml[s][row][1] = l;
      }
      // (A unit without tiles is left out: nothing would hold one warpgroup back
      // from its next arrival until the other has seen this one.)
      if (has0) {
        __syncwarp();
        if (lane == 0) bar_arrive(&sh.ml_full[s]);
        if (!bar_wait_warp(&sh.ml_full[1 - s], n_merge & 1, ab)) return;
        ++n_merge;
      }
      const bool other = s == 0 ? has1 : has0;
      const float mo = other ? sh.ml[1 - s][row][0] : -INFINITY;
      const float lo = other ? sh.ml[1 - s][row][1] : 0.f;
      top = fmaxf(m, mo);
      const float r = top == -INFINITY ? 0.f : top;
      const float am = m == top ? 1.f : ex2((m - r) * sc), ao = mo == top ? 1.f : ex2((mo - r) * sc);
      total = s == 0 ? fmaf(l, am, lo * ao) : fmaf(lo, ao, l * am);
      a0 = s == 0 ? am : ao;
      a1 = s == 0 ? ao : am;
    }
    fence_after();
    const float inv = total == 0.f ? 0.f : reciprocal(total);
    a0 *= inv;
    a1 *= inv;
    const int64_t orow = (int64_t)u.q_row + shift + pos;
    const int head = u.kvh * a.group + hd;
    const bool patch = *(volatile int*)&sh.unit[nu % kUnitRing].patch != 0;
    const int64_t prow = ((int64_t)u.slot * a.per + (pair ? s : 0)) * kTileM + row;
    T* out = (T*)a.out.p + orow * a.out.row + head * a.out.head;
    for (int c = pair ? 0 : 16 * s; c < a.dv; c += pair ? 16 : 32) {
      float y[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = 0.f;
      if (use0) {
        uint32_t o[16];
        ld16(o_at + c, o);
        wait_ld();
        pin16(o);
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(o[i]) * a0;
      }
      if (use1) {
        uint32_t o[16];
        ld16(o_at + 128 + c, o);
        wait_ld();
        pin16(o);
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = fmaf(__uint_as_float(o[i]), a1, y[i]);
      }
      if (!mine) continue;
#pragma unroll
      for (int i = 0; i < 16; i += 8)
        if (c + i < a.dv) {
          if (u.slot >= 0) store8(a.part + prow * a.dv + c + i, y + i);
          else store8(out + c + i, y + i);
        }
    }
    if (patch && mine) {
      for (int k = u.edge * kTileN; k < lim; ++k) {
        const T* v = value_row<T, PAGED>(a, u, u.kb + k);
        if (!v) continue;
        for (int c = pair ? 0 : 16 * s; c < a.dv; c += pair ? 16 : 32) {
          if (u.slot >= 0) add_unusual(a.part + prow * a.dv, v, c, min(c + 16, a.dv));
          else add_unusual(out, v, c, min(c + 16, a.dv));
        }
      }
    }
    if (mine && (pair || s == 0)) {
      const float v = total == 0.f ? -INFINITY : fmaf(top, a.scale, (lg2(total) - Type16<T>::kLift) * 0.6931471805599453f);
      if (u.slot >= 0) a.part_lse[prow] = v;
      else if (a.lse) a.lse[orow * a.heads + head] = v;
    }
    fence_before();
    __syncwarp();
    if (lane == 0) {
      // Eight arrivals free an O that was used: four warps twice, or eight warps
      // once.  An O that was not gets none, so that its barrier never runs ahead
      // of the products' thread.
      if (pair) {
        if (s == 0 ? has0 : has1) bar_arrive(&sh.o_empty[s], 2);
      } else {
        if (has0) bar_arrive(&sh.o_empty[0]);
        if (has1) bar_arrive(&sh.o_empty[1]);
      }
      bar_arrive(&sh.u_empty[nu % kUnitRing]);
    }
  }
}

// The launch holds 384 x 168 registers = 64,512; the shares are 256 x 208 +
// 128 x 88 of them.
constexpr int kRegsRow = 208, kRegsRest = 88;
static_assert(256 * kRegsRow + 128 * kRegsRest <= 384 * 168, "registers");

template <typename T, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const __grid_constant__ TileArgs a, const __grid_constant__ CUtensorMap mq,
               const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  extern __shared__ __align__(1024) unsigned char sm[];  // the tiles, then Shared
  Shared& sh = *reinterpret_cast<Shared*>(sm + kQBytes + kSlots * kSlotBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    bar_init(&sh.q_full, 1);
    bar_init(&sh.q_empty, 1);
    for (int i = 0; i < kSlots; ++i) {
      bar_init(&sh.kv_full[i], 1);
      bar_init(&sh.kv_empty[i], 1);
      bar_init(&sh.v_raw[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&sh.s_full[i], 1);
      bar_init(&sh.p_full[i], 4);
      bar_init(&sh.o_full[i], 1);
      bar_init(&sh.both_full[i], 1);
      bar_init(&sh.o_empty[i], 8);
      bar_init(&sh.ml_full[i], 4);
    }
    for (int i = 0; i < kUnitRing; ++i) {
      bar_init(&sh.u_full[i], 1);
      bar_init(&sh.u_empty[i], 11);
    }
    bar_init(&sh.drain, 1);
    bar_init_fence();
    sh.abort = 0;
  }
  UnitSource source;
  if (warp == 8) {
    if (lane == 0) {
      prefetch_map(&mq);
      prefetch_map(&mk);
      prefetch_map(&mv);
    }
    __syncwarp();
    tmem_alloc(&sh.tmem, 512);
  } else if (warp == 10) {
    source.begin(a, lane);
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sh.tmem;
  let_next_start();
  if (warp < 8) {
    more_regs<kRegsRow>();
    row_role<T, PAGED>(a, sh, tmem, warp >> 2, tid & 127, lane);
  } else {
    fewer_regs<kRegsRest>();
    if (warp == 8) {
      load_role<PAGED>(a, &mq, &mk, &mv, sh, sm, lane);
    } else if (warp == 9) {
      if (elect_one()) mma_role<T>(a, sh, sm, tmem);
    } else if (warp == 10) {
      unit_role(a, sh, source, lane);
    } else {
      clean_role<T>(a, sh, sm, lane);
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (tid == 0 && sh.abort) attn_report(a.status, NYS_ATTN_GAVE_UP);
  if (warp == 8) {
    fence_after();
    tmem_free(tmem, 512);
  }
}

template <typename T, bool PAGED>
cudaError_t launch_t(const TileArgs& a, const TileMaps& m, unsigned grid, cudaStream_t stream) {
  const cudaError_t ready = ensure_smem<attn_tc_kernel<T, PAGED>>(kSmem);
  if (ready != cudaSuccess) return ready;
  attn_tc_kernel<T, PAGED><<<grid, kThreads, kSmem, stream>>>(a, m.q, m.k, m.v);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_tc(const TileArgs& a, const TileMaps& m, int dtype, unsigned grid,
                           cudaStream_t stream) {
  if (dtype == NYS_BF16)
    return a.pages ? launch_t<__nv_bfloat16, true>(a, m, grid, stream)
                   : launch_t<__nv_bfloat16, false>(a, m, grid, stream);
  return a.pages ? launch_t<__half, true>(a, m, grid, stream)
                 : launch_t<__half, false>(a, m, grid, stream);
}

}  // namespace nys
