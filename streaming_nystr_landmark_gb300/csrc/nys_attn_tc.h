// Shared parts of the tiled attention kernels: their launch arguments and the
// cutting of a batch into units of work.
#pragma once

#include "nys_attn.h"
#include "nys_device.h"
#include "nys_tc.h"

namespace nys {

constexpr int kTileM = 128;  // rows of a query tile: (position, head of the group) pairs
constexpr int kTileN = 128;  // keys of a tile

// How a prefix's key tiles are dealt out.  A unit (query tiles of one KV head)
// has nt tiles; the units' tiles, one after another, are cut into `ctas` equal
// shares, so that every CTA has the same work whatever the numbers; a unit's
// share with a CTA is a piece.
struct Shares {
  int32_t nt, ctas, units, rows;  // rows: requests of a unit
  int32_t tp;                     // of them in one query tile
  // Piece i of a unit lies in slot unit + cta_of(its first tile) + i: pieces and
  // CTAs ascend together, so no two pieces share a slot.
  __host__ __device__ int slots() const { return units + ctas; }
  // The CTA that has tile t of all.
  __host__ __device__ int cta_of(int64_t t) const {
    return (int)(((t + 1) * ctas - 1) / ((int64_t)units * nt));
  }
  __host__ __device__ int64_t begin(int cta) const {
    return (int64_t)cta * units * nt / ctas;
  }
  __host__ __device__ int pieces(int unit) const {
    return cta_of((int64_t)(unit + 1) * nt - 1) - cta_of((int64_t)unit * nt) + 1;
  }
};

// Exponents of one f32 tile of one KV head, for each group of 16 keys: keys are
// stored as k 2^-ek (k_mul = 2^ek), values as v 2^-ev.
struct TileExps {
  float k_mul[8];
  int32_t v_exp[8];
};

// Where the tiles of sequence i, whose first key row is k0, begin among all
// tiles: no sequence's tiles reach the next one's, and no sum over the
// sequences is needed.
__host__ __device__ constexpr int seq_tile(int k0, int i) { return k0 / kTileN + i; }
// Room for all tiles.
constexpr int64_t key_tiles(int64_t k_rows, int64_t n) { return k_rows / kTileN + n; }

// One batch of a tiled launch.  Causal prompts: q_off and k_off give the
// sequences.  Prefix of a shared batch (q_off null): one sequence of n_rows
// query positions, every one of which sees all n_keys keys.
struct TileArgs {
  const int32_t *q_off, *k_off;
  int64_t q_rows, k_rows;  // extents of the tensors
  int32_t n, causal;
  int32_t heads, kv_heads, group, tp;  // tp: positions of a query tile, 128 / group
  int32_t d, dv;
  int32_t per;     // query tiles of a unit: 2, or 1 (f32)
  Shares shares;   // prefix
  uint32_t* counter;  // prompts: units begun beyond the first of each CTA; null:
                      // every CTA takes every gridDim.x-th
  int32_t tail;    // prompts: cut the units of the last, partial round
  float scale;
  Rows q;               // (f32; the 16-bit kernel reads it by its map)
  Rows out;             // results of whole units
  float* lse;           // [q_rows][heads] or null
  float *part, *part_lse;  // pieces' results [slot][per * 128 rows][dv], [..]
  // Keys in pages (prefix): their numbers, tokens a page, pages in the pool.
  const int32_t* pages;
  int32_t page, box;
  int64_t n_pages;
  // f32: K and V as pieces, tile by tile (nys_attn_tc32.cu).
  unsigned char *k_image, *v_image;
  TileExps* exps;
  uint8_t* odd;  // [tile][KV head][keys, values][group]: what the group says of the range
                 // of its numbers (nys_attn_tc32.cu)
  // Values and keys for the checks of unusual values, and the pages' own rows.
  const void *k_raw, *v_raw;
  int64_t k_row, k_head, v_row, v_head;
  int32_t kv_y;  // 0 where all KV heads share one head's rows (head stride 0)
  int32_t* status;
  int32_t stall;  // test hook: what the first CTA withholds (kStall..)
};
enum : int32_t { kStallNone = 0, kStallCopies = 1, kStallProducts = 2 };
// The next tiled launch's `stall`, once (any thread).
void stall_next(int32_t what);

// One unit: two query tiles of one KV head that read the same keys ("pair"),
// or, where the second tile would be empty, one tile whose key tiles two
// streams take in turn.
struct Unit {
  int32_t valid;
  int32_t q_row;    // first query row
  int32_t np0, np1; // positions in the tiles; np1 == 0: one tile
  int32_t kvh;
  int32_t k_row;    // the sequence's first key row
  int32_t kb;       // first key of the piece
  int32_t nt;       // key tiles of the piece
  int32_t nt0;      // of them, those the first tile reads (pair)
  int32_t lim;      // keys that position 0 sees (may be <= 0)
  int32_t nkl;      // keys the piece ends before
  int32_t slot;     // where a piece's results go; -1: a whole unit, to `out`
  int32_t edge;     // first key tile in which some row does not see some key
  int32_t patch;    // (16-bit) set where the epilogue has to add values that are not finite
  int32_t tile;     // number of the piece's first key tile among all (f32)
};

struct TileMaps {
  CUtensorMap q, k, v;
};

// The prefix's pieces and a request's own keys: at most `pieces` (1: all of them,
// and the result is final) of at least `keys` keys, with their results
// [piece][n * heads][dv].
struct OwnArgs {
  Shares shares;  // units == 0: no prefix
  const float *part, *part_lse;  // the prefix's
  int32_t per;
  int32_t pieces, keys;
  int32_t cluster;  // a request's pieces are one cluster and join themselves
  int32_t lead;  // the prefix's keys, read with each request's own
  float *own, *own_lse;
};

// Workspace of the tiled kernels: nys_attn_prompt with n sequences of `rows` query
// rows and `keys` key rows in all; nys_attn_shared with n requests and a prefix of
// `keys`.
size_t prompt_workspace(const nys_attn_config& c, int64_t n, int64_t rows, int64_t keys);
size_t shared_workspace(const nys_attn_config& c, int64_t n, int64_t keys);
bool shared_tiled_fits(const SharedArgs& a);
cudaError_t launch_shared_tiled(const SharedArgs& a, void* workspace, cudaStream_t stream);
cudaError_t launch_own(const SharedArgs& a, const OwnArgs& o, cudaStream_t stream);
cudaError_t launch_join(const SharedArgs& a, const OwnArgs& o, cudaStream_t stream);

// Whether the tiled kernels take a prompt batch, and its launch.
bool prompt_tc_fits(const PromptArgs& a);
cudaError_t launch_prompt_tc(const PromptArgs& a, void* workspace, cudaStream_t stream);
cudaError_t launch_attn_tc(const TileArgs& a, const TileMaps& m, int dtype, unsigned grid,
                           cudaStream_t stream);

cudaError_t launch_attn_tc32(const TileArgs& a, unsigned grid, cudaStream_t stream);
// Joins the pieces of a prompt's cut units (after a launch of `ctas` CTAs).
cudaError_t launch_tail_join(const TileArgs& a, int dtype, unsigned ctas, cudaStream_t stream);

#ifdef __CUDACC__
// Launches `kernel` as a programmatic dependent of the launch before it: its
// CTAs may start while that one's last ones run, and wait for it themselves.
template <typename... P, typename... Q>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                                    cudaStream_t stream, Q... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

// Values that are not finite are 0 in what the products read; the rows that see
// their keys get them here, after their results were written: `out` is this
// thread's row, x += z (infinities stay, opposite ones and NaN give NaN).
template <typename T, typename V>
__device__ __forceinline__ void add_unusual(T* out, const V* v, int c0, int c1) {
  for (int c = c0; c < c1; ++c) {
    const float z = (float)v[c];
    if (!isfinite(z)) out[c] = (T)((float)out[c] + z);
  }
}

// Walks the launch's units in order; one warp.  32 sequences at a time, one a
// lane; among those the query tiles of the last positions of the longest prompts
// come first, because under the causal mask those are the longest, and short work
// fills the gaps that long work leaves.  Level l is the l-th unit of each
// sequence that has one; a level's units lie next to each other, each sequence's
// KV heads together.
struct UnitWalk {
  int32_t before = 0;  // units of the windows and levels before
  int s0 = 0;          // the window's first sequence, 32 of them
  int level = 0;
  int q0, nq, k0, nk, pairs;

  __device__ __forceinline__ void load(const TileArgs& a, int lane) {
    const int i = s0 + lane;
    q0 = nq = k0 = nk = 0;
    if (i < a.n) {
      bool bad = false;
      seq_range(a.q_off, i, a.q_rows, q0, nq, bad);
      seq_range(a.k_off, i, a.k_rows, k0, nk, bad);
      if (bad) attn_report(a.status, NYS_ATTN_BAD_OFFSETS);
    }
    pairs = (nq + a.per * a.tp - 1) / (a.per * a.tp);
    level = __reduce_max_sync(0xffffffffu, pairs) - 1;
  }

  // All units of the launch.
  static __device__ __forceinline__ int32_t total(const TileArgs& a, int lane) {
    UnitWalk w;
    int32_t sum = 0;
    for (w.s0 = 0; w.s0 < a.n; w.s0 += 32) {
      w.load(a, lane);
      sum += __reduce_add_sync(0xffffffffu, w.pairs) * a.kv_heads;
    }
    return sum;
  }

  // Unit number w (not descending from call to call) into `u` in every lane;
  // u.valid == 0 past the last.
  __device__ __forceinline__ void get(const TileArgs& a, int32_t w, int lane, Unit& u) {
    u.valid = 0;
    u.patch = 0;
    uint32_t have;  // sequences of this level
    for (;;) {
      have = __ballot_sync(0xffffffffu, pairs > level);
      const int32_t all = level >= 0 ? __popc(have) * a.kv_heads : 0;
      if (w < before + all) break;
      before += all;
      if (--level < 0) {
        s0 += 32;
        if (s0 >= a.n) return;
        load(a, lane);
      }
    }
    const int32_t r = w - before;
    const int src = __fns(have, 0, r / a.kv_heads + 1);
    const int sq0 = __shfl_sync(0xffffffffu, q0, src), snq = __shfl_sync(0xffffffffu, nq, src);
    const int sk0 = __shfl_sync(0xffffffffu, k0, src), snk = __shfl_sync(0xffffffffu, nk, src);
    u.slot = -1;
    u.kvh = r % a.kv_heads;
    const int p0 = level * a.per * a.tp;
    const int left = snq - p0;
    u.np0 = min(left, a.tp);
    u.np1 = a.per == 2 ? min(max(left - a.tp, 0), a.tp) : 0;
    u.q_row = sq0 + p0;
    u.k_row = sk0;
    u.tile = seq_tile(sk0, s0 + src);
    // Keys that the first position sees, and the last of each tile.
    u.lim = p0 + 1 + snk - snq;
    const int e0 = u.lim + u.np0 - 1, e1 = e0 + u.np1;
    const int t0 = (min(max(e0, 0), snk) + kTileN - 1) / kTileN;
    const int t1 = (min(max(e1, 0), snk) + kTileN - 1) / kTileN;  // t1 >= t0
    u.kb = 0;
    u.nt = t1;
    u.nt0 = t0;
    u.nkl = snk;
    u.edge = max(min(u.lim, u.nkl) - u.kb, 0) / kTileN;
    u.valid = 1;
  }
};

// Piece k of CTA `cta`'s share of a prefix; u.valid == 0 past the last.
__device__ __forceinline__ void prefix_unit(const TileArgs& a, int cta, int k, Unit& u) {
  u.valid = 0;
  u.patch = 0;
  const Shares& s = a.shares;
  const int64_t t0 = s.begin(cta), t1 = s.begin(cta + 1);
  const int unit = (int)(t0 / s.nt) + k;
  const int64_t first = (int64_t)unit * s.nt;
  if (first >= t1) return;
  const int tb = (int)(t0 > first ? t0 - first : 0);
  const int te = (int)(t1 - first < s.nt ? t1 - first : s.nt);
  const int p0 = unit / a.kv_heads * s.rows, left = (int)a.q_rows - p0;
  u.kvh = unit % a.kv_heads;
  u.np0 = min(left, a.tp);
  u.np1 = a.per == 2 ? min(max(left - a.tp, 0), a.tp) : 0;
  u.q_row = p0;
  u.k_row = 0;
  u.lim = (int)a.k_rows;
  u.kb = tb * kTileN;
  u.tile = tb;
  u.nt = u.nt0 = te - tb;
  u.nkl = min((int)a.k_rows, te * kTileN);
  u.edge = (u.nkl - u.kb) / kTileN;
  u.slot = unit + cta;
  u.valid = 1;
}

// Where a launch of `ctas` CTAs has units for some whole rounds and a rest, the
// rest's units are cut into as many pieces as there are CTAs for each.
struct Tail {
  int32_t full = INT32_MAX, cut = 1, units = 0;  // units before the rest; pieces; units of the rest
  __device__ __forceinline__ void find(const TileArgs& a, int ctas, int lane) {
    const int32_t all = UnitWalk::total(a, lane), rest = all % ctas;
    if (rest > 0 && ctas / rest >= 2) {
      full = all - rest;
      cut = ctas / rest;
      units = rest;
    }
  }
};
// Of `cut` pieces of a whole unit, those that are not empty: of two tiles at least,
// and more than 32 only of 16 and more (the join reads a piece after the other).
__device__ __forceinline__ int cut_pieces(const Unit& u, int cut) {
  return min(min(cut, max(u.nt / 2, 1)), max(32, u.nt / 16));
}
// Piece p of `cut` of a whole unit.
__device__ __forceinline__ void cut_unit(Unit& u, int p, int cut, int slot) {
  const int c = cut_pieces(u, cut);
  const int tb = p < c ? u.nt * p / c : u.nt, te = p < c ? u.nt * (p + 1) / c : u.nt;
  u.slot = slot;
  u.kb = tb * kTileN;
  u.tile += tb;
  u.nt0 = min(max(u.nt0 - tb, 0), te - tb);
  u.nt = te - tb;
  u.nkl = min(u.nkl, te * kTileN);
  u.edge = max(min(u.lim, u.nkl) - u.kb, 0) / kTileN;
}

// The next unit of this CTA, one warp's work.  Calls give k = 0, 1, ..
struct UnitSource {
  UnitWalk walk;
  Tail tail;
  __device__ __forceinline__ void begin(const TileArgs& a, int lane) {
    if (!a.q_off) return;
    walk.load(a, lane);
    if (a.tail) tail.find(a, gridDim.x, lane);
  }
  __device__ __forceinline__ void next(const TileArgs& a, int k, int lane, Unit& u) {
    if (!a.q_off) {
      prefix_unit(a, blockIdx.x, k, u);
      return;
    }
    // Without a counter every other round runs backwards, so that no CTA gets
    // the longer unit of every round.
    int32_t w = k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    if (a.counter) {
      w = blockIdx.x;
      if (k > 0) {
        uint32_t c = 0;
        if (lane == 0) c = atomicAdd(a.counter, 1u);
        w = gridDim.x + __shfl_sync(0xffffffffu, c, 0);
      }
    }
    if (w < tail.full) {
      walk.get(a, w, lane, u);
    } else {
      const int32_t v = w - tail.full, r = v / tail.cut;
      u.valid = 0;
      if (r >= tail.units) return;
      walk.get(a, tail.full + r, lane, u);
      if (u.valid) cut_unit(u, v - r * tail.cut, tail.cut, v);
    }
  }
};

// The kernel launched next (a programmatic dependent) may start; and: all that
// kernels before this one wrote is visible.
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
#endif

}  // namespace nys
