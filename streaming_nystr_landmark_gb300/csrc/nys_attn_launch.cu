// Host side of the tiled attention kernels: which calls they take, tensor maps
// and launch shapes.
#include <atomic>
#include <cstdint>
#include <cstring>

#include "nys_attn_tc.h"

namespace nys {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// CUDA's encoder of tensor maps, looked up once (the library links no libcuda).
EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return (EncodeTiled) nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// Map of a [rows][heads][dim] tensor of 16-bit elements for tiles in shared
// memory of [64-column block][row][head][64 columns], 128-byte swizzle: its
// dimensions are 64 columns, heads, rows, blocks, so that one copy of a full
// tile's 128 rows brings all blocks (a copy costs its thread about 200 clocks to
// issue); smaller boxes bring one block.  A dim that is no multiple of 64 has one
// block of `dim` columns instead, of which a copy takes 64, with zeros past the
// end.  Strides in elements; those of extents of one are not used and replaced
// by valid ones.
bool make_map(CUtensorMap* m, int dtype, const void* p, int64_t rows, int64_t heads, int64_t dim,
              int64_t row, int64_t head, int box_h, int box_r) {
  const bool whole = dim % 64 == 0;
  const cuuint64_t blocks = whole ? (cuuint64_t)(dim / 64) : 1;
  const cuuint64_t dims[4] = {(cuuint64_t)(whole ? 64 : dim), (cuuint64_t)heads, (cuuint64_t)rows,
                              blocks};
  const cuuint64_t line = (cuuint64_t)((dim * 2 + 15) & ~int64_t(15));
  const cuuint64_t st[3] = {heads > 1 ? (cuuint64_t)head * 2 : line,
                            rows > 1 ? (cuuint64_t)row * 2 : line * (cuuint64_t)heads,
                            blocks > 1 ? 128 : line * (cuuint64_t)heads * (cuuint64_t)rows};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_h, (cuuint32_t)box_r,
                             box_h * box_r == kTileM ? (cuuint32_t)blocks : 1u};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const EncodeTiled enc = encoder();
  return enc && enc(m,
                    dtype == NYS_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                    4, const_cast<void*>(p), dims, st, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A tensor that TMA can read and 16-byte stores can write: aligned base and
// strides; `bcast`: a head stride of 0 is taken (all heads read one head).
bool tileable(const Rows& r, int64_t rows, int heads, int elem, bool bcast) {
  const int64_t row = r.row * elem, head = r.head * elem;
  if (reinterpret_cast<uintptr_t>(r.p) % 16) return false;
  if (rows > 1 && (row <= 0 || row % 16 || row >= (int64_t(1) << 40))) return false;
  if (heads > 1 && !(bcast && head == 0) &&
      (head <= 0 || head % 16 || head >= (int64_t(1) << 40)))
    return false;
  return true;
}

constexpr int kSms = 152;
constexpr int kMostPieces = 64;

// Query tiles of a unit: tensor memory holds two of 16-bit types, one of f32.
int query_tiles(int dtype) { return dtype == NYS_F32 ? 1 : 2; }
int64_t div_up(int64_t x, int64_t y) { return (x + y - 1) / y; }
int clamp_int(int64_t x, int lo, int hi) { return (int)(x < lo ? lo : (x > hi ? hi : x)); }

// How a prefix of `tiles` key tiles is dealt out: an even share for each SM, but
// at least two tiles a CTA (a CTA's start costs about three tiles' time; four in
// f32, where the own pages are read beside it on the SMs that it leaves) and no
// more pieces of a unit than the join takes.  tiles == 0: a prefix without end
// (bounds the workspace by the batch alone).
Shares shares_of(int64_t n, int kv_heads, int group, int dtype, int64_t tiles) {
  Shares s{};
  s.tp = kTileM / group;
  s.rows = query_tiles(dtype) * s.tp;
  s.units = (int32_t)(div_up(n, s.rows) * kv_heads);
  s.nt = (int32_t)(tiles > 0 ? tiles : INT32_MAX / 2);
  const int64_t all = (int64_t)s.units * s.nt;
  int64_t ctas = kSms;
  if (ctas > (int64_t)s.units * (kMostPieces - 2)) ctas = (int64_t)s.units * (kMostPieces - 2);
  const int least = dtype == NYS_F32 ? 4 : 2;
  if (ctas > div_up(all, least)) ctas = div_up(all, least);
  s.ctas = (int32_t)ctas;
  return s;
}
// CTAs of the own keys' kernel for one piece a request: each has up to 8 (f32) or
// 16 heads of a group.
int64_t own_ctas(int64_t n, int kv_heads, int group, int dtype) {
  return n * kv_heads * div_up(group, dtype == NYS_F32 ? 8 : 16);
}
// Pieces of a request's own keys at most.  Requests differ in length and one CTA
// reads at a fraction of the memory's rate, so long ones are cut: 64 requests of
// 97 to 1025 keys, 8 KV heads, f32, whole call: two pieces 45 us, five 39 us.
// With six CTAs a SM's worth of requests the lengths even out by themselves, and
// whole requests need no join: 256 requests of 1 to 517 keys, 4 KV heads, over a
// prefix of 32,768, bf16, 147 us whole and 155 us cut.
int most_own_pieces(int64_t ctas) {
  if (ctas >= 6 * kSms) return 1;
  return clamp_int(div_up(16 * kSms, ctas), 1, kMostPieces);
}
// Keys of a piece at least.  With few CTAs a piece's own length is the call's time
// (one request of 346 keys, 8 KV heads, f32, joined by a launch: 128 keys 8.6 us, 192
// 10.7 us; four of 500 to 700: 10.7 and 11.6 us); with more, the pieces that are joined are (40
// requests of 500 to 700: 256 keys 38 us, 192 43 us).
int least_own_keys(int64_t ctas) { return ctas <= 48 ? 128 : 256; }
// Pieces of a request where they are one cluster, which joins them in shared memory
// instead of by another launch; 0: they are not.  Clusters hold their places until
// their last piece is done, so they pay where all CTAs run at once, three a SM: 4
// requests of 500 to 700 keys, 16 heads on 8, f32 10.7 -> 8.4 us, 16 of them (384
// CTAs) 15.5 -> 13.7 us, 64 (1,536 CTAs) 57.9 -> 64.5 us.  More than 8 pieces, a
// cluster's most, are worth giving up to 512 keys each (one request of up to 4,000,
// bf16, 16.3 -> 13.6 us), but not in f32 with many heads on a key (22 -> 26 us).
int cluster_pieces(int64_t ctas, int64_t cap, int pieces, int group, int dtype) {
  constexpr int kMost = 8;
  if (pieces > kMost && (cap > kMost * 512 || (dtype == NYS_F32 && group > 2))) return 0;
  if (pieces > kMost) pieces = kMost;
  return pieces > 1 && ctas * pieces <= 3 * kSms ? pieces : 0;
}
// Whether each request reads the prefix's keys for itself, in front of its own: no
// tile kernel, no split, one join less.  It pays until the rows read again weigh
// more (few requests or a short prefix): 4 requests of 3 to 45 keys over 301, bf16,
// 8 KV heads, 6.6 us against 14.4 us; f32 7.1 against 20.6 us; 64 over 301, 4 KV
// heads (77,000 rows), bf16 20.6 against 26.8 us, f32 29.0 against 25.5 us; 16 over
// 1,000, 8 KV heads (128,000 rows), bf16 21.5 against 14.0 us.
bool read_with_own(int64_t ctas, int64_t prefix, int dtype) {
  return prefix > 0 && ctas * prefix <= (dtype == NYS_F32 ? 60000 : 80000);
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// The f32 images' part of a workspace: K, V, exponents, flags.
struct Images {
  size_t v, exps, odd, end;
};
Images images_of(int kv_heads, int d, int dv, int64_t n, int64_t keys) {
  const size_t count = (size_t)key_tiles(keys, n) * kv_heads;
  Images im;
  im.v = count * 2 * (size_t)((d + 63) / 64) * 16384;
  im.exps = im.v + count * 2 * (size_t)((dv + 63) / 64) * 16384;
  im.odd = im.exps + count * sizeof(TileExps);
  im.end = (im.odd + count * 16 + 255) & ~size_t(255);
  return im;
}
void place_images(TileArgs& a, void* workspace, int64_t n, int64_t keys) {
  unsigned char* w = static_cast<unsigned char*>(workspace);
  const Images im = images_of(a.kv_heads, a.d, a.dv, n, keys);
  a.k_image = w;
  a.v_image = w + im.v;
  a.exps = reinterpret_cast<TileExps*>(w + im.exps);
  a.odd = w + im.odd;
}

constexpr size_t kCounterBytes = 256;
size_t slot_bytes(int dtype, int dv) {
  return (size_t)query_tiles(dtype) * kTileM * ((size_t)dv + 1) * 4;
}
// Units of a prompt batch, at most: a partial one a sequence on top of the full
// ones.
int64_t prompt_units(int64_t n, int64_t rows, int kv_heads, int group, int dtype) {
  return (rows / (query_tiles(dtype) * (kTileM / group)) + n) * kv_heads;
}
// Whether the last round's units are cut; where units are fewer than CTAs, that
// is all of them.  It pays where rounds are few and long: 2 prompts' last 1,021 and
// 1,500 tokens over 5,003 earlier ones, f32, 320 units of 45 tiles on 152 CTAs,
// take 303 us whole and 277 us cut (whole calls, the join's 11 us among them); one
// new token over 4,000, 8 KV heads, 72 and 32 us, over 30,000 in bf16 183 and 38 us;
// over 1,100, f32 28 and 25 us, but bf16 15.5 and 16.3 us.
bool cut_tail(int64_t n, int64_t rows, int64_t keys, int kv_heads, int group, int dtype) {
  const int64_t units = prompt_units(n, rows, kv_heads, group, dtype);
  return n <= 128 && keys >= (dtype == NYS_F32 ? 1024 : 1536) * n && units <= 8 * kSms;
}
// Whether CTAs take their units from a counter: where each has some, and they
// may differ.
bool count_units(int64_t units) { return units > kSms; }

std::atomic<int32_t> stalled{kStallNone};
int32_t take_stall() {
  return stalled.load(std::memory_order_relaxed) == kStallNone ? kStallNone
                                                               : stalled.exchange(kStallNone);
}

}  // namespace

void stall_next(int32_t what) { stalled.store(what); }

// Images (f32), a counter, pieces of cut units.
size_t prompt_workspace(const nys_attn_config& c, int64_t n, int64_t rows, int64_t keys) {
  if (n == 0 || keys == 0 || c.d > 128 || c.dv > 128) return 0;
  const int group = c.heads / c.kv_heads;
  size_t all = c.dtype == NYS_F32 ? images_of(c.kv_heads, c.d, c.dv, n, keys).end : 0;
  all += kCounterBytes;
  if (cut_tail(n, rows, keys, c.kv_heads, group, c.dtype)) all += kSms * slot_bytes(c.dtype, c.dv);
  return all;
}

// Images (f32), the prefix's pieces, the own keys' pieces.
size_t shared_workspace(const nys_attn_config& c, int64_t n, int64_t keys) {
  if (n == 0 || c.d > 128 || c.dv > 128) return 0;
  size_t all = c.dtype == NYS_F32 && keys > 0 ? images_of(c.kv_heads, c.d, c.dv, 1, keys).end : 0;
  if (keys > 0)
    all += shares_of(n, c.kv_heads, c.heads / c.kv_heads, c.dtype, 0).slots() *
           slot_bytes(c.dtype, c.dv);
  const int64_t ctas = own_ctas(n, c.kv_heads, c.heads / c.kv_heads, c.dtype);
  return all + (size_t)most_own_pieces(ctas) * n * c.heads * ((size_t)c.dv + 1) * 4;
}

bool shared_tiled_fits(const SharedArgs& a) {
  const int elem = a.dtype == NYS_F32 ? 4 : 2, unit = 16 / elem;
  if (a.d > 128 || a.dv > 128 || a.d % unit || a.dv % unit || a.n_pages == 0) return false;
  if (reinterpret_cast<uintptr_t>(a.k) % 16 || reinterpret_cast<uintptr_t>(a.v) % 16) return false;
  if (a.n_pages * a.page > (1 << 30) || a.n_pages * a.page * a.kv_heads > INT32_MAX) return false;
  if ((int64_t)a.width * a.page > (1 << 30)) return false;
  if (!tileable(a.q, a.n, a.heads, elem, false)) return false;
  if (a.prefix_len > 0 && a.dtype != NYS_F32 && a.page % 8 &&
      !read_with_own(own_ctas(a.n, a.kv_heads, a.group, a.dtype), a.prefix_len, a.dtype))
    return false;
  return true;
}

cudaError_t launch_shared_tiled(const SharedArgs& s, void* workspace, cudaStream_t stream) {
  const int64_t row = (int64_t)s.n * s.heads;
  OwnArgs o{};
  const int64_t ctas = own_ctas(s.n, s.kv_heads, s.group, s.dtype);
  if (read_with_own(ctas, s.prefix_len, s.dtype)) o.lead = s.prefix_len;
  else if (s.prefix_len > 0)
    o.shares = shares_of(s.n, s.kv_heads, s.group, s.dtype, div_up(s.prefix_len, kTileN));
  const int64_t cap = o.lead + (int64_t)s.width * s.page;
  o.keys = least_own_keys(ctas);
  o.pieces = clamp_int(div_up(cap, o.keys), 1, most_own_pieces(ctas));
  if (o.shares.units == 0) {
    const int pieces = cluster_pieces(ctas, cap, o.pieces, s.group, s.dtype);
    o.cluster = pieces > 1;
    if (o.cluster) o.pieces = pieces;
  }
  const size_t images = s.dtype == NYS_F32 && o.shares.units > 0
                            ? images_of(s.kv_heads, s.d, s.dv, 1, s.prefix_len).end
                            : 0;
  // The prefix's pieces, the own pieces, then both's sums.
  const int64_t rows = (int64_t)o.shares.slots() * query_tiles(s.dtype) * kTileM;
  float* part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + images);
  o.per = query_tiles(s.dtype);
  o.own = part + rows * s.dv;
  float* part_lse = o.own + (int64_t)o.pieces * row * s.dv;
  o.own_lse = part_lse + rows;
  o.part = part;
  o.part_lse = part_lse;
  if (o.shares.units > 0) {
    TileArgs a{};
    a.q_rows = s.n;
    a.k_rows = s.prefix_len;
    a.n = 1;
    a.heads = s.heads;
    a.kv_heads = s.kv_heads;
    a.group = s.group;
    a.tp = kTileM / s.group;
    a.d = s.d;
    a.dv = s.dv;
    a.shares = o.shares;
    a.scale = s.scale;
    a.part = part;
    a.part_lse = part_lse;
    a.pages = s.prefix_pages;
    a.page = s.page;
    a.n_pages = s.n_pages;
    a.k_raw = s.k;
    a.v_raw = s.v;
    a.k_row = (int64_t)s.kv_heads * s.d;
    a.k_head = s.d;
    a.v_row = (int64_t)s.kv_heads * s.dv;
    a.v_head = s.dv;
    a.kv_y = 1;
    a.status = s.status;
    a.stall = take_stall();
    a.q = s.q;
    a.per = query_tiles(s.dtype);
    const unsigned grid = (unsigned)o.shares.ctas;
    cudaError_t e;
    if (s.dtype == NYS_F32) {
      place_images(a, workspace, 1, s.prefix_len);
      e = launch_attn_tc32(a, grid, stream);
    } else {
      a.box = gcd(s.page, kTileN);
      const int64_t slots = s.n_pages * s.page;
      TileMaps m;
      if (!make_map(&m.q, s.dtype, s.q.p, s.n, s.heads, s.d, s.q.row, s.q.head, s.group, a.tp) ||
          !make_map(&m.k, s.dtype, s.k, slots, s.kv_heads, s.d, a.k_row, a.k_head, 1, a.box) ||
          !make_map(&m.v, s.dtype, s.v, slots, s.kv_heads, s.dv, a.v_row, a.v_head, 1, a.box))
        return cudaErrorInvalidValue;
      e = launch_attn_tc(a, m, s.dtype, grid, stream);
    }
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = launch_own(s, o, stream);
  if (e != cudaSuccess || o.pieces == 1 || o.cluster) return e;
  return launch_join(s, o, stream);
}

bool prompt_tc_fits(const PromptArgs& a) {
  const int elem = a.dtype == NYS_F32 ? 4 : 2, unit = 16 / elem;
  if (a.d > 128 || a.dv > 128 || a.d % unit || a.dv % unit) return false;
  if (a.k_rows == 0 || a.k_rows > (1 << 30) || a.q_rows > (1 << 30)) return false;
  if ((a.q_rows / (kTileM / a.group) + a.n) * a.kv_heads > (1 << 30)) return false;  // units
  // K and V share the choice between a KV head's own rows and one head's rows.
  const bool kb = a.kv_heads > 1 && a.k.head == 0, vb = a.kv_heads > 1 && a.v.head == 0;
  return kb == vb && tileable(a.q, a.q_rows, a.heads, elem, false) &&
         tileable(a.k, a.k_rows, a.kv_heads, elem, true) &&
         tileable(a.v, a.k_rows, a.kv_heads, elem, true) &&
         tileable(a.out, a.q_rows, a.heads, elem, false);
}

cudaError_t launch_prompt_tc(const PromptArgs& p, void* workspace, cudaStream_t stream) {
  TileArgs a{};
  a.q_off = p.q_off;
  a.k_off = p.k_off;
  a.q_rows = p.q_rows;
  a.k_rows = p.k_rows;
  a.n = p.n;
  a.causal = 1;
  a.heads = p.heads;
  a.kv_heads = p.kv_heads;
  a.group = p.group;
  a.tp = kTileM / p.group;
  a.d = p.d;
  a.dv = p.dv;
  a.scale = p.scale;
  a.out = p.out;
  a.lse = p.lse;
  a.k_raw = p.k.p;
  a.v_raw = p.v.p;
  a.k_row = p.k.row;
  a.k_head = p.k.head;
  a.v_row = p.v.row;
  a.v_head = p.v.head;
  a.kv_y = !(p.kv_heads > 1 && p.k.head == 0);
  a.status = p.status;
  a.stall = take_stall();
  a.q = p.q;
  a.per = query_tiles(p.dtype);
  const int64_t units = prompt_units(p.n, p.q_rows, p.kv_heads, p.group, p.dtype);
  a.tail = workspace && cut_tail(p.n, p.q_rows, p.k_rows, p.kv_heads, p.group, p.dtype);
  const unsigned grid = (unsigned)(units < kSms && !a.tail ? units : kSms);
  if (workspace) {
    unsigned char* w = static_cast<unsigned char*>(workspace);
    if (p.dtype == NYS_F32) {
      place_images(a, workspace, p.n, p.k_rows);
      w += images_of(p.kv_heads, p.d, p.dv, p.n, p.k_rows).end;
    }
    if (count_units(units)) a.counter = reinterpret_cast<uint32_t*>(w);
    a.part = reinterpret_cast<float*>(w + kCounterBytes);
    a.part_lse = a.part + (int64_t)kSms * a.per * kTileM * p.dv;
  }
  const auto join = [&](cudaError_t e) {
    return e == cudaSuccess && a.tail ? launch_tail_join(a, p.dtype, grid, stream) : e;
  };
  if (p.dtype == NYS_F32) return join(launch_attn_tc32(a, grid, stream));
  if (a.counter) {
    const cudaError_t e = cudaMemsetAsync(a.counter, 0, sizeof(uint32_t), stream);
    if (e != cudaSuccess) return e;
  }
  TileMaps m;
  const int64_t kvh = a.kv_y ? p.kv_heads : 1;
  if (!make_map(&m.q, p.dtype, p.q.p, p.q_rows, p.heads, p.d, p.q.row, p.q.head, p.group, a.tp) ||
      !make_map(&m.k, p.dtype, p.k.p, p.k_rows, kvh, p.d, p.k.row, p.k.head, 1, kTileN) ||
      !make_map(&m.v, p.dtype, p.v.p, p.k_rows, kvh, p.dv, p.v.row, p.v.head, 1, kTileN))
    return cudaErrorInvalidValue;
  return join(launch_attn_tc(a, m, p.dtype, grid, stream));
}

}  // namespace nys
