// Host side of the tiled attention kernels: which calls they take, tensor maps
// and launch shapes.
#include <cstdint>
#include <cstring>

#include "nys_attn_tc.h"

namespace nys {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (the library links no libcuda).
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

// Map of a [rows][heads][dim] tensor of 16-bit elements; boxes of 64 columns,
// `box_h` heads and `box_r` rows, 128-byte swizzle.  Strides in elements; those
// of extents of one are not used and replaced by valid ones.
bool make_map(CUtensorMap* m, bool bf16, const void* p, int64_t rows, int64_t heads, int64_t dim,
              int64_t row, int64_t head, int box_h, int box_r) {
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t line = (cuuint64_t)((dim * 2 + 15) & ~int64_t(15));
  const cuuint64_t st[2] = {heads > 1 ? (cuuint64_t)head * 2 : line,
                            rows > 1 ? (cuuint64_t)row * 2 : line * (cuuint64_t)heads};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_h, (cuuint32_t)box_r};
  const cuuint32_t one[3] = {1, 1, 1};
  const EncodeTiled enc = encoder();
  return enc && enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                    3, const_cast<void*>(p), dims, st, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
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

}  // namespace

bool prompt_tc_fits(const PromptArgs& a) {
  if (a.dtype == NYS_F32 || a.d > 128 || a.dv > 128 || a.d % 8 || a.dv % 8) return false;
  if (a.k_rows == 0 || a.k_rows > (1 << 30) || a.q_rows > (1 << 30)) return false;
  // K and V share the choice between a KV head's own rows and one head's rows.
  const bool kb = a.kv_heads > 1 && a.k.head == 0, vb = a.kv_heads > 1 && a.v.head == 0;
  return kb == vb && tileable(a.q, a.q_rows, a.heads, 2, false) &&
         tileable(a.k, a.k_rows, a.kv_heads, 2, true) &&
         tileable(a.v, a.k_rows, a.kv_heads, 2, true) &&
         tileable(a.out, a.q_rows, a.heads, 2, false);
}

cudaError_t launch_prompt_tc(const PromptArgs& p, cudaStream_t stream) {
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
  TileMaps m;
  const bool bf16 = p.dtype == NYS_BF16;
  const int64_t kvh = a.kv_y ? p.kv_heads : 1;
  if (!make_map(&m.q, bf16, p.q.p, p.q_rows, p.heads, p.d, p.q.row, p.q.head, p.group, a.tp) ||
      !make_map(&m.k, bf16, p.k.p, p.k_rows, kvh, p.d, p.k.row, p.k.head, 1, kTileN) ||
      !make_map(&m.v, bf16, p.v.p, p.k_rows, kvh, p.dv, p.v.row, p.v.head, 1, kTileN))
    return cudaErrorInvalidValue;
  // At most this many units: a partial pair a sequence on top of the full ones.
  const int64_t most = (p.q_rows / (2 * a.tp) + p.n) * p.kv_heads;
  return launch_attn_tc(a, m, p.dtype, (unsigned)(most < kSms ? most : kSms), stream);
}

}  // namespace nys
