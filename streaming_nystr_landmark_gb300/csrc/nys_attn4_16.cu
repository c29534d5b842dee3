// Attention over a cache in 4 bits for 16-bit rows: the kernels are in nys_attn4.cuh.
#include "nys_attn4.cuh"

namespace nys {

cudaError_t launch_attn4_16(const Attn4Args& a, void* workspace, cudaStream_t stream) {
  return launch_any<false>(a, workspace, stream);
}

size_t attn4_workspace(const nys_attn_config& c, int64_t n, int64_t keys) {
  if (n == 0) return 0;
  const int G = groups4(c.d, c.dv);
  const Plan4 p = plan_of(G, n, c.kv_heads, c.heads / c.kv_heads, keys);
  if (p.pieces == 0) return 0;
  return up256(p.units * sizeof(Cut4)) + up256(p.pieces * p.heads * sizeof(float2)) +
         up256(p.pieces * p.heads * sizeof(float) * 64 * G);
}

cudaError_t launch_attn4(const Attn4Args& a, void* workspace, cudaStream_t stream) {
  return a.dtype == NYS_F32 ? launch_attn4_f32(a, workspace, stream) : launch_attn4_16(a, workspace, stream);
}

}  // namespace nys
