// Attention over a cache in 4 bits for f32 rows: the kernels are in nys_attn4.cuh.
#include "nys_attn4.cuh"

namespace nys {

cudaError_t launch_attn4_f32(const Attn4Args& a, void* workspace, cudaStream_t stream) {
  return launch_any<true>(a, workspace, stream);
}

}  // namespace nys
