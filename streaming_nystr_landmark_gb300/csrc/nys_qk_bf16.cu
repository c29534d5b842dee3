// Rows of bf16 between the projections and attention: the kernels are in nys_qk.cuh.
#include "nys_qk.cuh"

namespace nys {

cudaError_t launch_qk_bf16(const QkArgs& a, cudaStream_t stream) {
  return a.blocks ? launch_of<__nv_bfloat16, true>(a, stream) : launch_of<__nv_bfloat16, false>(a, stream);
}
cudaError_t launch_read4_bf16(const Read4Args& a, cudaStream_t stream) {
  return launch_read_of<__nv_bfloat16>(a, stream);
}

}  // namespace nys
