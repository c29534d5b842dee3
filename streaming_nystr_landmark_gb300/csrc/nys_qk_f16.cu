// Rows of f16 between the projections and attention: the kernels are in nys_qk.cuh.
#include "nys_qk.cuh"

namespace nys {

cudaError_t launch_qk_f16(const QkArgs& a, cudaStream_t stream) {
  return a.blocks ? launch_of<__half, true>(a, stream) : launch_of<__half, false>(a, stream);
}
cudaError_t launch_read4_f16(const Read4Args& a, cudaStream_t stream) {
  return launch_read_of<__half>(a, stream);
}

}  // namespace nys
