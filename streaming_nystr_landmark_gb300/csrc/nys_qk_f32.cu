// Rows of f32 between the projections and attention: the kernels are in nys_qk.cuh.
#include "nys_qk.cuh"

namespace nys {

cudaError_t launch_qk_f32(const QkArgs& a, cudaStream_t stream) {
  return a.blocks ? launch_of<float, true>(a, stream) : launch_of<float, false>(a, stream);
}
cudaError_t launch_read4_f32(const Read4Args& a, cudaStream_t stream) {
  return launch_read_of<float>(a, stream);
}

cudaError_t launch_qk(const QkArgs& a, cudaStream_t stream) {
  if (a.tokens == 0) return cudaSuccess;
  return a.dtype == NYS_F32 ? launch_qk_f32(a, stream)
         : a.dtype == NYS_BF16 ? launch_qk_bf16(a, stream) : launch_qk_f16(a, stream);
}
cudaError_t launch_read4(const Read4Args& a, cudaStream_t stream) {
  if (a.tokens == 0) return cudaSuccess;
  return a.dtype == NYS_F32 ? launch_read4_f32(a, stream)
         : a.dtype == NYS_BF16 ? launch_read4_bf16(a, stream) : launch_read4_f16(a, stream);
}

}  // namespace nys
