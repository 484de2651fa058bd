// Kernels of the norms' backward pass, by type (residual stream, block).
#include "block_norm_grad.cuh"

namespace prm {

template <>
cudaError_t norm_grad_launch<float, __nv_bfloat16>(NormGradParams& p, const NormShape& s, const NormGradArgs& a,
                                 cudaStream_t stream) {
  return launch_shape<float, __nv_bfloat16>(p, s, a, stream);
}

template <>
cudaError_t norm_grad_launch<float, __half>(NormGradParams& p, const NormShape& s, const NormGradArgs& a,
                                 cudaStream_t stream) {
  return launch_shape<float, __half>(p, s, a, stream);
}

}  // namespace prm
