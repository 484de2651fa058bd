// Kernels of the norms' backward pass, by type (residual stream, block).
#include "block_norm_grad.cuh"

namespace prm {

template <>
cudaError_t norm_grad_launch<__nv_bfloat16, __nv_bfloat16>(NormGradParams& p, const NormShape& s, const NormGradArgs& a,
                                 cudaStream_t stream) {
  return launch_shape<__nv_bfloat16, __nv_bfloat16>(p, s, a, stream);
}

template <>
cudaError_t norm_grad_launch<__half, __half>(NormGradParams& p, const NormShape& s, const NormGradArgs& a,
                                 cudaStream_t stream) {
  return launch_shape<__half, __half>(p, s, a, stream);
}

}  // namespace prm
