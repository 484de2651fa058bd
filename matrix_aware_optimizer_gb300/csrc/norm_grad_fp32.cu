// Kernels of the norms' backward pass, by type (residual stream, block).
#include "block_norm_grad.cuh"

namespace prm {

template <>
cudaError_t norm_grad_launch<float, float>(NormGradParams& p, const NormShape& s, const NormGradArgs& a,
                                 cudaStream_t stream) {
  return launch_shape<float, float>(p, s, a, stream);
}

}  // namespace prm
