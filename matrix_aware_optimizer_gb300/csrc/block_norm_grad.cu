// Planning and checks of the backward pass of the norms around a block; the
// kernels are in block_norm_grad.cuh.
#include "block_norm_grad.cuh"

namespace prm {
namespace {

struct NormGradSpace {
  size_t mod, w;
};
NormGradSpace space(const prm_block_norm_desc& c) {
  const size_t rows = static_cast<size_t>(std::min<int64_t>(c.rows, NORM_CTAS)) * ((c.d + 3) & ~int64_t(3)) *
                      sizeof(float);
  NormGradSpace s{};
  if (c.gate != nullptr || c.scale != nullptr || c.shift != nullptr) s.mod = round_up(6 * rows, 256);
  if (c.post_weight != nullptr || c.pre_weight != nullptr) s.w = 2 * rows;
  return s;
}

}  // namespace
}  // namespace prm

extern "C" int prm_block_norm_workspace(const prm_block_norm_desc* desc, size_t* bytes) {
  using namespace prm;
  if (bytes == nullptr) return PRM_ERR_INVALID_ARG;
  NormParams p;
  const int rc = norm_check(desc, &p);
  if (rc != PRM_OK) return rc;
  const NormGradSpace s = space(*desc);
  *bytes = s.mod + s.w;
  return PRM_OK;
}

extern "C" int prm_block_norm_backward(const prm_block_norm_desc* desc, const void* dy, const void* dr, const void* r,
                                       const void* z, const float* stats, void* dx, void* dz, float* dpost,
                                       void* dgate, float* dpre, void* dscale, void* dshift, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  using namespace prm;
  NormGradParams p{};
  int rc = norm_check(desc, &p.n);
  if (rc != PRM_OK) return rc;
  if (p.n.rows == 0) return PRM_OK;
  if ((dy == nullptr && dr == nullptr) || (dy != nullptr && (r == nullptr || stats == nullptr)))
    return PRM_ERR_INVALID_ARG;
  if (z == nullptr && (desc->post_weight != nullptr || desc->gate != nullptr || dz != nullptr))
    return PRM_ERR_INVALID_ARG;
  if (dy == nullptr && (desc->pre_weight != nullptr || desc->scale != nullptr || desc->shift != nullptr))
    return PRM_ERR_INVALID_ARG;
  if (desc->post_weight != nullptr && (dpost == nullptr || stats == nullptr)) return PRM_ERR_INVALID_ARG;
  if ((desc->gate != nullptr && dgate == nullptr) || (desc->pre_weight != nullptr && dpre == nullptr) ||
      (desc->scale != nullptr && dscale == nullptr) || (desc->shift != nullptr && dshift == nullptr))
    return PRM_ERR_INVALID_ARG;
  if (!aligned_to(stats, 16) || !aligned_to(workspace, 16)) return PRM_ERR_ALIGNMENT;
  const NormGradSpace sp = space(*desc);
  if (sp.mod + sp.w > 0 && (workspace == nullptr || workspace_bytes < sp.mod + sp.w)) return PRM_ERR_WORKSPACE;
  const BlockDevice* dev;
  if ((rc = block_device(&dev)) != PRM_OK) return rc;

  const void* rows[9] = {dy, dr, r, z, dx, dz, dgate, dscale, dshift};
  const bool vec = norm_aligned(*desc, rows, 9) && aligned_to(dpost, 16) && aligned_to(dpre, 16);
  bool ring = true;
  for (int i = 0; i < 6; ++i) ring = ring && aligned_to(rows[i], 16);
  const bool mod = desc->gate != nullptr || desc->scale != nullptr || desc->shift != nullptr;
  const bool w = desc->post_weight != nullptr || desc->pre_weight != nullptr;
  const NormShape s =
      grad_shape(desc->d, row_bytes(*desc, dy != nullptr, dr != nullptr, z != nullptr, stats != nullptr),
                 (dy != nullptr ? 2 : 0) + (dr != nullptr) + (z != nullptr), vec, ring, w, mod);
  const void* present[SUM_COUNT] = {desc->gate, desc->scale, desc->shift, desc->post_weight, desc->pre_weight};
  for (int k = 0; k < SUM_COUNT; ++k) p.has[k] = present[k] != nullptr;
  if (p.n.rows / NORM_CTAS > (int64_t(1) << 30)) return PRM_ERR_UNSUPPORTED;
  p.n.tpr = s.tpr;
  p.groups = s.groups;
  p.stages = s.stages;
  p.sample_rows = mod ? p.n.rps : p.n.rows;
  const int64_t at_once = s.half ? NORM_CTAS : NORM_CTAS / 2;
  p.ctas = std::min<int64_t>(at_once, (p.n.rows + s.groups * s.rows - 1) / (s.groups * s.rows));
  p.partial_mod = static_cast<float*>(workspace);
  p.partial_w = reinterpret_cast<float*>(static_cast<char*>(workspace) + sp.mod);
  p.err = dev->d_err;
  const NormGradArgs a{dy, dr, r, z, stats, dx, dz, dpost, dgate, dpre, dscale, dshift};
  cudaError_t e = cudaErrorInvalidValue;
  norm_types(desc->stream_dtype, desc->block_dtype, [&](auto rt, auto bt) {
    e = norm_grad_launch<decltype(rt), decltype(bt)>(p, s, a, static_cast<cudaStream_t>(stream));
  });
  return e == cudaSuccess ? PRM_OK : PRM_ERR_CUDA;
}
