// Forward pass of the norms around a transformer block, one pass over the
// rows:
//   P = N(z) post (or z),  r = alpha x + gate_b P,  y = N(r) pre (1 + scale_b) + shift_b
// with N the root-mean-square or the layer norm. Bound by memory: x, z, r
// and y move once. Each row stays in the registers of its threads between
// the reductions; the deviation of the layer norm is summed from v - mean in
// a second reduction over the same registers, so that a large mean costs no
// digits.
#include <cmath>

#include "block_norm.cuh"

namespace prm {

int norm_check(const prm_block_norm_desc* c, NormParams* p) {
  if (c == nullptr || c->reserved != 0) return PRM_ERR_INVALID_ARG;
  if (c->kind != PRM_NORM_RMS && c->kind != PRM_NORM_LAYER) return PRM_ERR_INVALID_ARG;
  if (!is_dtype(c->stream_dtype) || !is_dtype(c->block_dtype)) return PRM_ERR_INVALID_ARG;
  if (c->stream_dtype != PRM_FP32 && c->stream_dtype != c->block_dtype) return PRM_ERR_INVALID_ARG;
  if (!std::isfinite(c->alpha) || !std::isfinite(c->eps) || !(c->eps >= 0.f)) return PRM_ERR_INVALID_ARG;
  if (c->rows < 0 || c->d < 1 || c->rows_per_sample < 1 || c->rows % c->rows_per_sample != 0) return PRM_ERR_SHAPE;
  if (c->d > NORM_MAX_D) return PRM_ERR_UNSUPPORTED;
  if (c->rows / c->rows_per_sample > 0x7fffffff || c->rows > (int64_t(1) << 40)) return PRM_ERR_UNSUPPORTED;
  if ((c->gate != nullptr && c->gate_ld < c->d) || (c->scale != nullptr && c->scale_ld < c->d) ||
      (c->shift != nullptr && c->shift_ld < c->d))
    return PRM_ERR_SHAPE;
  p->rows = c->rows;
  p->rps = c->rows_per_sample;
  p->d = static_cast<int>(c->d);
  p->layer = c->kind == PRM_NORM_LAYER;
  p->alpha = c->alpha;
  p->eps = c->eps;
  p->inv_d = 1.f / static_cast<float>(c->d);
  p->post = c->post_weight;
  p->pre = c->pre_weight;
  p->gate = c->gate;
  p->scale = c->scale;
  p->shift = c->shift;
  p->gate_ld = c->gate_ld;
  p->scale_ld = c->scale_ld;
  p->shift_ld = c->shift_ld;
  return PRM_OK;
}

bool norm_aligned(const prm_block_norm_desc& c, const void* const* rows, int count) {
  if (c.d % 8 != 0) return false;
  bool ok = true;
  for (int i = 0; i < count; ++i) ok = ok && aligned_to(rows[i], 16);
  ok = ok && aligned_to(c.post_weight, 16) && aligned_to(c.pre_weight, 16);
  const int64_t unit = 16 / static_cast<int64_t>(dtype_bytes(c.block_dtype));
  const void* mod[3] = {c.gate, c.scale, c.shift};
  const int64_t ld[3] = {c.gate_ld, c.scale_ld, c.shift_ld};
  for (int i = 0; i < 3; ++i) ok = ok && (mod[i] == nullptr || (aligned_to(mod[i], 16) && ld[i] % unit == 0));
  return ok;
}

namespace {

template <typename RT, typename BT, int NV, bool VEC, bool MULTI>
__global__ void __launch_bounds__(norm_threads(VEC, MULTI))
    norm_forward_kernel(const __grid_constant__ NormParams p, const RT* x, const BT* __restrict__ z, RT* r,
                        BT* __restrict__ y, float4* __restrict__ stats) {
  __shared__ float2 scratch[MULTI ? 64 : 1];
  int turn = 0;
  const int tpr = p.tpr, d = p.d;
  const int tid = MULTI ? threadIdx.x : threadIdx.x & (tpr - 1);
  const int64_t row = MULTI ? static_cast<int64_t>(blockIdx.x)
                            : static_cast<int64_t>(blockIdx.x) * (NORM_WARP_CTA / tpr) + threadIdx.x / tpr;
  const bool live = MULTI || row < p.rows;  // a dead row's threads still take part in the shuffles
  const int64_t at = live ? row * d : 0;
  const int dd = live ? d : 0;
  pdl_wait();
  pdl_launch_dependents();
  NormRow<RT, NV, VEC> xr;
  NormRow<BT, NV, VEC> zr;
  xr.load(x + at, dd, tid, tpr);
  if (z != nullptr) zr.load(z + at, dd, tid, tpr);
  const bool mod = p.gate != nullptr || p.scale != nullptr || p.shift != nullptr;
  const int64_t sample = live && mod ? row / p.rps : 0;

  float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
  float rv[NV][8];
  if (z != nullptr) {
    if (p.post != nullptr) {
      if (p.layer) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float zz[8];
          zr.get(v, zz);
#pragma unroll
          for (int e = 0; e < 8; ++e) s += zz[e];
        }
        st.z = norm_reduce<MULTI>(s, 0.f, tpr, scratch, turn).x * p.inv_d;
      }
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float zz[8];
        zr.get(v, zz);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float c = norm_inside<VEC>(v, e, dd, tid, tpr) ? zz[e] - st.z : 0.f;
          s = fmaf(c, c, s);
        }
      }
      st.w = rsqrtf(norm_reduce<MULTI>(s, 0.f, tpr, scratch, turn).x * p.inv_d + p.eps);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float zz[8], xx[8], o[8];
      zr.get(v, zz);
      xr.get(v, xx);
      if (p.post != nullptr) {
        float w[8];
        norm_param<float, VEC>(p.post, v, dd, tid, tpr, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) zz[e] = (zz[e] - st.z) * st.w * w[e];
      }
      if (p.gate != nullptr) {
        float g[8];
        norm_param<BT, VEC>(static_cast<const BT*>(p.gate) + sample * p.gate_ld, v, dd, tid, tpr, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) zz[e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(p.alpha, xx[e], zz[e]);
      norm_store<RT, VEC>(r + at, v, dd, tid, tpr, o);
      // the norm reads r as it is stored
#pragma unroll
      for (int e = 0; e < 8; ++e) rv[v][e] = to_f32(from_f32<RT>(o[e]));
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) xr.get(v, rv[v]);
  }
  if (y == nullptr) {
    if (stats != nullptr && live && tid == 0) stats[row] = st;
    return;
  }

  if (p.layer) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (norm_inside<VEC>(v, e, dd, tid, tpr)) s += rv[v][e];
    st.x = norm_reduce<MULTI>(s, 0.f, tpr, scratch, turn).x * p.inv_d;
  }
  float s = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = norm_inside<VEC>(v, e, dd, tid, tpr) ? rv[v][e] - st.x : 0.f;
      s = fmaf(c, c, s);
    }
  st.y = rsqrtf(norm_reduce<MULTI>(s, 0.f, tpr, scratch, turn).x * p.inv_d + p.eps);
  if (stats != nullptr && live && tid == 0) stats[row] = st;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = (rv[v][e] - st.x) * st.y;
    if (p.pre != nullptr) {
      float w[8];
      norm_param<float, VEC>(p.pre, v, dd, tid, tpr, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] *= w[e];
    }
    if (p.scale != nullptr) {
      float w[8];
      norm_param<BT, VEC>(static_cast<const BT*>(p.scale) + sample * p.scale_ld, v, dd, tid, tpr, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(o[e], w[e], o[e]);
    }
    if (p.shift != nullptr) {
      float w[8];
      norm_param<BT, VEC>(static_cast<const BT*>(p.shift) + sample * p.shift_ld, v, dd, tid, tpr, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] += w[e];
    }
    norm_store<BT, VEC>(y + at, v, dd, tid, tpr, o);
  }
}

template <typename RT, typename BT, int NV, bool VEC, bool MULTI>
cudaError_t launch_forward(const NormParams& p, const void* x, const void* z, void* r, void* y, float* stats,
                           cudaStream_t stream) {
  const int threads = MULTI ? p.tpr : NORM_WARP_CTA;
  const int64_t per_cta = MULTI ? 1 : NORM_WARP_CTA / p.tpr;
  const int64_t blocks = (p.rows + per_cta - 1) / per_cta;
  return launch_dependent(norm_forward_kernel<RT, BT, NV, VEC, MULTI>, dim3(static_cast<unsigned>(blocks)),
                          dim3(threads), 0, stream, p, static_cast<const RT*>(x), static_cast<const BT*>(z),
                          static_cast<RT*>(r), static_cast<BT*>(y), reinterpret_cast<float4*>(stats));
}

template <typename RT, typename BT, bool VEC>
cudaError_t launch_shape(NormParams p, const void* x, const void* z, void* r, void* y, float* stats,
                         cudaStream_t stream) {
  const NormShape s = norm_shape(p.d, VEC);
  p.tpr = s.tpr;
  if constexpr (VEC) {
    if (s.nv == 2)
      return s.multi ? launch_forward<RT, BT, 2, VEC, true>(p, x, z, r, y, stats, stream)
                     : launch_forward<RT, BT, 2, VEC, false>(p, x, z, r, y, stats, stream);
    return launch_forward<RT, BT, 1, VEC, false>(p, x, z, r, y, stats, stream);
  } else {
    return s.multi ? launch_forward<RT, BT, 1, VEC, true>(p, x, z, r, y, stats, stream)
                   : launch_forward<RT, BT, 1, VEC, false>(p, x, z, r, y, stats, stream);
  }
}

}  // namespace
}  // namespace prm

extern "C" int prm_block_norm_forward(const prm_block_norm_desc* desc, const void* x, const void* z, void* r, void* y,
                                      float* stats, void* stream) {
  using namespace prm;
  NormParams p;
  const int rc = norm_check(desc, &p);
  if (rc != PRM_OK) return rc;
  if (p.rows == 0) return PRM_OK;
  if (x == nullptr || (z == nullptr && (y == nullptr || desc->alpha != 1.f || desc->gate != nullptr ||
                                        desc->post_weight != nullptr)) ||
      (z != nullptr && r == nullptr))
    return PRM_ERR_INVALID_ARG;
  if (y == nullptr && (desc->pre_weight != nullptr || desc->scale != nullptr || desc->shift != nullptr))
    return PRM_ERR_INVALID_ARG;
  if (!aligned_to(stats, 16)) return PRM_ERR_ALIGNMENT;
  if (p.rows > 0x7fffffff) return PRM_ERR_UNSUPPORTED;
  const void* rows[4] = {x, z, r, y};
  const bool vec = norm_aligned(*desc, rows, 4);
  cudaError_t e = cudaErrorInvalidValue;
  norm_types(desc->stream_dtype, desc->block_dtype, [&](auto rt, auto bt) {
    using RT = decltype(rt);
    using BT = decltype(bt);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    e = vec ? launch_shape<RT, BT, true>(p, x, z, r, y, stats, st)
            : launch_shape<RT, BT, false>(p, x, z, r, y, stats, st);
  });
  return e == cudaSuccess ? PRM_OK : PRM_ERR_CUDA;
}
