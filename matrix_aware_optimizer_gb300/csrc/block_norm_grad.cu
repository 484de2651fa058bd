// Backward pass of the norms around a transformer block. With n = (r - m_r) s_r,
// q = (z - m_z) s_z, P = q post (or z), and dr arriving from r's later uses:
//   dn  = dy (1 + scale_b) pre
//   D   = dr + s_r (dn - n mean(dn n) [- mean(dn)])         (gradient of r in all)
//   dx  = alpha D,   dP = gate_b D,   dq = dP post
//   dz  = s_z (dq - q mean(dq q) [- mean(dq)])              (dP without post)
//   dshift_b = sum dy, dscale_b = sum dy n pre, dgate_b = sum D P,
//   dpre = sum dy (1 + scale_b) n, dpost = sum dP q         (over rows)
// the bracketed terms for the layer norm only. Bound by memory: dy, dr, r and
// z are read once, dx and dz written once. A CTA walks the rows of one part
// of a sample (or several whole samples) with a fixed thread per column, so
// the column sums need no atomics: each thread adds to its own fp32 columns
// in shared memory, and the parts' sums are added in order by a second
// kernel.
#include <algorithm>

#include "block_norm.cuh"

namespace prm {
namespace {

constexpr int SUM_GATE = 0, SUM_SCALE = 1, SUM_SHIFT = 2, SUM_POST = 3, SUM_PRE = 4, SUM_COUNT = 5;

struct NormGradParams {
  NormParams n;
  int64_t samples;      // rows that share modulation (1 without any)
  int64_t sample_rows;
  int64_t parts;        // CTAs per sample; 1: a CTA takes per_cta whole samples
  int64_t part_rows;
  int64_t per_cta;
  int64_t ctas;
  int groups;           // rows a CTA works on at once (1 when a row spans it)
  int slot[SUM_COUNT];  // index of each sum in shared memory, or -1
  int sums;
  float* partial_mod;   // [ctas][3][d] (parts > 1)
  float* partial_w;     // [ctas][2][d]
};

template <typename RT, typename BT, int NV, bool VEC, bool MULTI>
__global__ void __launch_bounds__(norm_threads(VEC, MULTI))
    norm_backward_kernel(const __grid_constant__ NormGradParams p, const BT* dy, const RT* dr,
                         const RT* __restrict__ r, const BT* __restrict__ z, const float4* __restrict__ stats,
                         RT* dx, BT* dz, BT* __restrict__ dgate, BT* __restrict__ dscale, BT* __restrict__ dshift) {
  extern __shared__ float4 sums4[];  // [sums][groups][2][NV * tpr]: the halves of this thread's vectors apart
  __shared__ float2 scratch[MULTI ? 64 : 1];
  int turn = 0;
  const int tpr = p.n.tpr, d = p.n.d;
  const int tid = MULTI ? threadIdx.x : threadIdx.x & (tpr - 1);
  const int group = MULTI ? 0 : threadIdx.x / tpr;
  const int groups = MULTI ? 1 : p.groups;
  const int width = NV * tpr;
  auto sum_at = [&](int which, int v, int half) -> float4& {
    return sums4[((p.slot[which] * groups + group) * 2 + half) * width + v * tpr + tid];
  };
  auto add_sum = [&](int which, int v, const float(&o)[8]) {
    float4& lo = sum_at(which, v, 0);
    float4& hi = sum_at(which, v, 1);
    lo = make_float4(lo.x + o[0], lo.y + o[1], lo.z + o[2], lo.w + o[3]);
    hi = make_float4(hi.x + o[4], hi.y + o[5], hi.z + o[6], hi.w + o[7]);
  };
  auto clear = [&](int which) {
    if (p.slot[which] < 0) return;
#pragma unroll
    for (int v = 0; v < NV; ++v) sum_at(which, v, 0) = sum_at(which, v, 1) = make_float4(0.f, 0.f, 0.f, 0.f);
  };
  // The sum over the CTA's row groups of one column vector, in group order.
  auto total = [&](int which, int v, float(&o)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.f;
    for (int g = 0; g < groups; ++g) {
      const int base = (p.slot[which] * groups + g) * 2 * width + v * tpr + tid;
      const float4 lo = sums4[base], hi = sums4[base + width];
      o[0] += lo.x, o[1] += lo.y, o[2] += lo.z, o[3] += lo.w;
      o[4] += hi.x, o[5] += hi.y, o[6] += hi.z, o[7] += hi.w;
    }
  };

  for (int k = 0; k < SUM_COUNT; ++k) clear(k);
  pdl_wait();
  pdl_launch_dependents();
  const int64_t cta = blockIdx.x;
  const int64_t first_sample = p.parts > 1 ? cta / p.parts : cta * p.per_cta;
  const int64_t last_sample = p.parts > 1 ? first_sample + 1 : min(p.samples, first_sample + p.per_cta);
  const int64_t part = p.parts > 1 ? cta % p.parts : 0;
  for (int64_t sample = first_sample; sample < last_sample; ++sample) {
    const int64_t row0 = sample * p.sample_rows + part * p.part_rows;
    const int64_t row1 = min((sample + 1) * p.sample_rows, row0 + p.part_rows);
    for (int64_t base = row0; base < row1; base += groups) {
      const int64_t row = base + group;
      const bool live = row < row1;
      const int64_t at = live ? row * d : 0;
      const int dd = live ? d : 0;
      NormRow<BT, NV, VEC> dyr, zr;
      NormRow<RT, NV, VEC> drr, rr;
      if (dy != nullptr) {
        dyr.load(dy + at, dd, tid, tpr);
        rr.load(r + at, dd, tid, tpr);
      }
      if (dr != nullptr) drr.load(dr + at, dd, tid, tpr);
      if (z != nullptr) zr.load(z + at, dd, tid, tpr);
      const float4 st = live && stats != nullptr ? stats[row] : make_float4(0.f, 0.f, 0.f, 0.f);

      float D[NV][8];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (dr != nullptr) {
          drr.get(v, D[v]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) D[v][e] = 0.f;
        }
      }
      if (dy != nullptr) {
        float dn[NV][8], nn[NV][8];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float rv[8];
          dyr.get(v, dn[v]);
          rr.get(v, rv);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            nn[v][e] = norm_inside<VEC>(v, e, dd, tid, tpr) ? (rv[e] - st.x) * st.y : 0.f;
          if (p.slot[SUM_SHIFT] >= 0) add_sum(SUM_SHIFT, v, dn[v]);
          float w[8];
          if (p.n.pre != nullptr) norm_param<float, VEC>(p.n.pre, v, dd, tid, tpr, w);
          if (p.n.scale != nullptr) {
            float o[8], sc[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = dn[v][e] * nn[v][e] * (p.n.pre != nullptr ? w[e] : 1.f);
            add_sum(SUM_SCALE, v, o);
            norm_param<BT, VEC>(static_cast<const BT*>(p.n.scale) + sample * p.n.scale_ld, v, dd, tid, tpr, sc);
#pragma unroll
            for (int e = 0; e < 8; ++e) dn[v][e] = fmaf(dn[v][e], sc[e], dn[v][e]);
          }
          if (p.n.pre != nullptr) {
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = dn[v][e] * nn[v][e];
            add_sum(SUM_PRE, v, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) dn[v][e] *= w[e];
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            s1 = fmaf(dn[v][e], nn[v][e], s1);
            s2 += dn[v][e];
          }
        }
        const float2 t = norm_reduce<MULTI>(s1, s2, tpr, scratch, turn);
        const float m1 = t.x * p.n.inv_d, m2 = p.n.layer ? t.y * p.n.inv_d : 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) D[v][e] = fmaf(st.y, dn[v][e] - fmaf(nn[v][e], m1, m2), D[v][e]);
      }
      if (dx != nullptr && live) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = p.n.alpha * D[v][e];
          norm_store<RT, VEC>(dx + at, v, dd, tid, tpr, o);
        }
      }
      if (z == nullptr) continue;
      float s1 = 0.f, s2 = 0.f;
      float q[NV][8];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        zr.get(v, q[v]);
        float w[8];
        if (p.n.post != nullptr) {
          norm_param<float, VEC>(p.n.post, v, dd, tid, tpr, w);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            q[v][e] = norm_inside<VEC>(v, e, dd, tid, tpr) ? (q[v][e] - st.z) * st.w : 0.f;
        }
        if (p.n.gate != nullptr) {
          float o[8], g[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = D[v][e] * q[v][e] * (p.n.post != nullptr ? w[e] : 1.f);
          add_sum(SUM_GATE, v, o);
          norm_param<BT, VEC>(static_cast<const BT*>(p.n.gate) + sample * p.n.gate_ld, v, dd, tid, tpr, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) D[v][e] *= g[e];
        }
        if (p.n.post != nullptr) {
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = D[v][e] * q[v][e];
          add_sum(SUM_POST, v, o);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            D[v][e] *= w[e];
            s1 = fmaf(D[v][e], q[v][e], s1);
            s2 += D[v][e];
          }
        }
      }
      if (p.n.post != nullptr) {
        const float2 t = norm_reduce<MULTI>(s1, s2, tpr, scratch, turn);
        const float m1 = t.x * p.n.inv_d, m2 = p.n.layer ? t.y * p.n.inv_d : 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) D[v][e] = st.w * (D[v][e] - fmaf(q[v][e], m1, m2));
      }
      if (dz != nullptr && live) {
#pragma unroll
        for (int v = 0; v < NV; ++v) norm_store<BT, VEC>(dz + at, v, dd, tid, tpr, D[v]);
      }
    }
    // the sample's (or its part's) modulation sums
    BT* const mod_out[3] = {dgate, dscale, dshift};
    bool any = false;
#pragma unroll
    for (int k = 0; k < 3; ++k) any = any || p.slot[k] >= 0;
    if (any) {
      if (!MULTI) __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          if (p.slot[k] < 0) continue;
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            float o[8];
            total(k, v, o);
            if (p.parts > 1)
              norm_store<float, VEC>(p.partial_mod + (cta * 3 + k) * static_cast<int64_t>(d), v, d, tid, tpr, o);
            else
              norm_store<BT, VEC>(mod_out[k] + sample * static_cast<int64_t>(d), v, d, tid, tpr, o);
          }
        }
      }
      if (!MULTI) __syncthreads();
#pragma unroll
      for (int k = 0; k < 3; ++k) clear(k);
    }
  }
  if (!MULTI) __syncthreads();
  if (group == 0) {
#pragma unroll
    for (int k = SUM_POST; k < SUM_COUNT; ++k) {
      if (p.slot[k] < 0) continue;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float o[8];
        total(k, v, o);
        norm_store<float, VEC>(p.partial_w + (cta * 2 + k - SUM_POST) * static_cast<int64_t>(d), v, d, tid, tpr, o);
      }
    }
  }
}

// One output row of column sums: `count` partial rows, `stride` floats apart.
struct NormJoin {
  const float* from;
  int64_t stride, count;
};

// out[row][column] = sum of the row's partial sums. A block takes 32 columns;
// its 8 warps add every eighth partial row, and warp 0 adds their totals.
template <typename BT>
__global__ void __launch_bounds__(256) norm_join_kernel(const __grid_constant__ NormGradParams p, BT* dgate, BT* dscale,
                                                        BT* dshift, float* dpost, float* dpre) {
  __shared__ float part[8][33];
  pdl_wait();
  pdl_launch_dependents();
  const int d = p.n.d;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const int64_t mod_rows = p.parts > 1 ? 3 * p.samples : 0;
  const int64_t job = blockIdx.y;
  NormJoin j{};
  int k;
  int64_t sample = 0;
  if (job < mod_rows) {
    k = static_cast<int>(job % 3);
    sample = job / 3;
    j = {p.partial_mod + (sample * p.parts * 3 + k) * static_cast<int64_t>(d), 3 * static_cast<int64_t>(d), p.parts};
  } else {
    k = SUM_POST + static_cast<int>(job - mod_rows);
    j = {p.partial_w + (k - SUM_POST) * static_cast<int64_t>(d), 2 * static_cast<int64_t>(d), p.ctas};
  }
  if (p.slot[k] < 0) return;
  float s = 0.f;
  if (col < d) {
#pragma unroll 8
    for (int64_t i = warp; i < j.count; i += 8) s += j.from[i * j.stride + col];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || col >= d) return;
  for (int w = 1; w < 8; ++w) s += part[w][lane];
  if (k < 3) {
    BT* out = k == SUM_GATE ? dgate : k == SUM_SCALE ? dscale : dshift;
    out[sample * d + col] = from_f32<BT>(s);
  } else {
    (k == SUM_POST ? dpost : dpre)[col] = s;
  }
}

struct NormGradArgs {
  const void *dy, *dr, *r, *z;
  const float* stats;
  void *dx, *dz;
  float* dpost;
  void* dgate;
  float* dpre;
  void *dscale, *dshift;
};

size_t sums_bytes(const NormShape& s, int groups, int sums) {
  return static_cast<size_t>(sums) * groups * 2 * s.nv * s.tpr * sizeof(float4);
}

template <typename RT, typename BT, int NV, bool VEC, bool MULTI>
cudaError_t launch_backward(const NormGradParams& p, const NormGradArgs& a, cudaStream_t stream) {
  const NormShape s = norm_shape(p.n.d, VEC);
  const size_t smem = sums_bytes(s, p.groups, p.sums);
  auto kernel = norm_backward_kernel<RT, BT, NV, VEC, MULTI>;
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = launch_dependent(
      kernel, dim3(static_cast<unsigned>(p.ctas)), dim3(MULTI ? s.tpr : NORM_WARP_CTA), smem, stream, p,
      static_cast<const BT*>(a.dy), static_cast<const RT*>(a.dr), static_cast<const RT*>(a.r),
      static_cast<const BT*>(a.z), reinterpret_cast<const float4*>(a.stats), static_cast<RT*>(a.dx),
      static_cast<BT*>(a.dz), static_cast<BT*>(a.dgate), static_cast<BT*>(a.dscale), static_cast<BT*>(a.dshift));
  if (e != cudaSuccess) return e;
  const bool mod = p.parts > 1 && (p.slot[0] >= 0 || p.slot[1] >= 0 || p.slot[2] >= 0);
  const bool w = p.slot[SUM_POST] >= 0 || p.slot[SUM_PRE] >= 0;
  if (!mod && !w) return cudaSuccess;
  const int64_t jobs = (p.parts > 1 ? 3 * p.samples : 0) + (w ? 2 : 0);
  return launch_dependent(norm_join_kernel<BT>, dim3((p.n.d + 31) / 32, static_cast<unsigned>(jobs)), dim3(256), 0,
                          stream, p, static_cast<BT*>(a.dgate), static_cast<BT*>(a.dscale), static_cast<BT*>(a.dshift),
                          a.dpost, a.dpre);
}

template <typename RT, typename BT, bool VEC>
cudaError_t launch_shape(const NormGradParams& p, const NormGradArgs& a, cudaStream_t stream) {
  const NormShape s = norm_shape(p.n.d, VEC);
  if constexpr (VEC) {
    if (s.nv == 2)
      return s.multi ? launch_backward<RT, BT, 2, VEC, true>(p, a, stream)
                     : launch_backward<RT, BT, 2, VEC, false>(p, a, stream);
    return launch_backward<RT, BT, 1, VEC, false>(p, a, stream);
  } else {
    return s.multi ? launch_backward<RT, BT, 1, VEC, true>(p, a, stream)
                   : launch_backward<RT, BT, 1, VEC, false>(p, a, stream);
  }
}

// How the rows are spread over CTAs. Every CTA's column sums go through the
// workspace, so there are a few CTAs per SM and no more.
constexpr int64_t NORM_GRAD_CTAS = 152 * 8;

int plan(const prm_block_norm_desc* desc, bool vec, NormGradParams* p, size_t* bytes) {
  const int rc = norm_check(desc, &p->n);
  if (rc != PRM_OK) return rc;
  const NormShape s = norm_shape(desc->d, vec);
  p->n.tpr = s.tpr;
  const bool mod = desc->gate != nullptr || desc->scale != nullptr || desc->shift != nullptr;
  p->sample_rows = mod ? p->n.rps : p->n.rows;
  p->samples = p->n.rows == 0 ? 0 : p->n.rows / p->sample_rows;
  p->groups = s.multi ? 1 : NORM_WARP_CTA / s.tpr;
  const bool has[SUM_COUNT] = {desc->gate != nullptr, desc->scale != nullptr, desc->shift != nullptr,
                               desc->post_weight != nullptr, desc->pre_weight != nullptr};
  p->sums = 0;
  for (int k = 0; k < SUM_COUNT; ++k) p->slot[k] = has[k] ? p->sums++ : -1;
  p->parts = 1;
  p->per_cta = 1;
  p->ctas = 0;
  p->part_rows = p->sample_rows;
  *bytes = 0;
  if (p->samples == 0) return PRM_OK;
  const int64_t most = (p->sample_rows + p->groups - 1) / p->groups;
  p->parts = std::min<int64_t>(most, std::max<int64_t>(1, NORM_GRAD_CTAS / p->samples));
  if (p->parts > 1) {
    p->part_rows = (p->sample_rows + p->parts - 1) / p->parts;
    p->part_rows = (p->part_rows + p->groups - 1) / p->groups * p->groups;
    p->parts = (p->sample_rows + p->part_rows - 1) / p->part_rows;
  }
  if (p->parts > 1) {
    p->ctas = p->samples * p->parts;
  } else {
    p->part_rows = p->sample_rows;
    p->per_cta = (p->samples + NORM_GRAD_CTAS - 1) / NORM_GRAD_CTAS;
    p->ctas = (p->samples + p->per_cta - 1) / p->per_cta;
  }
  const size_t row = static_cast<size_t>(p->ctas) * p->n.d * sizeof(float);
  const size_t mod_bytes = mod && p->parts > 1 ? round_up(3 * row, 256) : 0;
  const size_t w_bytes = has[SUM_POST] || has[SUM_PRE] ? 2 * row : 0;
  p->partial_mod = nullptr;
  p->partial_w = reinterpret_cast<float*>(mod_bytes);  // offset, until the workspace is known
  *bytes = mod_bytes + w_bytes;
  return PRM_OK;
}

}  // namespace
}  // namespace prm

extern "C" int prm_block_norm_workspace(const prm_block_norm_desc* desc, size_t* bytes) {
  if (bytes == nullptr) return PRM_ERR_INVALID_ARG;
  prm::NormGradParams p;
  size_t vec = 0, scalar = 0;
  int rc = prm::plan(desc, true, &p, &vec);
  if (rc == PRM_OK) rc = prm::plan(desc, false, &p, &scalar);
  *bytes = vec > scalar ? vec : scalar;  // which path runs depends on the pointers
  return rc;
}

extern "C" int prm_block_norm_backward(const prm_block_norm_desc* desc, const void* dy, const void* dr, const void* r,
                                       const void* z, const float* stats, void* dx, void* dz, float* dpost,
                                       void* dgate, float* dpre, void* dscale, void* dshift, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  using namespace prm;
  NormGradParams p;
  size_t need = 0;
  int rc = norm_check(desc, &p.n);
  if (rc != PRM_OK) return rc;
  const void* rows[9] = {dy, dr, r, z, dx, dz, dgate, dscale, dshift};
  const bool vec = norm_aligned(*desc, rows, 9) && aligned_to(dpost, 16) && aligned_to(dpre, 16);
  rc = plan(desc, vec, &p, &need);
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
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return PRM_ERR_WORKSPACE;
  const size_t w_offset = reinterpret_cast<size_t>(p.partial_w);
  p.partial_mod = static_cast<float*>(workspace);
  p.partial_w = reinterpret_cast<float*>(static_cast<char*>(workspace) + w_offset);
  const NormGradArgs a{dy, dr, r, z, stats, dx, dz, dpost, dgate, dpre, dscale, dshift};
  cudaError_t e = cudaErrorInvalidValue;
  norm_types(desc->stream_dtype, desc->block_dtype, [&](auto rt, auto bt) {
    using RT = decltype(rt);
    using BT = decltype(bt);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    e = vec ? launch_shape<RT, BT, true>(p, a, st) : launch_shape<RT, BT, false>(p, a, st);
  });
  return e == cudaSuccess ? PRM_OK : PRM_ERR_CUDA;
}
