// Forward pass of the norms around a transformer block, one pass over the
// rows:
//   P = N(z) post (or z),  r = alpha x + gate_b P,  y = N(r) pre (1 + scale_b) + shift_b
// with N the root-mean-square or the layer norm. Bound by memory: x, z, r
// and y move once. Each row stays in the registers of its threads between
// the reductions; the deviation of the layer norm is summed from v - mean in
// a second reduction over the same registers, so that a large mean costs no
// digits.
//
// One row per CTA (several per CTA where a row fits a warp) and as many CTAs
// per SM as registers allow: the chain load, reduce, store of one row hides
// behind those of the others. The backward pass's ring of shared-memory
// stages with two CTAs per SM was slower here (8191 x 5120 bf16 with both
// gains 127 us, this form 70; 16384 x 4096 fp32 220 us, 126).
//
// 32 x 1024 x 2048, layer norm with modulation, fp32 stream and bf16 block:
// 134 us, 6.0 TB/s (89 % of the copy rate); 12 x 256 fp32: 2.6 us on the device,
// where the call's host time of 18 counts.
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
  if (c->rows / c->rows_per_sample > 0x7fffffff || c->rows > 0xffffffffll) return PRM_ERR_UNSUPPORTED;
  // the forward pass has a CTA for each row that takes more than a warp
  if (c->rows > 0x7fffffff && c->d > 256) return PRM_ERR_UNSUPPORTED;
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

constexpr int FWD_WARP_CTA = 128;  // threads per CTA of rows that fit a warp

// Threads and 8-element vectors per thread of a row.
struct NormFwdShape {
  int tpr, nv;
  bool multi;  // a row has a CTA of its own
};
// Two vectors per thread, but one in layer norms of up to 2048 elements: with
// one more reduction, more threads per row pay (32 x 1024 x 2048 modulated:
// 135 us against 153).
NormFwdShape fwd_shape(int64_t d, bool vec, bool layer) {
  const int vectors = static_cast<int>((d + 7) / 8);
  NormFwdShape s{2, 1, false};
  if (vectors <= 32 || (vectors <= 64 && vec)) {
    s.nv = vectors <= 32 ? 1 : 2;
    while (s.tpr * s.nv < vectors) s.tpr *= 2;
    return s;
  }
  s.nv = (layer && d <= 2048) || !vec ? 1 : 2;
  if (vectors > 512) s.nv = 2;
  s.tpr = ((vectors + s.nv - 1) / s.nv + 31) / 32 * 32;
  s.multi = true;
  return s;
}

// Sum over a row's threads, the same in every one of them. `turn` alternates
// between two scratch rows, so one barrier per reduction is enough.
template <bool MULTI>
__device__ __forceinline__ float row_sum(float a, int tpr, float (&scratch)[2][32], int& turn) {
  if constexpr (!MULTI) {
    for (int o = tpr / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    float* s = scratch[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = a;
    __syncthreads();
    a = 0.f;
    for (int w = 0; w < tpr >> 5; w += 4) {  // (entries behind the last warp's stay zero)
      const float4 q = *reinterpret_cast<const float4*>(s + w);
      a += (q.x + q.y) + (q.z + q.w);
    }
    return a;
  }
}

// A row's vectors as loaded: all loads go out before the first value is used.
template <typename T, int NV, bool VEC_>
struct RowLoad {
  Raw8<T> raw[VEC_ ? NV : 1];
  F8 val[VEC_ ? 1 : NV];
  __device__ __forceinline__ void load(const T* row, const int (&col)[NV], const int (&left)[NV], int step) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if constexpr (VEC_) {
        if (left[v] > 0) raw[v].load(row + col[v]);
        else raw[v].zero();
      } else {
        val[v] = gather_f8(row + col[v], left[v], step);
      }
    }
  }
  __device__ __forceinline__ F8 get(int v) const {
    if constexpr (VEC_) {
      float f[8];
      raw[v].get(f);
      return {{f2_pack(f[0], f[1]), f2_pack(f[2], f[3]), f2_pack(f[4], f[5]), f2_pack(f[6], f[7])}};
    } else {
      return val[v];
    }
  }
};
// A per-column array is read through the read-only path, which the compiler
// may move ahead of the stores of r.
template <typename T, bool VEC_>
__device__ __forceinline__ F8 column8(const T* p, int left, int step) {
  if constexpr (VEC_) {
    Raw8<T> raw;
    raw.load_cached(p);
    float f[8];
    raw.get(f);
    return {{f2_pack(f[0], f[1]), f2_pack(f[2], f[3]), f2_pack(f[4], f[5]), f2_pack(f[6], f[7])}};
  } else {
    return gather_f8(p, left, step);
  }
}

template <typename RT, typename BT, int NV, bool VEC_, bool MULTI>
__global__ void __launch_bounds__(MULTI ? 512 : FWD_WARP_CTA)
    norm_forward_kernel(const __grid_constant__ NormParams p, const RT* x, const BT* __restrict__ z, RT* r,
                        BT* __restrict__ y, float4* __restrict__ stats) {
  __shared__ __align__(16) float scratch[2][32];
  int turn = 0;
  if (MULTI && threadIdx.x < 64) (&scratch[0][0])[threadIdx.x] = 0.f;
  if (MULTI) __syncthreads();
  const int tpr = p.tpr, d = p.d;
  const int tid = MULTI ? threadIdx.x : threadIdx.x & (tpr - 1);
  const int64_t row = MULTI ? static_cast<int64_t>(blockIdx.x)
                            : static_cast<int64_t>(blockIdx.x) * (FWD_WARP_CTA / tpr) + threadIdx.x / tpr;
  const bool live = MULTI || row < p.rows;  // a dead row's threads still take part in the shuffles
  int left[NV];
  int col[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    col[v] = VEC_ ? (v * tpr + tid) * 8 : v * 8 * tpr + tid;
    left[v] = live ? d - col[v] : 0;
  }
  pdl_wait();
  pdl_launch_dependents();
  const int64_t at = live ? row * d : 0;
  RowLoad<RT, NV, VEC_> xr;
  RowLoad<BT, NV, VEC_> zr;
  xr.load(x + at, col, left, tpr);
  if (z != nullptr) zr.load(z + at, col, left, tpr);
  F8 rv[NV];
  const bool mod = p.gate != nullptr || p.scale != nullptr || p.shift != nullptr;
  // (32-bit division: a 64-bit one was a fifth of the kernel's instructions)
  const int64_t sample = live && mod ? static_cast<uint32_t>(row) / static_cast<uint32_t>(p.rps) : 0;
  // mean (layer norm only) and reciprocal deviation; the row comes back centred
  auto statistics = [&](float& mean, float& rs) {
    if (p.layer) {
      uint64_t s = 0;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (left[v] > 0) s = f2_add(s, rv[v].p[k]);
      const float2 f = f2_unpack(s);
      mean = row_sum<MULTI>(f.x + f.y, tpr, scratch, turn) * p.inv_d;
      const uint64_t m = f2_pack(-mean, -mean);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (left[v] <= 0) continue;
          rv[v].p[k] = f2_add(rv[v].p[k], m);
          if constexpr (!VEC_) {  // strided vectors can straddle the row's end
            const float2 c = f2_unpack(rv[v].p[k]);
            rv[v].p[k] = f2_pack(2 * k * tpr < left[v] ? c.x : 0.f, (2 * k + 1) * tpr < left[v] ? c.y : 0.f);
          }
        }
    }
    uint64_t s = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (left[v] > 0) s = f2_fma(rv[v].p[k], rv[v].p[k], s);
    const float2 f = f2_unpack(s);
    rs = rsqrtf(row_sum<MULTI>(f.x + f.y, tpr, scratch, turn) * p.inv_d + p.eps);
  };

  float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
  if (z != nullptr) {
#pragma unroll
    for (int v = 0; v < NV; ++v) rv[v] = zr.get(v);
    if (p.post != nullptr) statistics(st.z, st.w);
    const uint64_t s = f2_pack(st.w, st.w), alpha = f2_pack(p.alpha, p.alpha);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (left[v] <= 0) continue;
      if (p.post != nullptr) {
        const F8 w = column8<float, VEC_>(p.post + col[v], left[v], tpr);
#pragma unroll
        for (int k = 0; k < 4; ++k) rv[v].p[k] = f2_mul(f2_mul(rv[v].p[k], s), w.p[k]);
      }
      if (p.gate != nullptr) {
        const F8 g = column8<BT, VEC_>(static_cast<const BT*>(p.gate) + sample * p.gate_ld + col[v], left[v], tpr);
#pragma unroll
        for (int k = 0; k < 4; ++k) rv[v].p[k] = f2_mul(rv[v].p[k], g.p[k]);
      }
      const F8 xv = xr.get(v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint64_t q = f2_fma(alpha, xv.p[k], rv[v].p[k]);
        if constexpr (sizeof(RT) == 2) {  // the norm reads r as it is stored
          const float2 f = f2_unpack(q);
          const float2 t = unpack2<RT>(pack2<RT>(f.x, f.y));
          q = f2_pack(t.x, t.y);
        }
        rv[v].p[k] = q;
      }
      write8<VEC_ ? VEC : DIRECT>(r + at + col[v], left[v], tpr, rv[v]);
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) rv[v] = xr.get(v);
  }
  if (y != nullptr) {
    statistics(st.x, st.y);
    const uint64_t s = f2_pack(st.y, st.y), one = f2_pack(1.f, 1.f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (left[v] <= 0) continue;
      F8 o;
#pragma unroll
      for (int k = 0; k < 4; ++k) o.p[k] = f2_mul(rv[v].p[k], s);
      if (p.pre != nullptr) {
        const F8 w = column8<float, VEC_>(p.pre + col[v], left[v], tpr);
#pragma unroll
        for (int k = 0; k < 4; ++k) o.p[k] = f2_mul(o.p[k], w.p[k]);
      }
      if (p.scale != nullptr) {
        const F8 w = column8<BT, VEC_>(static_cast<const BT*>(p.scale) + sample * p.scale_ld + col[v], left[v], tpr);
#pragma unroll
        for (int k = 0; k < 4; ++k) o.p[k] = f2_mul(o.p[k], f2_add(one, w.p[k]));
      }
      if (p.shift != nullptr) {
        const F8 w = column8<BT, VEC_>(static_cast<const BT*>(p.shift) + sample * p.shift_ld + col[v], left[v], tpr);
#pragma unroll
        for (int k = 0; k < 4; ++k) o.p[k] = f2_add(o.p[k], w.p[k]);
      }
      write8<VEC_ ? VEC : DIRECT>(y + at + col[v], left[v], tpr, o);
    }
  }
  if (stats != nullptr && live && tid == 0) stats[row] = st;
}

template <typename RT, typename BT, int NV, bool VEC_, bool MULTI>
cudaError_t launch_forward(const NormParams& p, const void* x, const void* z, void* r, void* y, float* stats,
                           cudaStream_t stream) {
  const int threads = MULTI ? p.tpr : FWD_WARP_CTA;
  const int64_t per_cta = MULTI ? 1 : FWD_WARP_CTA / p.tpr;
  const int64_t blocks = (p.rows + per_cta - 1) / per_cta;
  return launch_dependent(norm_forward_kernel<RT, BT, NV, VEC_, MULTI>, dim3(static_cast<unsigned>(blocks)),
                          dim3(threads), 0, stream, p, static_cast<const RT*>(x), static_cast<const BT*>(z),
                          static_cast<RT*>(r), static_cast<BT*>(y), reinterpret_cast<float4*>(stats));
}

template <typename RT, typename BT, bool VEC_>
cudaError_t launch_shape(NormParams p, const void* x, const void* z, void* r, void* y, float* stats,
                         cudaStream_t stream) {
  const NormFwdShape s = fwd_shape(p.d, VEC_, p.layer != 0);
  p.tpr = s.tpr;
  if (s.multi)
    return s.nv == 1 ? launch_forward<RT, BT, 1, VEC_, true>(p, x, z, r, y, stats, stream)
                     : launch_forward<RT, BT, 2, VEC_, true>(p, x, z, r, y, stats, stream);
  if constexpr (VEC_) {
    if (s.nv == 2) return launch_forward<RT, BT, 2, VEC_, false>(p, x, z, r, y, stats, stream);
  }
  return launch_forward<RT, BT, 1, VEC_, false>(p, x, z, r, y, stats, stream);
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
