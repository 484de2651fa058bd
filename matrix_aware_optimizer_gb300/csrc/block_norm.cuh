// Shared by the two passes of the norms around a block: launch geometry,
// element mapping and row reductions.
#pragma once

#include "blocks.cuh"

namespace prm {

// A row of d elements is held by `tpr` threads (a power of two), `nv`
// 8-element vectors each. Short rows share a warp (no barrier in their
// reductions), longer ones take a CTA of their own. Rows off the vector path
// keep one vector per thread: their loads are single elements.
struct NormShape {
  int tpr;
  int nv;      // 1 or 2
  bool multi;  // a row spans the CTA
};
constexpr int NORM_MAX_D = 8192;
constexpr int NORM_WARP_CTA = 128;  // threads per CTA of rows that fit a warp

inline NormShape norm_shape(int64_t d, bool vec) {
  const int nv = vec && d > 256 ? 2 : 1;
  int tpr = 2;
  while (static_cast<int64_t>(tpr) * 8 * nv < d) tpr *= 2;
  return {tpr, nv, tpr > 32};
}
constexpr int norm_threads(bool vec, bool multi) { return !multi ? NORM_WARP_CTA : vec ? 512 : 1024; }

struct NormParams {
  int64_t rows, rps;
  int d;
  int tpr;
  int layer;
  float alpha, eps, inv_d;
  const float* post;
  const float* pre;
  const void* gate;
  const void* scale;
  const void* shift;
  int64_t gate_ld, scale_ld, shift_ld;
};

// Element e of this thread's vector v: contiguous vectors where rows are
// 16-byte aligned, else strided by the row's thread count (coalesced).
template <bool VEC>
__device__ __forceinline__ int norm_index(int v, int e, int tid, int tpr) {
  return VEC ? (v * tpr + tid) * 8 + e : (v * 8 + e) * tpr + tid;
}

template <typename T, int NV, bool VEC>
struct NormRow {
  Raw8<T> raw[NV];
  float val[VEC ? 1 : 8 * NV];

  __device__ __forceinline__ void load(const T* row, int d, int tid, int tpr) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if constexpr (VEC) {
        const int i = norm_index<true>(v, 0, tid, tpr);
        if (i < d) raw[v].load(row + i);
        else raw[v].zero();
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = norm_index<false>(v, e, tid, tpr);
          val[8 * v + e] = i < d ? to_f32(row[i]) : 0.f;
        }
      }
    }
  }
  __device__ __forceinline__ void get(int v, float (&o)[8]) const {
    if constexpr (VEC) {
      raw[v].get(o);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = val[8 * v + e];
    }
  }
};

// One vector of a per-column array (a gain, or a sample's gate, scale or
// shift), re-read from L1 / L2.
template <typename T, bool VEC>
__device__ __forceinline__ void norm_param(const T* p, int v, int d, int tid, int tpr, float (&o)[8]) {
  if constexpr (VEC) {
    const int i = norm_index<true>(v, 0, tid, tpr);
    Raw8<T> r;
    if (i < d) r.load_cached(p + i);
    else r.zero();
    r.get(o);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = norm_index<false>(v, e, tid, tpr);
      o[e] = i < d ? to_f32(p[i]) : 0.f;
    }
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void norm_store(T* row, int v, int d, int tid, int tpr, const float (&o)[8]) {
  if constexpr (VEC) {
    const int i = norm_index<true>(v, 0, tid, tpr);
    if (i < d) {
      Raw8<T> r;
      r.set(o);
      r.store(row + i);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = norm_index<false>(v, e, tid, tpr);
      if (i < d) row[i] = from_f32<T>(o[e]);
    }
  }
}

// Whether element e of vector v lies inside the row.
template <bool VEC>
__device__ __forceinline__ bool norm_inside(int v, int e, int d, int tid, int tpr) {
  return norm_index<VEC>(v, VEC ? 0 : e, tid, tpr) < d;
}

// Sum of two values over a row's threads, the same in every one of them.
// `turn` alternates between two scratch rows, so one barrier per reduction
// is enough (a row is rewritten only after the next reduction's barrier).
template <bool MULTI>
__device__ __forceinline__ float2 norm_reduce(float a, float b, int tpr, float2* scratch, int& turn) {
  if constexpr (!MULTI) {
    for (int o = tpr / 2; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    return make_float2(a, b);
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    float2* s = scratch + 32 * turn;
    turn ^= 1;
    const int warps = tpr / 32;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 t = make_float2(0.f, 0.f);
    for (int w = 0; w < warps; ++w) {
      t.x += s[w].x;
      t.y += s[w].y;
    }
    return t;
  }
}

// Runs f with (stream type, block type) tags for the supported pairs.
template <typename F>
inline bool norm_types(int stream_dtype, int block_dtype, F&& f) {
  if (stream_dtype == PRM_FP32 && block_dtype == PRM_FP32) return f(float{}, float{}), true;
  if (stream_dtype == PRM_FP32 && block_dtype == PRM_BF16) return f(float{}, __nv_bfloat16{}), true;
  if (stream_dtype == PRM_FP32 && block_dtype == PRM_FP16) return f(float{}, __half{}), true;
  if (stream_dtype == PRM_BF16 && block_dtype == PRM_BF16) return f(__nv_bfloat16{}, __nv_bfloat16{}), true;
  if (stream_dtype == PRM_FP16 && block_dtype == PRM_FP16) return f(__half{}, __half{}), true;
  return false;
}

// Shared argument checks of the two passes; fills the kernel parameters.
int norm_check(const prm_block_norm_desc* desc, NormParams* p);
// Vector path: every row of every array starts on 16 bytes.
bool norm_aligned(const prm_block_norm_desc& desc, const void* const* rows, int count);

}  // namespace prm
