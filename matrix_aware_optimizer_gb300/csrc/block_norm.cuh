// Shared by the two passes of the norms around a block: launch geometry,
// element mapping and row reductions.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "blocks.cuh"

namespace prm {

constexpr int NORM_MAX_D = 8192;

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

// Eight elements at p as fp32 pairs.
__device__ __forceinline__ F8 load_f8(const float* p) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2*>(p)[0], b = reinterpret_cast<const ulonglong2*>(p)[1];
  return {{a.x, a.y, b.x, b.y}};
}
template <typename T>
__device__ __forceinline__ F8 load_f8(const T* p) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  F8 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<T>(w[i]);
    o.p[i] = f2_pack(f.x, f.y);
  }
  return o;
}
// p[0], p[step], ..., zero from `left` elements on.
template <typename T>
__device__ __forceinline__ F8 gather_f8(const T* p, int left, int step) {
  F8 o;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int a = 2 * k * step, b = a + step;
    o.p[k] = f2_pack(a < left ? to_f32(p[a]) : 0.f, b < left ? to_f32(p[b]) : 0.f);
  }
  return o;
}
template <int ACCESS, typename T>
__device__ __forceinline__ F8 read8(const T* p, int left, int step) {
  if constexpr (ACCESS == VEC) return load_f8(p);
  else return gather_f8(p, left, step);
}
template <int ACCESS, typename T>
__device__ __forceinline__ void write8(T* p, int left, int step, const F8& v) {
  float o[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = f2_unpack(v.p[k]);
    o[2 * k] = f.x;
    o[2 * k + 1] = f.y;
  }
  if constexpr (ACCESS == VEC) {
    Raw8<T> raw;
    raw.set(o);
    raw.store(p);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e * step < left) p[e * step] = from_f32<T>(o[e]);
  }
}

// Threads per CTA that a kernel is compiled for: rows of up to 2048, 5120 and
// 8192 elements.
__host__ __device__ constexpr int norm_threads(int size) { return size == 0 ? 256 : size == 1 ? 320 : 512; }

// Vectors of 8 elements per thread.
__host__ __device__ constexpr int norm_vectors(int size) { return size == 0 ? 1 : 2; }

// Sums of two values per row over the row's threads, R rows at a time. With
// each exchange half the lanes go on with one half of the values (6 shuffles
// for four values instead of 20); rows of more than a warp meet at a named
// barrier of their own, and each warp adds the warps' totals. `turn`
// alternates between two scratch rows, so one barrier per call is enough.
template <int SIZE, int R>
__device__ __forceinline__ void row_sums(float (&a)[R][2], int tpr, int group, float (&scratch)[2][128], int& turn) {
  const int lane = threadIdx.x & 31;
  if (SIZE == 0 && tpr < 32) {
    for (int o = tpr / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        a[i][0] += __shfl_xor_sync(0xffffffffu, a[i][0], o);
        a[i][1] += __shfl_xor_sync(0xffffffffu, a[i][1], o);
      }
    return;
  }
  constexpr int VALUES = 2 * R;
  constexpr int SPAN = 32 / VALUES;  // lanes that carry one value in the end
  float t;
  const bool low = lane < 16;
  if constexpr (R == 2) {
    const float k0 = (low ? a[0][0] : a[R - 1][0]) + __shfl_xor_sync(0xffffffffu, low ? a[R - 1][0] : a[0][0], 16);
    const float k1 = (low ? a[0][1] : a[R - 1][1]) + __shfl_xor_sync(0xffffffffu, low ? a[R - 1][1] : a[0][1], 16);
    const bool even = (lane & 8) == 0;
    t = (even ? k0 : k1) + __shfl_xor_sync(0xffffffffu, even ? k1 : k0, 8);
  } else {
    t = (low ? a[0][0] : a[0][1]) + __shfl_xor_sync(0xffffffffu, low ? a[0][1] : a[0][0], 16);
  }
#pragma unroll
  for (int o = SPAN / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  int from = SPAN;  // lane distance of the values
  if (SIZE > 0 || tpr > 32) {
    float* s = scratch[turn];
    turn ^= 1;
    if ((lane & (SPAN - 1)) == 0) s[(threadIdx.x >> 5) * VALUES + lane / SPAN] = t;
    named_barrier_sync(1 + group, tpr);
    constexpr int MOST_WARPS = norm_threads(SIZE) / 32;
    const int warps = tpr >> 5;
    s += group * warps * VALUES;
    t = 0.f;
#pragma unroll
    for (int k = 0; k < (MOST_WARPS + SPAN - 1) / SPAN; ++k) {
      const int w = lane / VALUES + k * SPAN;
      if (w < warps) t += s[w * VALUES + lane % VALUES];
    }
#pragma unroll
    for (int o = 16; o >= VALUES; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    from = 1;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    a[i][0] = __shfl_sync(0xffffffffu, t, 2 * i * from);
    a[i][1] = __shfl_sync(0xffffffffu, t, (2 * i + 1) * from);
  }
}

template <int R>
__device__ __forceinline__ void join_halves(const uint64_t (&part)[R][2], float (&sums)[R][2]) {
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 f = f2_unpack(part[i][k]);
      sums[i][k] = f.x + f.y;
    }
}

// Geometry of a ring kernel for rows of d elements whose `arrays` arrays take
// row_bytes in all.
struct NormShape {
  int size;          // see norm_threads
  int access;
  int tpr, groups;   // threads per row, groups of rows at once
  int rows;          // rows per group and step
  int stages;
  int threads;
  bool half;         // two CTAs share an SM
  size_t smem;
};
constexpr int MAX_STAGES = 8;
constexpr uint64_t NORM_WAIT_NS = 2000000000ull;

// `behind(threads, groups, nv, direct)`: bytes of shared memory behind the
// ring. `ring`: the arrays start on 16 bytes; `vec`: and so does every row.
template <typename F>
inline NormShape norm_shape(int64_t d, size_t row_bytes, int arrays, bool vec, bool ring, F&& behind) {
  NormShape s{};
  s.size = d <= 2048 ? 0 : d <= 5120 ? 1 : 2;
  const int nv = norm_vectors(s.size);
  const int vectors = static_cast<int>((d + 8 * nv - 1) / (8 * nv));
  if (vectors <= 32) {
    s.tpr = 2;
    while (s.tpr < vectors) s.tpr *= 2;
  } else {
    s.tpr = (vectors + 31) / 32 * 32;
  }
  s.groups = s.size == 2 ? 1 : std::max(1, norm_threads(s.size) / s.tpr);
  s.threads = s.tpr * s.groups;
  const size_t extra = behind(s.size, s.threads, s.groups, false);
  s.access = vec ? VEC : ELEM;
  // two stages at least, in half an SM's shared memory, else in all of it,
  // else one stage
  const size_t half = 110 * 1024, whole = 220 * 1024;
  const struct {
    int rows, stages;
    size_t room;
  } tries[5] = {{2, 2, half}, {1, 2, half}, {2, 2, whole}, {1, 2, whole}, {1, 1, whole}};
  for (int k = s.size == 0 ? 0 : s.size == 1 ? 2 : 3; ring && k < 5; ++k) {
    s.rows = tries[k].rows;
    const size_t stage = row_bytes * s.groups * s.rows + (vec ? 0 : 32 * arrays);
    s.stages =
        extra < tries[k].room ? static_cast<int>(std::min<size_t>((tries[k].room - extra) / stage, MAX_STAGES)) : 0;
    s.smem = stage * s.stages + extra;
    s.half = tries[k].room == half;
    if (s.stages >= tries[k].stages && (vec || s.rows == 1)) return s;
  }
  s.access = DIRECT;
  s.rows = 1;
  s.stages = 0;
  s.smem = behind(s.size, s.threads, s.groups, true);
  s.half = s.size == 0 && s.smem <= half;
  return s;
}

// Sets a kernel up once per device for what norm_shape may ask of it.
template <typename K>
inline cudaError_t norm_setup(K kernel, std::atomic<bool> (&set)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (set[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess) set[dev].store(true, std::memory_order_relaxed);
  return e;
}

// Two CTAs on each of the 152 SMs; also the bound that sizes the backward
// pass's workspace.
constexpr int64_t NORM_CTAS = 304;

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
