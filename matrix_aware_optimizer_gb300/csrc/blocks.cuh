// Shared by the transformer-block operators (ffn*.cu, block_norm*.cu,
// embedding.cu): element conversion, 8-element vector access, programmatic
// dependent launches, 2-D TMA of CTA pairs and the per-device state.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "prm_blocks.h"
#include "ptx.cuh"

namespace prm {

// Per-device state of the block operators, set up by the first call there:
// SM count and the device error word of the bounded waits.
struct BlockDevice {
  int num_sms = 0;
  int* d_err = nullptr;
  bool ready = false;
};
int block_device(const BlockDevice** out);

inline bool is_dtype(int t) { return t == PRM_FP32 || t == PRM_BF16 || t == PRM_FP16; }
inline size_t dtype_bytes(int t) { return t == PRM_FP32 ? 4 : 2; }
inline bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t round_up(size_t n, size_t a) { return (n + a - 1) / a * a; }

// ------------------------------------------------------------ conversions
template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) {
  return __half2float(v);
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  return pack2_bf16(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  return pack2_f16(lo, hi);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Eight consecutive elements in raw form: a load keeps no more registers
// than the bytes it brought until the values are used.
template <typename T>
struct Raw8 {
  uint4 a;
  __device__ __forceinline__ void load(const T* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void load_cached(const T* p) { a = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<T>(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
  }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = a; }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void load_cached(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
};

// Eight fp32 values as four packed pairs: sm_100 multiplies and adds two fp32
// values per instruction (each half rounded as the scalar operation).
struct F8 {
  uint64_t p[4];
};
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f2_unpack(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F8 f8_zero() { return {{0, 0, 0, 0}}; }

// ------------------------------------------- programmatic dependent launch
// A kernel launched with launch_dependent() may start while its predecessor
// on the stream drains; it calls pdl_wait() before its first access to
// memory that another kernel writes or reads.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... KArgs, typename... Args>
inline cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                                    Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// ------------------------------------------------------------- bulk copies
// Contiguous copy of `bytes` (a multiple of 16; both addresses 16-byte
// aligned) from global to this CTA's shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// How a thread's eight elements of a row lie: consecutive in the stage (VEC),
// strided by the row's thread count in the stage (ELEM: d % 8 != 0, whose
// rows start anywhere), or strided in memory (DIRECT: no ring).
enum Access { VEC, ELEM, DIRECT };

// Bulk copies of n elements from any element of a tensor that itself starts
// on 16 bytes, to shared memory at the same offset from a 16-byte boundary.
// ring_bytes: what the copy brings (its start rounded down, its end up, but
// not past the last whole 16 bytes before `end`, the tensor's end);
// ring_tail: the elements behind those, stored by this thread. Any n elements
// that end less than 16 bytes before the tensor can have some.
template <typename T>
__device__ __forceinline__ uint32_t ring_bytes(const T* src, uint32_t n, const T* end) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(src) & ~uintptr_t(15);
  const uintptr_t last = reinterpret_cast<uintptr_t>(end) & ~uintptr_t(15);
  uintptr_t hi = (reinterpret_cast<uintptr_t>(src + n) + 15) & ~uintptr_t(15);
  hi = hi < last ? hi : last;
  return hi > lo ? static_cast<uint32_t>(hi - lo) : 0u;
}
template <typename T>
__device__ __forceinline__ void ring_tail(uint8_t* dst, const T* src, uint32_t n, const T* end) {
  const T* last = reinterpret_cast<const T*>(reinterpret_cast<uintptr_t>(end) & ~uintptr_t(15));
  const T* lo = reinterpret_cast<const T*>(reinterpret_cast<uintptr_t>(src) & ~uintptr_t(15));
  T* out = reinterpret_cast<T*>(dst);
  for (const T* p = last > src ? last : src; p < src + n; ++p) out[p - lo] = *p;
}
template <typename T>
__device__ __forceinline__ void ring_load(uint8_t* dst, const T* src, uint32_t bytes, uint64_t* bar) {
  if (bytes > 0)
    bulk_load(dst, reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(src) & ~uintptr_t(15)), bytes, bar);
}
// Where an ELEM row that starts at src lies in its stage region.
template <typename T>
__device__ __forceinline__ uint32_t ring_offset(const T* src) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src) & 15u);
}

// -------------------------------------------------------- TMA of CTA pairs
// 2-D tile load into this CTA's shared memory whose completion is counted on
// the mbarrier at `bar_cluster_addr`, which may belong to the peer CTA.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* tm, uint32_t bar_cluster_addr, int x,
                                                 int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar_cluster_addr), "r"(x), "r"(y)
      : "memory");
}

// 2-D tile store of a box staged in shared memory, in the thread's current
// bulk async-group. Elements outside the tensor are not written.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* tm, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tm)),
               "r"(smem_u32(src)), "r"(x), "r"(y)
               : "memory");
}

// Quotient of n < 2^31 by a divisor of 1 .. 2^31: floor(n m / 2^(32 + s)) with
// s = ceil(log2 d) - 1 and m = floor(2^(32 + s) / d) + 1 (Granlund and
// Montgomery, 1994: exact as m d - 2^(32 + s) <= d <= 2^(s + 1)).
struct Divisor {
  uint32_t d, m, s;
  static Divisor of(uint32_t d) {
    uint32_t s = 0;
    while ((uint64_t(1) << (s + 1)) < d) ++s;
    return {d, d == 1 ? 0u : static_cast<uint32_t>((uint64_t(1) << (32 + s)) / d + 1), s};
  }
  __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return d == 1 ? n : __umulhi(n, m) >> s; }
};

}  // namespace prm
