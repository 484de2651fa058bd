// Dropout whose mask is a function of the element's index: y = residual +
// (kept ? x / (1 - p) : 0), forward and (without residual) backward.
//
// The random words are those of the ten-round Philox 4x32 generator (Salmon,
// Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011):
// a counter is a block of four words, so any element's word is computed on its
// own and nothing is stored between the passes. A thread takes eight elements,
// two blocks. A dropped element is left out, not multiplied by zero: an
// infinity there leaves no NaN behind.
//
// 32768 x 2048 bf16: 62.7 us with a residual (6.4 TB/s, 95 % of the copy rate)
// and 62 without, where the bytes would take 40: there the generator's 40 wide
// multiplications per eight elements bound it.
#include "blocks.cuh"
#include "prm_attention.h"

namespace prm {
namespace {

constexpr int DROP_THREADS = 256;

struct DropParams {
  const void* x;
  const void* residual;
  void* y;
  int64_t n;
  uint64_t offset;
  const uint64_t* seed_device;  // where not NULL the round keys come from what it holds
  uint32_t keys[20];            // of the ten rounds
  uint32_t threshold;  // a smaller word drops its element
  int none;            // p is 1: nothing is kept
  float scale;
};

constexpr uint32_t KEY_STEP0 = 0x9E3779B9u, KEY_STEP1 = 0xBB67AE85u;

// key(r): round r's two key words.
template <typename Key>
__device__ __forceinline__ uint4 philox10(uint64_t counter, Key key) {
  uint32_t c0 = static_cast<uint32_t>(counter), c1 = static_cast<uint32_t>(counter >> 32), c2 = 0, c3 = 0;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    const uint2 k = key(r);
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k.x;
    c1 = static_cast<uint32_t>(b);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k.y;
    c3 = static_cast<uint32_t>(a);
  }
  return make_uint4(c0, c1, c2, c3);
}

// VEC: every pointer 16-byte aligned; the elements behind the last eight are
// taken one by one all the same.
template <typename T, typename R, bool RES, bool VEC>
__global__ void __launch_bounds__(DROP_THREADS) dropout_kernel(const __grid_constant__ DropParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * DROP_THREADS + threadIdx.x) * 8;
  if (i0 >= p.n) return;
  const T* x = static_cast<const T*>(p.x) + i0;
  const R* res = static_cast<const R*>(p.residual) + i0;
  R* y = static_cast<R*>(p.y) + i0;
  const bool whole = VEC && i0 + 8 <= p.n;
  Raw8<T> xv;
  Raw8<R> rv;
  if (whole) {
    xv.load(x);
    if (RES) rv.load(res);
  }
  const uint64_t block = p.offset + static_cast<uint64_t>(i0) / 4;
  uint4 a, b;
  if (p.seed_device == nullptr) {
    auto key = [&](int r) { return make_uint2(p.keys[2 * r], p.keys[2 * r + 1]); };
    a = philox10(block, key);
    b = philox10(block + 1, key);
  } else {
    const uint64_t seed = *p.seed_device;
    const uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
    auto key = [&](int r) { return make_uint2(k0 + r * KEY_STEP0, k1 + r * KEY_STEP1); };
    a = philox10(block, key);
    b = philox10(block + 1, key);
  }
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (whole) {
    float v[8], r[8];
    xv.get(v);
    if (RES) rv.get(r);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool kept = w[e] >= p.threshold && !p.none;
      v[e] = RES ? (kept ? fmaf(v[e], p.scale, r[e]) : r[e]) : (kept ? v[e] * p.scale : 0.f);
    }
    rv.set(v);
    rv.store(y);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (i0 + e >= p.n) break;
      const bool kept = w[e] >= p.threshold && !p.none;
      const float base = RES ? to_f32(res[e]) : 0.f;
      y[e] = from_f32<R>(kept ? (RES ? fmaf(to_f32(x[e]), p.scale, base) : to_f32(x[e]) * p.scale) : base);
    }
  }
}

template <typename T, typename R, bool RES>
cudaError_t launch(const DropParams& p, cudaStream_t stream) {
  const int64_t blocks = (p.n + 8 * DROP_THREADS - 1) / (8 * DROP_THREADS);
  const bool vec = aligned_to(p.x, 16) && aligned_to(p.residual, 16) && aligned_to(p.y, 16);
  return launch_dependent(vec ? dropout_kernel<T, R, RES, true> : dropout_kernel<T, R, RES, false>,
                          dim3(static_cast<unsigned>(blocks)), dim3(DROP_THREADS), 0, stream, p);
}

template <typename T>
cudaError_t launch(const DropParams& p, cudaStream_t stream) {
  return p.residual != nullptr ? launch<T, T, true>(p, stream) : launch<T, T, false>(p, stream);
}

}  // namespace
}  // namespace prm

extern "C" int prm_dropout(const void* x, int dtype, const void* residual, void* y, int y_dtype, int64_t n, double p,
                           uint64_t seed, const uint64_t* seed_device, uint64_t offset, void* stream) {
  using namespace prm;
  if (!is_dtype(dtype) || !is_dtype(y_dtype) || n < 0 || !(p >= 0.0 && p <= 1.0)) return PRM_ERR_INVALID_ARG;
  // a 16-bit x joins a residual stream in fp32, whose gradient goes back to 16 bits
  if (y_dtype != dtype && (residual != nullptr ? y_dtype : dtype) != PRM_FP32) return PRM_ERR_INVALID_ARG;
  if (n == 0) return PRM_OK;
  if (x == nullptr || y == nullptr) return PRM_ERR_INVALID_ARG;
  if (n > (int64_t(1) << 41)) return PRM_ERR_UNSUPPORTED;  // blocks of a launch: 31 bits
  const BlockDevice* dev;
  const int rc = block_device(&dev);
  if (rc != PRM_OK) return rc;
  const double limit = p * 4294967296.0 + 0.5;
  DropParams q{};
  q.x = x;
  q.residual = residual;
  q.y = y;
  q.n = n;
  q.offset = offset;
  q.seed_device = seed_device;
  for (uint32_t r = 0; r < 10; ++r) {
    q.keys[2 * r] = static_cast<uint32_t>(seed) + r * KEY_STEP0;
    q.keys[2 * r + 1] = static_cast<uint32_t>(seed >> 32) + r * KEY_STEP1;
  }
  q.none = limit >= 4294967296.0;
  q.threshold = q.none ? 0u : static_cast<uint32_t>(limit);
  q.scale = p < 1.0 ? static_cast<float>(1.0 / (1.0 - p)) : 0.f;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == y_dtype)
    e = dtype == PRM_FP32 ? launch<float>(q, st) : dtype == PRM_BF16 ? launch<__nv_bfloat16>(q, st) : launch<__half>(q, st);
  else if (residual != nullptr)
    e = dtype == PRM_BF16 ? launch<__nv_bfloat16, float, true>(q, st) : launch<__half, float, true>(q, st);
  else
    e = y_dtype == PRM_BF16 ? launch<float, __nv_bfloat16, false>(q, st) : launch<float, __half, false>(q, st);
  return e == cudaSuccess ? PRM_OK : PRM_ERR_CUDA;
}
