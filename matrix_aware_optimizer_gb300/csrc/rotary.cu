// Rotary positions: pairs (a, b) of a head's first `dim` elements turn by
// angle = position * frequency, (a cos - b sin, b cos + a sin) times an
// amplitude; the elements behind them are copied.
//
// Frequencies come as 64-bit fractions of a turn per position, so that the
// angle modulo one turn is a 64-bit integer product without any rounding; it
// is rounded once, to fp32, where its sine and cosine are taken (2^-25 of a
// turn at most). A CTA takes a few tokens: it forms each token's sines and
// cosines once, in shared memory, for all heads, while the first vectors are on
// their way. Bound by memory: x is read once and y written once. 4 x 4096
// tokens of 32 heads of 128, bf16: 48 us either way, 5.6 TB/s (82 % of the copy
// rate); 16 tokens of 20 heads 2.3 us, the launch.
#include <algorithm>
#include <type_traits>

#include "blocks.cuh"
#include "prm_attention.h"

namespace prm {
namespace {

constexpr int ROT_THREADS = 256;
constexpr int ROT_AHEAD = 2;       // units in flight per thread
constexpr int ROT_TABLE = 2048;    // sines and cosines of a CTA
constexpr int ROT_TOKENS = 64;     // tokens of a CTA at most

struct RotParams {
  const void* x;
  void* y;
  const void* positions;
  const uint64_t* turns;
  int64_t x_sample, x_token, x_head, y_sample, y_token, y_head, position_sample, position_token;
  int64_t rows;            // samples * tokens
  Divisor tokens;          // of a sample
  Divisor token_units, head_units;
  int pairs;               // dim / 2
  int turned_units;        // units of a head with pairs; copies behind them
  int cta_tokens;
  int position_bytes;
  float amplitude, sign;
};

// N consecutive elements in raw form.
template <typename T, int N>
struct Elements {
  using Word = typename std::conditional<
      sizeof(T) * N >= 16, uint4,
      typename std::conditional<sizeof(T) * N == 8, uint2,
                                typename std::conditional<sizeof(T) * N == 4, uint32_t, uint16_t>::type>::type>::type;
  static constexpr int WORDS = sizeof(T) * N > 16 ? sizeof(T) * N / 16 : 1;
  union {
    Word w[WORDS];
    T e[N];
  };
  __device__ __forceinline__ Elements() {}
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = __ldcs(reinterpret_cast<const Word*>(p) + i);
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) reinterpret_cast<Word*>(p)[i] = w[i];
  }
};

// A unit is N elements, or 2 N where its pairs lie apart: HALF, and
// interleaved pairs of single elements (N = 1).
template <typename T, int N, bool HALF>
__global__ void __launch_bounds__(ROT_THREADS) rotary_kernel(const __grid_constant__ RotParams p) {
  __shared__ float2 table[ROT_TABLE];
  constexpr bool APART = HALF || N == 1;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.cta_tokens;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(p.cta_tokens), p.rows - first));
  const int units = tokens * static_cast<int>(p.token_units.d);
  const int apart = HALF ? p.pairs : 1;  // elements between the two of a pair that lies apart

  struct Unit {
    int table;  // first sine and cosine, or -1 for a copy
    int64_t y;
    Elements<T, N> a, b;
  };
  auto fetch = [&](int u, Unit& v) {
    const uint32_t tok = p.token_units.quotient(u);
    const uint32_t in_token = u - tok * p.token_units.d;
    const uint32_t head = p.head_units.quotient(in_token);
    const int at = static_cast<int>(in_token - head * p.head_units.d);
    const uint64_t row = static_cast<uint64_t>(first) + tok;
    const int64_t sample = row >> 31 == 0 ? p.tokens.quotient(static_cast<uint32_t>(row)) : row / p.tokens.d;
    const int64_t token = static_cast<int64_t>(row) - sample * p.tokens.d;
    int64_t element;
    if (at < p.turned_units) {
      v.table = static_cast<int>(tok) * p.pairs + (HALF || N == 1 ? at * N : at * (N / 2));
      element = HALF ? at * N : N == 1 ? at * 2 : at * N;
    } else {
      v.table = -1;
      element = 2 * p.pairs + (at - p.turned_units) * N;
    }
    const T* x = static_cast<const T*>(p.x) + sample * p.x_sample + token * p.x_token + head * p.x_head + element;
    v.y = sample * p.y_sample + token * p.y_token + head * p.y_head + element;
    v.a.load(x);
    if (APART && v.table >= 0) v.b.load(x + apart);
  };
  auto finish = [&](Unit& v) {
    T* y = static_cast<T*>(p.y) + v.y;
    if (v.table >= 0) {
      if constexpr (APART) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float2 cs = table[v.table + e];
          const float a = to_f32(v.a.e[e]), b = to_f32(v.b.e[e]);
          v.a.e[e] = from_f32<T>(fmaf(a, cs.x, -b * cs.y));
          v.b.e[e] = from_f32<T>(fmaf(b, cs.x, a * cs.y));
        }
        v.b.store(y + apart);
      } else {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const float2 cs = table[v.table + e / 2];
          const float a = to_f32(v.a.e[e]), b = to_f32(v.a.e[e + 1]);
          v.a.e[e] = from_f32<T>(fmaf(a, cs.x, -b * cs.y));
          v.a.e[e + 1] = from_f32<T>(fmaf(b, cs.x, a * cs.y));
        }
      }
    }
    v.a.store(y);
  };

  Unit unit[ROT_AHEAD];
  int u = threadIdx.x;
#pragma unroll
  for (int k = 0; k < ROT_AHEAD; ++k)
    if (u + k * ROT_THREADS < units) fetch(u + k * ROT_THREADS, unit[k]);

  for (int i = threadIdx.x; i < tokens * p.pairs; i += ROT_THREADS) {
    const int tok = i / p.pairs, pair = i - tok * p.pairs;
    const int64_t row = first + tok, sample = row / p.tokens.d;
    const int64_t at = sample * p.position_sample + (row - sample * p.tokens.d) * p.position_token;
    const int64_t position = p.position_bytes == 8 ? static_cast<const int64_t*>(p.positions)[at]
                                                   : static_cast<const int32_t*>(p.positions)[at];
    const int64_t turn = static_cast<int64_t>(static_cast<uint64_t>(position) * p.turns[pair]);  // of 2^64, signed
    float s, c;
    sincospif(__ll2float_rn(turn) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
    table[i] = make_float2(c * p.amplitude, s * p.amplitude * p.sign);
  }
  __syncthreads();

  while (u < units) {
#pragma unroll
    for (int k = 0; k < ROT_AHEAD; ++k)
      if (u + k * ROT_THREADS < units) finish(unit[k]);
    u += ROT_AHEAD * ROT_THREADS;
#pragma unroll
    for (int k = 0; k < ROT_AHEAD; ++k)
      if (u + k * ROT_THREADS < units) fetch(u + k * ROT_THREADS, unit[k]);
  }
}

template <typename T, int N>
cudaError_t launch(const RotParams& p, bool half, unsigned grid, cudaStream_t stream) {
  return launch_dependent(half ? rotary_kernel<T, N, true> : rotary_kernel<T, N, false>, dim3(grid), dim3(ROT_THREADS),
                          0, stream, p);
}

template <typename T>
cudaError_t launch(const RotParams& p, int width, bool half, unsigned grid, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2) {
    if (width == 8) return launch<T, 8>(p, half, grid, stream);
  }
  if (width == 4) return launch<T, 4>(p, half, grid, stream);
  if (width == 2) return launch<T, 2>(p, half, grid, stream);
  return launch<T, 1>(p, half, grid, stream);
}

}  // namespace
}  // namespace prm

extern "C" int prm_rotary(const prm_rotary_desc* d, const void* x, const void* positions, const uint64_t* turns, void* y,
                          void* stream) {
  using namespace prm;
  if (d == nullptr || d->reserved != 0 || !is_dtype(d->dtype) || d->layout < PRM_ROTARY_HALF ||
      d->layout > PRM_ROTARY_INTERLEAVED || (d->position_bytes != 4 && d->position_bytes != 8) ||
      d->samples < 0 || d->tokens < 0 || d->heads < 0 || !(d->amplitude - d->amplitude == 0.f))
    return PRM_ERR_INVALID_ARG;
  if (d->head < 1 || d->dim < 2 || d->dim % 2 != 0 || d->dim > d->head) return PRM_ERR_SHAPE;
  if (d->samples == 0 || d->tokens == 0 || d->heads == 0) return PRM_OK;
  if (x == nullptr || positions == nullptr || turns == nullptr || y == nullptr) return PRM_ERR_INVALID_ARG;
  // units of a CTA's tokens are counted in 31 bits, its sines and cosines lie in shared memory
  if (d->dim > 2 * ROT_TABLE || d->head > (1 << 16) || d->heads > (1 << 14) || d->samples > (int64_t(1) << 40) ||
      d->tokens >= (int64_t(1) << 31) || d->samples > (int64_t(1) << 40) / d->tokens)
    return PRM_ERR_UNSUPPORTED;
  const bool in_place = x == y;
  if (in_place && ((d->samples > 1 && d->x_sample != d->y_sample) || (d->tokens > 1 && d->x_token != d->y_token) ||
                   (d->heads > 1 && d->x_head != d->y_head)))
    return PRM_ERR_INVALID_ARG;
  const BlockDevice* dev;
  const int rc = block_device(&dev);
  if (rc != PRM_OK) return rc;
  RotParams p{};
  p.x_sample = d->samples > 1 ? d->x_sample : 0;  // (the stride of a single sample, token or head is never used)
  p.x_token = d->tokens > 1 ? d->x_token : 0;
  p.x_head = d->heads > 1 ? d->x_head : 0;
  p.y_sample = d->samples > 1 ? d->y_sample : 0;
  p.y_token = d->tokens > 1 ? d->y_token : 0;
  p.y_head = d->heads > 1 ? d->y_head : 0;

  // the widest vectors that pairs, copies, strides and pointers allow
  const bool half = d->layout == PRM_ROTARY_HALF;
  const int64_t size = static_cast<int64_t>(dtype_bytes(d->dtype));
  int width = size == 4 ? 4 : 8;
  auto fits = [&](int w) {
    const int64_t strides[6] = {p.x_sample, p.x_token, p.x_head, p.y_sample, p.y_token, p.y_head};
    for (int64_t s : strides)
      if (s % w != 0) return false;
    return (half ? d->dim / 2 : d->dim) % w == 0 && (d->head - d->dim) % w == 0 && aligned_to(x, w * size) &&
           aligned_to(y, w * size);
  };
  while (width > 1 && !fits(width)) width /= 2;
  const bool apart = half || width == 1;
  p.x = x;
  p.y = y;
  p.positions = positions;
  p.turns = turns;
  p.position_sample = d->position_sample;
  p.position_token = d->position_token;
  p.rows = d->samples * d->tokens;
  p.tokens = Divisor::of(static_cast<uint32_t>(d->tokens));
  p.pairs = static_cast<int>(d->dim / 2);
  p.turned_units = static_cast<int>(d->dim / (apart ? 2 * width : width));
  const int copies = in_place ? 0 : static_cast<int>((d->head - d->dim) / width);
  p.head_units = Divisor::of(p.turned_units + copies);
  p.token_units = Divisor::of(static_cast<uint32_t>(d->heads) * p.head_units.d);
  p.position_bytes = d->position_bytes;
  p.amplitude = d->amplitude;
  p.sign = d->inverse ? -1.f : 1.f;
  // about two rounds of units to a CTA, and all SMs in use before a second round
  const int64_t want = std::max<int64_t>(1, ROT_THREADS * ROT_AHEAD * 2 / p.token_units.d);
  const int64_t fill = std::max<int64_t>(1, p.rows / (4 * dev->num_sms));
  p.cta_tokens = static_cast<int>(std::min<int64_t>({want, fill, ROT_TABLE / p.pairs, ROT_TOKENS}));
  const int64_t grid = (p.rows + p.cta_tokens - 1) / p.cta_tokens;
  if (grid >= (int64_t(1) << 31)) return PRM_ERR_UNSUPPORTED;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned g = static_cast<unsigned>(grid);
  const cudaError_t e = d->dtype == PRM_FP32   ? launch<float>(p, width, half, g, st)
                        : d->dtype == PRM_BF16 ? launch<__nv_bfloat16>(p, width, half, g, st)
                                               : launch<__half>(p, width, half, g, st);
  return e == cudaSuccess ? PRM_OK : PRM_ERR_CUDA;
}
