// Activations of the gated feed-forward block, in fp32, and its kernels for a
// few tokens.
#pragma once

#include <atomic>
#include <type_traits>

#include "blocks.cuh"

namespace prm {

// 1 / (1 + exp(-v)).
__device__ __forceinline__ float ffn_sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

constexpr float FFN_SQRT_2_PI = 0.7978845608028654f;      // sqrt(2 / pi)
constexpr float FFN_SQRT_HALF = 0.7071067811865476f;
constexpr float FFN_INV_SQRT_2PI = 0.3989422804014327f;

// (1 + tanh(t)) / 2 = 1 / (1 + exp(-2 t)), so the tanh form of gelu is
// g sigmoid(2 t): no cancellation for negative g.
template <int ACT>
__device__ __forceinline__ float ffn_act(float g) {
  if constexpr (ACT == PRM_ACT_SILU) return g * ffn_sigmoid(g);
  if constexpr (ACT == PRM_ACT_GELU) return 0.5f * g * (1.f + erff(g * FFN_SQRT_HALF));
  return g * ffn_sigmoid(2.f * FFN_SQRT_2_PI * fmaf(0.044715f * g * g, g, g));
}

// act(g) and act'(g).
template <int ACT>
__device__ __forceinline__ void ffn_act_grad(float g, float* a, float* da) {
  if constexpr (ACT == PRM_ACT_SILU) {
    const float s = ffn_sigmoid(g);
    *a = g * s;
    *da = s * fmaf(g, 1.f - s, 1.f);
  } else if constexpr (ACT == PRM_ACT_GELU) {
    const float c = 0.5f * (1.f + erff(g * FFN_SQRT_HALF));
    *a = g * c;
    *da = fmaf(g * FFN_INV_SQRT_2PI, __expf(-0.5f * g * g), c);
  } else {
    const float t2 = 2.f * FFN_SQRT_2_PI * fmaf(0.044715f * g * g, g, g);
    const float s = ffn_sigmoid(t2);
    *a = g * s;
    *da = fmaf(g * s * (1.f - s), 2.f * FFN_SQRT_2_PI * fmaf(3.f * 0.044715f * g, g, 1.f), s);
  }
}

// Forward pass on CUDA cores for up to FFN_FEW_TOKENS tokens: h and y, and g
// and u in the tensor-core kernels' packed layout where gu is not NULL.
// CUDA cores up to 4 tokens, up to 8 with small weights: at d 2048, f 8192 and
// 4 tokens 26 us against 41 on the tensor cores, with 8 tokens 51 against 42; at
// d 512, f 1536 and 8 tokens 8.2 against 19.
constexpr int FFN_FEW_TOKENS = 8;
inline bool ffn_few(int64_t tokens, int64_t d, int64_t f) {
  return tokens <= 4 || (tokens <= FFN_FEW_TOKENS && d * f <= (int64_t(1) << 21));
}
cudaError_t ffn_few_forward(const void* x, int64_t ldx, const void* w_gate, const void* w_up, const void* w_down,
                            void* h, uint4* gu, void* y, int tokens, int d, int f, int act, int dtype,
                            cudaStream_t stream);

}  // namespace prm
