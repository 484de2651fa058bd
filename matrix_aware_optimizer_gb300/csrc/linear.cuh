// The linear layer's product for few tokens (linear_skinny.cu).
#pragma once

#include "attn.cuh"
#include "ffn.cuh"

namespace prm {

// How D^T (rows x tokens) is cut: tokens of a CTA, CTAs of a cluster that
// share a sum, and whether it pays over the larger tiles.
struct SkinnyPlan {
  int cols, parts;
  bool two;  // CTAs of half an SM's shared memory
  bool use;
};
SkinnyPlan skinny_plan(int64_t tokens, int64_t rows, int64_t k, int num_sms);

// y[token][row] = act(sum over k of a[row][k] b[token][k] + bias[row]) + residual.
struct SkinnyCall {
  const void* a;       // rows x k, or (a_mn) k x rows; contiguous
  const void* b;       // tokens x k, row pitch ldb
  int64_t ldb, tokens, rows, k;
  int a_mn;
  const float* bias;
  const void* residual;
  int64_t ld_residual;
  void* y;
  float* pre;
  int act, dtype;
  bool wide;           // y and residual are fp32
  int* err;
};
cudaError_t skinny_product(const SkinnyPlan& s, const SkinnyCall& c, cudaStream_t stream);

// Map of a row-major rows x cols matrix of 16-bit elements with row pitch ld:
// boxes of box_rows x 64 elements, in the 128-byte swizzle.
bool encode_box(CUtensorMap* map, const void* base, int dtype, int64_t rows, int64_t cols, int64_t ld, int box_rows);

}  // namespace prm
