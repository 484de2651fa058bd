// Gated feed-forward block and linear layer for a few tokens (a sampling step): the products
// are matrix-vector products, bound by reading each weight once, and run on
// CUDA cores. A 256-row tensor-core tile would be empty but for these rows.
//
// A warp takes four weight rows (GLU: two features of w_gate and of w_up;
// down projection: four outputs) and all tokens; a lane takes 8 consecutive
// elements of K per step, multiplies them as packed fp32 pairs and adds in
// fp32. Where there are few rows, up to eight warps of a CTA share a row
// along K and add their sums in order through shared memory. The tokens'
// elements come from L1 / L2; a weight vector is unpacked once for all of
// them. The down projection's CTAs start while the first kernel drains and
// load their first weights before they wait for h.
//
// One token at d 2048, f 8192 bf16, weights not in L2: 20.5 us, 4.9 TB/s (72 %
// of the copy rate); 17.2 back to back, where L2 keeps a part of the 101 MB.
// What is left is the start and the end of two short launches. A linear layer
// 2048 -> 6144 for one token: 7.0 us back to back (3.6 TB/s), 12 - 14 with the
// host's call.
#include <algorithm>

#include "ffn.cuh"

namespace prm {
namespace {

constexpr int FEW_THREADS = 256;
constexpr int FEW_WARPS = FEW_THREADS / 32;
constexpr int FEW_ROWS = 4;

struct FewParams {
  const void* x;        // tokens x K, row pitch ldx
  int64_t ldx;
  const void* w[2];     // GLU: w_gate, w_up (rows x K); else w_down
  void* out;            // tokens x rows
  uint4* gu;            // GLU: packed g and u for the backward pass, or NULL
  int tokens, rows, K;
  int split;            // warps that share a row: 1, 2, 4 or 8
  // LINEAR alone (see LinearFew)
  const float* bias = nullptr;
  const void* residual = nullptr;
  int64_t ld_residual = 0;
  float* pre = nullptr;
  bool wide = false;
};

// What the sums become: h, y of the down projection, or a linear layer's y.
constexpr int FEW_GLU = 0, FEW_DOWN = 1, FEW_LINEAR = 2;

template <typename T, int NT, int USE, int ACT>
__global__ void __launch_bounds__(FEW_THREADS, USE == FEW_LINEAR && NT == 1 ? 4 : NT <= 4 ? 2 : 1) ffn_few_kernel(const __grid_constant__ FewParams p) {
  constexpr bool GLU = USE == FEW_GLU;
  __shared__ float part[FEW_WARPS][NT * FEW_ROWS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int piece = warp % p.split;  // this warp's part of K
  const int group = warp / p.split;
  const int64_t first =
      (static_cast<int64_t>(blockIdx.x) * (FEW_WARPS / p.split) + group) * (GLU ? FEW_ROWS / 2 : FEW_ROWS);
  const T* w[FEW_ROWS];
#pragma unroll
  for (int r = 0; r < FEW_ROWS; ++r) {
    // GLU: rows 0, 1 of w_gate and 0, 1 of w_up; a row past the end repeats the last one
    const int64_t row = min(first + (GLU ? (r & 1) : r), static_cast<int64_t>(p.rows) - 1);
    w[r] = static_cast<const T*>(p.w[GLU ? (r >> 1) : 0]) + row * p.K;
  }
  const T* x[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) x[t] = static_cast<const T*>(p.x) + min(t, p.tokens - 1) * p.ldx;

  uint64_t acc[NT][FEW_ROWS];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < FEW_ROWS; ++r) acc[t][r] = 0;
  const int step = p.split * 256;
  const int k0 = (piece * 32 + lane) * 8;
  // steps whose weights are in flight
  constexpr int AHEAD = NT == 1 && USE != FEW_LINEAR ? 4 : 2;
  uint4 wv[AHEAD][FEW_ROWS];
  auto load_w = [&](int k) {
#pragma unroll
    for (int a = 0; a < AHEAD; ++a)
#pragma unroll
      for (int r = 0; r < FEW_ROWS; ++r)
        wv[a][r] = k + a * step < p.K ? __ldcs(reinterpret_cast<const uint4*>(w[r] + k + a * step))
                                      : make_uint4(0, 0, 0, 0);
  };
  if (USE != FEW_DOWN) {
    pdl_wait();  // the weights and x may be the kernels' before this one
    pdl_launch_dependents();
    load_w(k0);
  } else {
    load_w(k0);  // (whatever wrote the weights was waited for by the first kernel)
    pdl_wait();
    pdl_launch_dependents();
  }
  for (int k = k0; k < p.K; k += AHEAD * step) {
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      if (k + a * step >= p.K) break;
      F8 wf[FEW_ROWS];
#pragma unroll
      for (int r = 0; r < FEW_ROWS; ++r) {
        const uint32_t q[4] = {wv[a][r].x, wv[a][r].y, wv[a][r].z, wv[a][r].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack2<T>(q[i]);
          wf[r].p[i] = f2_pack(f.x, f.y);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint4 xv = *reinterpret_cast<const uint4*>(x[t] + k + a * step);
        const uint32_t q[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack2<T>(q[i]);
          const uint64_t xf = f2_pack(f.x, f.y);
#pragma unroll
          for (int r = 0; r < FEW_ROWS; ++r) acc[t][r] = f2_fma(wf[r].p[i], xf, acc[t][r]);
        }
      }
    }
    if (k + AHEAD * step < p.K) load_w(k + AHEAD * step);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < FEW_ROWS; ++r) {
      const float2 f = f2_unpack(acc[t][r]);
      float v = f.x + f.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == (t * FEW_ROWS + r) % 32) part[warp][t * FEW_ROWS + r] = v;
    }
  __syncthreads();
  // one thread per (row group, token, output)
  constexpr int OUTS = GLU ? FEW_ROWS / 2 : FEW_ROWS;
  const int outs = FEW_WARPS / p.split * NT * OUTS;
  if (static_cast<int>(threadIdx.x) >= outs) return;
  const int g = threadIdx.x / (NT * OUTS), t = threadIdx.x / OUTS % NT, o = threadIdx.x % OUTS;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * (FEW_WARPS / p.split) + g) * OUTS + o;
  if (row >= p.rows || t >= p.tokens) return;
  float v = 0.f, u = 0.f;
  for (int q = 0; q < p.split; ++q) {
    v += part[g * p.split + q][t * FEW_ROWS + o];
    if (GLU) u += part[g * p.split + q][t * FEW_ROWS + 2 + o];
  }
  if constexpr (GLU) {
    if (p.gu != nullptr) {
      // this element's place in the packed layout of the tensor-core kernels (all tokens lie in the first row of boxes)
      const int j = static_cast<int>(row), c = j & 31;
      uint32_t* box = reinterpret_cast<uint32_t*>(p.gu + static_cast<int64_t>(j >> 5) * 384 + t);
      box[(c >> 2) * 128 + (c & 3)] = __byte_perm(__float_as_uint(v), __float_as_uint(u), 0x7632);
      reinterpret_cast<uint16_t*>(box + (8 + (c >> 3)) * 128)[c & 7] =
          static_cast<uint16_t>(__byte_perm(__float_as_uint(v), __float_as_uint(u), 0x0051));
    }
    v = ffn_act<ACT>(v) * u;
  }
  if constexpr (USE == FEW_LINEAR) {
    const int64_t at = static_cast<int64_t>(t) * p.rows + row;
    if (p.bias != nullptr) v += p.bias[row];
    if (p.pre != nullptr) p.pre[at] = v;
    v = ffn_act<ACT>(v);
    const int64_t from = t * p.ld_residual + row;
    if (p.residual != nullptr)
      v += p.wide ? static_cast<const float*>(p.residual)[from] : to_f32(static_cast<const T*>(p.residual)[from]);
    if (p.wide) {
      static_cast<float*>(p.out)[at] = v;
      return;
    }
  }
  static_cast<T*>(p.out)[static_cast<int64_t>(t) * p.rows + row] = from_f32<T>(v);
}

template <typename T, int NT, int USE, int ACT>
cudaError_t launch(FewParams p, cudaStream_t stream) {
  constexpr bool GLU = USE == FEW_GLU;
  const int64_t groups = (static_cast<int64_t>(p.rows) * (GLU ? 2 : 1) + FEW_ROWS - 1) / FEW_ROWS;
  // about 24 warps per SM, each with a full step of K at least
  p.split = 1;
  while (p.split < FEW_WARPS && groups * p.split < 152 * 24 && p.split * 2 * 256 <= p.K) p.split *= 2;
  const int64_t per_cta = FEW_WARPS / p.split;
  return launch_dependent(ffn_few_kernel<T, NT, USE, ACT>, dim3(static_cast<unsigned>((groups + per_cta - 1) / per_cta)),
                          dim3(FEW_THREADS), 0, stream, p);
}

template <typename T, int NT>
cudaError_t both(const FewParams& up, const FewParams& down, int act, cudaStream_t stream) {
  const cudaError_t e = act == PRM_ACT_SILU   ? launch<T, NT, FEW_GLU, PRM_ACT_SILU>(up, stream)
                        : act == PRM_ACT_GELU ? launch<T, NT, FEW_GLU, PRM_ACT_GELU>(up, stream)
                                              : launch<T, NT, FEW_GLU, PRM_ACT_GELU_TANH>(up, stream);
  return e == cudaSuccess ? launch<T, NT, FEW_DOWN, 0>(down, stream) : e;
}

template <typename T>
cudaError_t by_tokens(const FewParams& up, const FewParams& down, int act, cudaStream_t stream) {
  if (up.tokens == 1) return both<T, 1>(up, down, act, stream);
  if (up.tokens == 2) return both<T, 2>(up, down, act, stream);
  if (up.tokens <= 4) return both<T, 4>(up, down, act, stream);
  return both<T, 8>(up, down, act, stream);
}

template <typename T, int ACT>
cudaError_t linear(const FewParams& p, cudaStream_t stream) {
  if (p.tokens == 1) return launch<T, 1, FEW_LINEAR, ACT>(p, stream);
  if (p.tokens == 2) return launch<T, 2, FEW_LINEAR, ACT>(p, stream);
  if (p.tokens <= 4) return launch<T, 4, FEW_LINEAR, ACT>(p, stream);
  return launch<T, 8, FEW_LINEAR, ACT>(p, stream);
}

template <typename T>
cudaError_t linear(const FewParams& p, int act, cudaStream_t stream) {
  if (act == PRM_ACT_SILU) return linear<T, PRM_ACT_SILU>(p, stream);
  if (act == PRM_ACT_GELU) return linear<T, PRM_ACT_GELU>(p, stream);
  if (act == PRM_ACT_GELU_TANH) return linear<T, PRM_ACT_GELU_TANH>(p, stream);
  return linear<T, ACT_NONE>(p, stream);
}

}  // namespace

cudaError_t linear_few_forward(const LinearFew& p, int act, int dtype, cudaStream_t stream) {
  FewParams q{p.x, p.ldx, {p.w, nullptr}, p.y, nullptr, p.tokens, p.n, p.k, 1};
  q.bias = p.bias;
  q.residual = p.residual;
  q.ld_residual = p.ld_residual;
  q.pre = p.pre;
  q.wide = p.wide;
  return dtype == PRM_BF16 ? linear<__nv_bfloat16>(q, act, stream) : linear<__half>(q, act, stream);
}

cudaError_t ffn_few_forward(const void* x, int64_t ldx, const void* w_gate, const void* w_up, const void* w_down,
                            void* h, uint4* gu, void* y, int tokens, int d, int f, int act, int dtype,
                            cudaStream_t stream) {
  const FewParams up{x, ldx, {w_gate, w_up}, h, gu, tokens, f, d, 1};
  const FewParams down{h, f, {w_down, nullptr}, y, nullptr, tokens, d, f, 1};
  return dtype == PRM_BF16 ? by_tokens<__nv_bfloat16>(up, down, act, stream) : by_tokens<__half>(up, down, act, stream);
}

}  // namespace prm
