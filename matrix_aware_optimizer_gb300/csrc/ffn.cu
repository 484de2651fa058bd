// Gated feed-forward block on the tensor cores, forward and backward:
//   g = x Wg^T, u = x Wu^T, h = act(g) u, y = h Wd^T
//   dh = dy Wd, dg = dh u act'(g), du = dh act(g)
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T h
//
// Four launches of one persistent tcgen05 kernel with three epilogues:
//   GLU   : x against Wg and Wu at once. A pair of CTAs computes 256 tokens x
//           128 features of g and of u in one accumulator (the even CTA holds
//           the rows of Wg, the odd one those of Wu), so the activation and
//           the product happen in registers: g and u never go to memory as
//           GEMM outputs, only h does (and, for training, g and u once, packed)
//   DGLU  : dh = dy Wd; dh stays in the accumulator, dg and du come out
//   STORE : plain products: y; and dx, dWd, dWg, dWu from one tile queue
// Operands are read in the layout the caller has: K-major or MN-major tiles
// by TMA, without a transposed copy. dx sums over both projections in one
// accumulator (two operand pairs, one after the other, along K).
//
// Rounding: products accumulate in fp32. h, dg and du are rounded to 16 bits
// because they are operands of the next product. g and u are kept for the
// backward pass with 16 significand bits (24-bit floats: fp32 with the low
// byte cut off, 6 bytes for the two), so that the derivative adds no error
// next to those roundings: in an fp64 model of these steps (1024 tokens,
// 512 x 2048) the gradients were 0.0023 from the exact ones, as with g and u
// kept exactly, and with bf16 g and u 0.0029 - 0.0035.
//
// Bound by the tensor cores for more than a few hundred tokens. 8192 tokens,
// 2048 x 8192, bf16: forward 488 us (1.69 PFLOP/s), with g and u saved 515,
// backward 1185 (1.39), both passes 1.65 - 1.77 ms (1.50 - 1.40 PFLOP/s: the SM
// clock under the power cap decides); those of 4096 tokens, 5120 x 20480 4.87 -
// 5.20 ms (1.59 - 1.49). 16384 tokens, 768 x 2048: 0.43 ms (1.07); 65536 tokens, 256 x 704,
// where the tensors' bytes weigh more: 0.66 ms. Each launch alone (8192 tokens,
// 2048 x 8192): GLU 314 us (1.75 PFLOP/s, with 400 MB of g and u written), down
// 193 (1.43), DGLU 198 (1.39, 790 MB moved), gradients 870 (1.58); the tensor
// pipe is active 79, 65, 67 and 68 % of the time: every pair loads all of its
// operands itself, the last rounds are part empty, and DGLU's epilogue waits
// for g and u.
//
// The kernel is in block_gemm.cuh.
#include "block_gemm.cuh"

namespace prm {
namespace {

struct FfnSizes {
  size_t saved_h, saved;                                     // gu at saved_h
  size_t fwd_h, fwd_partial, fwd_counters, fwd;              // offsets and size of the forward workspace
  size_t bwd_du, bwd_partial, bwd_counters, bwd;             // dg at 0
  Split down;
};

FfnSizes sizes(int64_t T, int64_t d, int64_t f) {
  FfnSizes s{};
  if (T == 0) return s;
  const size_t act = round_up(static_cast<size_t>(T) * f * 2, 256);
  s.saved_h = act;
  s.saved = act + static_cast<size_t>((T + 31) / 32) * ((f + 31) / 32) * 384 * 16;
  s.down = split_last_wave(T, d, f);
  s.fwd_partial = act;
  s.fwd_counters = act + partial_bytes(s.down);
  s.fwd = s.fwd_counters + round_up(counter_bytes(s.down), 256);
  s.bwd_du = act;
  s.bwd = 2 * act;
  return s;
}

int check(int64_t T, int64_t d, int64_t f) {
  if (T < 0 || d < 1 || f < 1) return PRM_ERR_INVALID_ARG;
  if (d % 8 != 0 || f % 8 != 0) return PRM_ERR_ALIGNMENT;
  if (T >= (int64_t(1) << 31) - 256 || d >= (int64_t(1) << 24) || f >= (int64_t(1) << 24)) return PRM_ERR_UNSUPPORTED;
  // tiles are counted in 32 bits
  constexpr int64_t MOST = int64_t(1) << 30;
  if (tiles_of(T, f, BN_HALF) > MOST || 3 * tiles_of(d, f, BN) + tiles_of(T, d, BN) > MOST) return PRM_ERR_UNSUPPORTED;
  return PRM_OK;
}

}  // namespace
}  // namespace prm

extern "C" int prm_gated_ffn_sizes(int64_t tokens, int64_t d, int64_t f, size_t* saved, size_t* forward_workspace,
                                   size_t* backward_workspace) {
  using namespace prm;
  if (saved == nullptr || forward_workspace == nullptr || backward_workspace == nullptr) return PRM_ERR_INVALID_ARG;
  const int rc = check(tokens, d, f);
  if (rc != PRM_OK) return rc;
  const FfnSizes s = sizes(tokens, d, f);
  *saved = s.saved;
  *forward_workspace = s.fwd;
  *backward_workspace = s.bwd;
  return PRM_OK;
}

extern "C" int prm_gated_ffn_forward(const void* x, int64_t ldx, const void* w_gate, const void* w_up,
                                     const void* w_down, void* y, void* saved, void* workspace,
                                     size_t workspace_bytes, int64_t tokens, int64_t d, int64_t f, int act, int dtype,
                                     void* stream) {
  using namespace prm;
  if ((dtype != PRM_BF16 && dtype != PRM_FP16) || act < PRM_ACT_SILU || act > PRM_ACT_GELU_TANH)
    return PRM_ERR_INVALID_ARG;
  int rc = check(tokens, d, f);
  if (rc != PRM_OK || tokens == 0) return rc;
  if (x == nullptr || w_gate == nullptr || w_up == nullptr || w_down == nullptr || y == nullptr || ldx < d)
    return PRM_ERR_INVALID_ARG;
  if (ldx % 8 != 0 || !aligned_to(x, 16) || !aligned_to(w_gate, 16) || !aligned_to(w_up, 16) ||
      !aligned_to(w_down, 16) || !aligned_to(y, 16) || !aligned_to(saved, 256) || !aligned_to(workspace, 256))
    return PRM_ERR_ALIGNMENT;
  const FfnSizes sz = sizes(tokens, d, f);
  if (workspace == nullptr || workspace_bytes < sz.fwd) return PRM_ERR_WORKSPACE;
  const BlockDevice* dev;
  if ((rc = block_device(&dev)) != PRM_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  void* h = saved != nullptr ? saved : ws;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (ffn_few(tokens, d, f))
    return ffn_few_forward(x, ldx, w_gate, w_up, w_down, h,
                           saved != nullptr ? reinterpret_cast<uint4*>(static_cast<char*>(saved) + sz.saved_h) : nullptr,
                           y, static_cast<int>(tokens), static_cast<int>(d), static_cast<int>(f), act, dtype,
                           st) == cudaSuccess
               ? PRM_OK
               : PRM_ERR_CUDA;

  BlockGemmParams p{};
  p.err = dev->d_err;
  p.gu = saved != nullptr ? reinterpret_cast<uint4*>(static_cast<char*>(saved) + sz.saved_h) : nullptr;
  uint32_t* counters = reinterpret_cast<uint32_t*>(ws + sz.fwd_counters);
  p.zero = counters;
  p.zero_count = static_cast<int>(counter_bytes(sz.down) / 4);
  GemmSegment sg{};
  if (!encode(&sg.a[0], x, dtype, tokens, d, ldx, MAP_ROWS) || !encode(&sg.b[0], w_gate, dtype, f, d, d, MAP_ROWS) ||
      !encode(&sg.b[1], w_up, dtype, f, d, d, MAP_ROWS) || !encode(&sg.out[0], h, dtype, tokens, f, f, MAP_STORE))
    return PRM_ERR_CUDA;
  queue(p, sg, tokens, f, d, 0, false, false, BN_HALF);
  if (launch_act<EPI_GLU>(p, act, dtype, dev->num_sms, st) != cudaSuccess) return PRM_ERR_CUDA;

  BlockGemmParams q{};
  q.err = dev->d_err;
  GemmSegment dn{};
  if (!encode(&dn.a[0], h, dtype, tokens, f, f, MAP_ROWS) || !encode(&dn.b[0], w_down, dtype, d, f, f, MAP_ROWS) ||
      !encode(&dn.out[0], y, dtype, tokens, d, d, MAP_STORE))
    return PRM_ERR_CUDA;
  dn.whole = static_cast<int>(sz.down.whole);
  dn.splits = sz.down.splits;
  dn.partial = reinterpret_cast<float*>(ws + sz.fwd_partial);
  dn.arrived = counters;
  queue(q, dn, tokens, d, f, 0, false, false, BN);
  return launch<EPI_STORE>(q, dtype, dev->num_sms, st) == cudaSuccess ? PRM_OK : PRM_ERR_CUDA;
}

extern "C" int prm_gated_ffn_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w_gate,
                                      const void* w_up, const void* w_down, const void* saved, void* dx,
                                      void* dw_gate, void* dw_up, void* dw_down, void* workspace,
                                      size_t workspace_bytes, int64_t tokens, int64_t d, int64_t f, int act,
                                      int dtype, void* stream) {
  using namespace prm;
  if ((dtype != PRM_BF16 && dtype != PRM_FP16) || act < PRM_ACT_SILU || act > PRM_ACT_GELU_TANH)
    return PRM_ERR_INVALID_ARG;
  int rc = check(tokens, d, f);
  if (rc != PRM_OK) return rc;
  const bool weights = dw_gate != nullptr || dw_up != nullptr || dw_down != nullptr;
  if (weights && (dw_gate == nullptr || dw_up == nullptr || dw_down == nullptr)) return PRM_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    const size_t n = static_cast<size_t>(d) * f * 2;
    if (weights && (cudaMemsetAsync(dw_gate, 0, n, st) != cudaSuccess ||
                    cudaMemsetAsync(dw_up, 0, n, st) != cudaSuccess ||
                    cudaMemsetAsync(dw_down, 0, n, st) != cudaSuccess))
      return PRM_ERR_CUDA;
    return PRM_OK;
  }
  if (dy == nullptr || x == nullptr || w_gate == nullptr || w_up == nullptr || w_down == nullptr ||
      saved == nullptr || lddy < d || ldx < d)
    return PRM_ERR_INVALID_ARG;
  const void* ptrs[9] = {dy, x, w_gate, w_up, w_down, dx, dw_gate, dw_up, dw_down};
  for (const void* q : ptrs)
    if (!aligned_to(q, 16)) return PRM_ERR_ALIGNMENT;
  if (lddy % 8 != 0 || ldx % 8 != 0 || !aligned_to(saved, 256) || !aligned_to(workspace, 256))
    return PRM_ERR_ALIGNMENT;
  const FfnSizes sz = sizes(tokens, d, f);
  if (workspace == nullptr || workspace_bytes < sz.bwd) return PRM_ERR_WORKSPACE;
  if (dx == nullptr && !weights) return PRM_OK;
  const BlockDevice* dev;
  if ((rc = block_device(&dev)) != PRM_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  void* dg = ws;
  void* du = ws + sz.bwd_du;
  const void* h = saved;

  BlockGemmParams p{};
  p.err = dev->d_err;
  p.gu = reinterpret_cast<uint4*>(const_cast<char*>(static_cast<const char*>(saved)) + sz.saved_h);
  GemmSegment sg{};
  if (!encode(&sg.a[0], dy, dtype, tokens, d, lddy, MAP_ROWS) || !encode(&sg.b[0], w_down, dtype, d, f, f, MAP_COLS) ||
      !encode(&sg.out[0], dg, dtype, tokens, f, f, MAP_STORE) ||
      !encode(&sg.out[1], du, dtype, tokens, f, f, MAP_STORE))
    return PRM_ERR_CUDA;
  queue(p, sg, tokens, f, d, 0, false, true, BN);
  if (launch_act<EPI_DGLU>(p, act, dtype, dev->num_sms, st) != cudaSuccess) return PRM_ERR_CUDA;

  // dx (K = 2 f) and the weight gradients (K = tokens) from one queue, the
  // longer sums first, so that the last tiles of the queue are short.
  BlockGemmParams q{};
  q.err = dev->d_err;
  bool ok = true;
  auto add_dx = [&] {
    if (dx == nullptr) return;
    GemmSegment s{};
    ok = ok && encode(&s.a[0], dg, dtype, tokens, f, f, MAP_ROWS) &&
         encode(&s.a[1], du, dtype, tokens, f, f, MAP_ROWS) &&
         encode(&s.b[0], w_gate, dtype, f, d, d, MAP_COLS) && encode(&s.b[1], w_up, dtype, f, d, d, MAP_COLS) &&
         encode(&s.out[0], dx, dtype, tokens, d, d, MAP_STORE);
    queue(q, s, tokens, d, f, f, false, true, BN);
  };
  auto add_weight = [&](const void* a, int64_t lda, int64_t m, const void* b, int64_t ldb, int64_t n, void* out) {
    GemmSegment s{};
    ok = ok && encode(&s.a[0], a, dtype, tokens, m, lda, MAP_COLS) &&
         encode(&s.b[0], b, dtype, tokens, n, ldb, MAP_COLS) && encode(&s.out[0], out, dtype, m, n, n, MAP_STORE);
    queue(q, s, m, n, tokens, 0, true, true, BN);
  };
  const bool dx_first = 2 * f >= tokens;
  if (dx_first) add_dx();
  if (weights) {
    add_weight(dg, f, f, x, ldx, d, dw_gate);
    add_weight(du, f, f, x, ldx, d, dw_up);
    add_weight(dy, lddy, d, h, f, f, dw_down);
  }
  if (!dx_first) add_dx();
  if (!ok) return PRM_ERR_CUDA;
  return launch<EPI_STORE>(q, dtype, dev->num_sms, st) == cudaSuccess ? PRM_OK : PRM_ERR_CUDA;
}
