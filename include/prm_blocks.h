/*
 * prm_blocks.h -- C ABI of libprm, second part: the operators of a
 * transformer block whose parameters the optimizer of prm.h updates, forward
 * and backward, on one GB300 GPU:
 *
 *   gated feed-forward block   its three matrices are PR-Muon's
 *   norms around a block       their gains are AdamW's; gate, scale and shift
 *                              are the outputs of the adaLN matrix (PR-Muon's)
 *   token embedding            its table is AdamW's
 *
 * Conventions are prm.h's: PRM_OK or a PRM_ERR_* code, device pointers on the
 * current device, `void*` streams, the caller owns every buffer (workspaces
 * included), work is enqueued asynchronously. Element types are PRM_FP32,
 * PRM_BF16 and PRM_FP16. Every call with nothing to do (no rows) returns
 * PRM_OK; pointers may then be NULL. Sums are held in fp32 and taken in an
 * order fixed by the sizes: the same inputs give the same bits. The first
 * call of each kind on a device sets kernels up (attributes, an error word):
 * make it before any stream capture. Calls on different streams may overlap
 * when their outputs and workspaces differ.
 */
#ifndef PRM_BLOCKS_H
#define PRM_BLOCKS_H

#include "prm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Synchronises `stream`, one of the current device, and reads that device's
 * error word of the calls below (a bounded device-side wait that gave up; the
 * call's outputs are then worthless). Returns PRM_OK, TIMEOUT or CUDA; clears
 * the word. */
PRM_API int prm_blocks_sync_status(void* stream);

/* ---- gated feed-forward block ------------------------------------------
 *   g = x w_gate^T,  u = x w_up^T,  h = act(g) * u,  y = h w_down^T
 * x, y: tokens x d; w_gate, w_up: f x d; w_down: d x f; all row-major and of
 * one 16-bit type `dtype` (PRM_BF16 or PRM_FP16). x has row pitch ldx
 * elements, everything else is contiguous. d and f are multiples of 8,
 * pointers 16-byte aligned, ldx % 8 == 0 (TMA rows). tokens is any number. */
#define PRM_ACT_SILU      0  /* g / (1 + exp(-g)) */
#define PRM_ACT_GELU      1  /* g (1 + erf(g / sqrt 2)) / 2 */
#define PRM_ACT_GELU_TANH 2  /* g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2 */

/* Bytes of the buffer in which the forward pass leaves h, g and u for the
 * backward pass, and of the two passes' workspaces. Errors: INVALID_ARG,
 * ALIGNMENT (d or f not a multiple of 8). */
PRM_API int prm_gated_ffn_sizes(int64_t tokens, int64_t d, int64_t f, size_t* saved, size_t* forward_workspace,
                                size_t* backward_workspace);

/* y from x. saved: prm_gated_ffn_sizes' `saved` bytes, 256-byte aligned, or
 * NULL where no backward pass follows. workspace: 256-byte aligned, at least
 * `forward_workspace` bytes. h is rounded to dtype for the second product (in
 * fp16 an h beyond 65504 becomes infinite); saved holds h in dtype and g and u
 * with 16 significand bits each.
 * Errors: INVALID_ARG, ALIGNMENT, WORKSPACE, UNSUPPORTED, CUDA. */
PRM_API int prm_gated_ffn_forward(const void* x, int64_t ldx, const void* w_gate, const void* w_up,
                                  const void* w_down, void* y, void* saved, void* workspace, size_t workspace_bytes,
                                  int64_t tokens, int64_t d, int64_t f, int act, int dtype, void* stream);

/* From dy (row pitch lddy) and the forward pass's saved buffer:
 *   dh = dy w_down,  dg = dh * u * act'(g),  du = dh * act(g)   (dh in fp32; dg, du rounded to dtype)
 *   dx = dg w_gate + du w_up,  dw_gate = dg^T x,  dw_up = du^T x,  dw_down = dy^T h
 * dx may be NULL (not wanted), and so may all three weight gradients
 * together. The weight gradients are written, not added to; with no tokens
 * they are set to zero. `saved` is read only.
 * Errors as for the forward pass. */
PRM_API int prm_gated_ffn_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w_gate,
                                   const void* w_up, const void* w_down, const void* saved, void* dx, void* dw_gate,
                                   void* dw_up, void* dw_down, void* workspace, size_t workspace_bytes,
                                   int64_t tokens, int64_t d, int64_t f, int act, int dtype, void* stream);

/* ---- norms before and after a block ------------------------------------
 * Between a block that produced z and the next block's input y, over rows of
 * d elements:
 *   P = N(z) * post_weight           (z itself when post_weight is NULL)
 *   r = alpha x + gate_b * P         (gate_b = 1 when gate is NULL)
 *   y = N(r) * pre_weight * (1 + scale_b) + shift_b
 * with N(v) = v / sqrt(mean(v^2) + eps) (PRM_NORM_RMS) or
 * (v - mean(v)) / sqrt(var(v) + eps) (PRM_NORM_LAYER). r is the residual
 * stream: it is rounded to its type, and N reads the rounded r, so that the
 * backward pass differentiates what the forward pass computed.
 * z == NULL: no block yet, r is x (not written; alpha must be 1). y == NULL:
 * nothing follows, only r is written. */
#define PRM_NORM_RMS   0
#define PRM_NORM_LAYER 1

typedef struct {
  int64_t rows;             /* all rows of all samples, below 2^32, and below 2^31 where d > 256 */
  int64_t rows_per_sample;  /* rows that share a row of gate / scale / shift; divides rows (>= 1) */
  int64_t d;                /* 1 .. 8192 */
  int32_t kind;             /* PRM_NORM_* */
  int32_t stream_dtype;     /* x, r, dr, dx */
  int32_t block_dtype;      /* z, y, dy, dz and gate, scale, shift; fp32 only when the stream is, else fp32
                               stream or the same type */
  float alpha;
  float eps;
  int32_t reserved;         /* must be 0 */
  const float* post_weight; /* d, or NULL */
  const float* pre_weight;  /* d, or NULL for 1 */
  const void* gate;         /* samples x d with row pitch gate_ld, or NULL */
  const void* scale;        /* samples x d with row pitch scale_ld, or NULL for 0 */
  const void* shift;        /* samples x d with row pitch shift_ld, or NULL for 0 */
  int64_t gate_ld, scale_ld, shift_ld;
} prm_block_norm_desc;

/* x, z, r, y: rows x d, contiguous; stats: 4 fp32 per row, 16-byte aligned
 * (mean and reciprocal deviation of r, then of z; the mean is 0 for the rms
 * kind, z's pair is 0 without post_weight), or NULL where no backward pass
 * follows. r and x may be the same buffer. Any alignment and any d; rows of
 * 16-byte aligned buffers with d % 8 == 0 take the vector path.
 * Errors: INVALID_ARG, SHAPE, ALIGNMENT, UNSUPPORTED, CUDA. */
PRM_API int prm_block_norm_forward(const prm_block_norm_desc* desc, const void* x, const void* z, void* r, void* y,
                                   float* stats, void* stream);

/* Bytes of workspace of the backward pass (column sums). */
PRM_API int prm_block_norm_workspace(const prm_block_norm_desc* desc, size_t* bytes);

/* Gradients from dy (of y) and dr (of r, from the rows' later uses; NULL for
 * 0); r, z and stats as the forward pass left them (r: x where z was NULL).
 * Without post_weight and gate, z may be NULL here even if the forward pass had
 * one (dz is then not wanted); dx is alpha times r's gradient all the same.
 * dx (NULL allowed, as is dz) and dz are rows x d; dpost, dpre: d fp32;
 * dgate, dscale, dshift: samples x d contiguous of block_dtype. A gradient
 * pointer is required for each parameter that desc holds and ignored for the
 * others. dx may be the same buffer as dr, dz as dy.
 * dy == NULL: y was not used (dr alone).
 * Errors: INVALID_ARG, SHAPE, ALIGNMENT, WORKSPACE, UNSUPPORTED, CUDA. */
PRM_API int prm_block_norm_backward(const prm_block_norm_desc* desc, const void* dy, const void* dr, const void* r,
                                    const void* z, const float* stats, void* dx, void* dz, float* dpost, void* dgate,
                                    float* dpre, void* dscale, void* dshift, void* workspace, size_t workspace_bytes,
                                    void* stream);

/* ---- token embedding ----------------------------------------------------
 *   out[t] = scale * table[token[t]]
 * table: vocab x d of table_dtype, out: tokens x d of out_dtype, contiguous;
 * token: int64 (token_bytes 8) or int32 (4). A token outside [0, vocab) is
 * padding: its row of out is zero and it adds nothing to the gradient.
 * Any alignment and any d. Errors: INVALID_ARG, CUDA. */
PRM_API int prm_embedding_forward(const void* token, int token_bytes, const void* table, int table_dtype, void* out,
                                  int out_dtype, int64_t tokens, int64_t vocab, int64_t d, float scale, void* stream);

/* Bytes of workspace of the backward pass. */
PRM_API int prm_embedding_backward_workspace(int64_t tokens, int64_t vocab, int64_t d, size_t* bytes);

/*   grad[v] = scale * sum over t with token[t] == v of dout[t]   (+ grad[v] when accumulate is not 0)
 * for every v in [0, vocab); a row without tokens is set to zero, or left as
 * it is when accumulating. Tokens are sorted (stably, by a radix sort) and
 * each row's sum is taken in the order of t in fp32, long runs as sums of
 * fixed pieces: no atomics on values. tokens < 2^31 - 2^16, vocab < 2^31.
 * workspace: 256-byte aligned, prm_embedding_backward_workspace's bytes.
 * Errors: INVALID_ARG, ALIGNMENT, WORKSPACE, UNSUPPORTED, CUDA. */
PRM_API int prm_embedding_backward(const void* dout, int dout_dtype, const void* token, int token_bytes, void* grad,
                                   int grad_dtype, int accumulate, int64_t tokens, int64_t vocab, int64_t d,
                                   float scale, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PRM_BLOCKS_H */
