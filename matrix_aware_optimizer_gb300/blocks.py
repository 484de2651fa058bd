"""torch glue over include/prm_blocks.h: the operators of a transformer block
whose parameters the optimizer updates. Each operator is a forward and a
backward call on tensors; PyTorch supplies memory and the stream, every
arithmetic step runs in libprm. Outputs and workspaces are allocated on the
stream the call runs on (`stream`, or the current one)."""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import native as N

_DTYPE = {torch.float32: N.PRM_FP32, torch.bfloat16: N.PRM_BF16, torch.float16: N.PRM_FP16}
_ACT = {"silu": N.PRM_ACT_SILU, "gelu": N.PRM_ACT_GELU, "gelu_tanh": N.PRM_ACT_GELU_TANH}
_KIND = {"rms": N.PRM_NORM_RMS, "layer": N.PRM_NORM_LAYER}


@contextlib.contextmanager
def _other_stream(dev, stream):
    with torch.cuda.device(dev):
        if stream is None:
            yield torch.cuda.current_stream().cuda_stream
        else:
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


class _Here:
    """The usual case of _on: current device, current stream."""
    __slots__ = ("handle",)

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        return False


def _on(dev: torch.device, stream: Optional[torch.cuda.Stream]):
    """Context in which tensors are allocated for, and work is enqueued on,
    the call's stream; yields the stream's handle."""
    if stream is None and (dev.index is None or dev.index == torch.cuda.current_device()):
        return _Here(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    return _other_stream(dev, stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def blocks_sync_status(stream: Optional[torch.cuda.Stream] = None) -> None:
    """Waits for the stream and raises if a device-side wait of a block
    operator gave up."""
    s = stream if stream is not None else torch.cuda.current_stream()
    N.check(N.load().prm_blocks_sync_status(s.cuda_stream), "prm_blocks_sync_status")


# ---------------------------------------------------------------- gated FFN
class FfnSaved(NamedTuple):
    """What gated_ffn leaves for gated_ffn_backward: h, g and u of one pass
    (8 bytes per token and feature), in the library's own layout."""
    buffer: torch.Tensor
    tokens: int


def _rows16(t: torch.Tensor, d: int, name: str) -> Tuple[torch.Tensor, int]:
    """t as rows of d elements with a pitch TMA can read: (tensor, pitch).
    Other layouts are copied."""
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= d and t.stride(0) % 8 == 0 and t.data_ptr() % 16 == 0:
        return t, t.stride(0)
    t = t.reshape(-1, d)
    if t.stride(1) != 1 or t.stride(0) < d or t.stride(0) % 8 or t.data_ptr() % 16:
        t = t.clone(memory_format=torch.contiguous_format)
    return t, t.stride(0)


def _ffn_check(x, w_gate, w_up, w_down, act):
    dt = x.dtype
    if act not in _ACT:
        raise ValueError(f"act must be one of {sorted(_ACT)}")
    if dt not in (torch.bfloat16, torch.float16) or not x.is_cuda:
        raise ValueError("x must be a bfloat16 or float16 CUDA tensor")
    d = x.shape[-1]
    f = w_gate.shape[0]
    if w_gate.shape != (f, d) or w_up.shape != (f, d) or w_down.shape != (d, f):
        raise ValueError("w_gate and w_up must be f x d and w_down d x f, d the last extent of x")
    for w in (w_gate, w_up, w_down):
        if w.dtype != dt or w.device != x.device or not w.is_contiguous():
            raise ValueError("weights must be contiguous, of x's type and on its device")
    if d % 8 or f % 8:
        raise ValueError("d and f must be multiples of 8")
    return d, f


def _ffn_sizes(tokens, d, f):
    saved, forward, backward = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    N.check(N.load().prm_gated_ffn_sizes(tokens, d, f, saved, forward, backward), "prm_gated_ffn_sizes")
    return saved.value, forward.value, backward.value


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, act: str = "silu",
              save: bool = False, stream: Optional[torch.cuda.Stream] = None):
    """Gated feed-forward block, y = (act(x w_gate^T) * (x w_up^T)) w_down^T.

    x: [..., d] bf16 or fp16; w_gate, w_up: [f, d]; w_down: [d, f], all of x's
    type; d and f multiples of 8. act: "silu", "gelu" (erf) or "gelu_tanh".
    Returns y, or (y, saved) with save=True, saved for gated_ffn_backward.
    """
    d, f = _ffn_check(x, w_gate, w_up, w_down, act)
    with _on(x.device, stream) as handle:
        x2, ldx = _rows16(x, d, "x")
        tokens = x2.shape[0]
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        n_saved, n_ws, _ = _ffn_sizes(tokens, d, f)
        saved = torch.empty(n_saved, dtype=torch.uint8, device=x.device) if save else None
        ws = torch.empty(n_ws, dtype=torch.uint8, device=x.device)
        N.check(N.load().prm_gated_ffn_forward(x2.data_ptr(), ldx, w_gate.data_ptr(), w_up.data_ptr(),
                                               w_down.data_ptr(), y.data_ptr(), _ptr(saved), ws.data_ptr(), n_ws,
                                               tokens, d, f, _ACT[act], _DTYPE[x.dtype], handle),
                "prm_gated_ffn_forward")
    return (y, FfnSaved(saved, tokens)) if save else y


def gated_ffn_backward(dy: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                       w_down: torch.Tensor, saved: FfnSaved, act: str = "silu", need_dx: bool = True,
                       grads: Optional[Sequence[torch.Tensor]] = None,
                       stream: Optional[torch.cuda.Stream] = None):
    """Gradients of gated_ffn: (dx, dw_gate, dw_up, dw_down), all of x's type.

    grads: three tensors of the weights' shapes and type to write the weight
    gradients into, e.g. the buffers that PeriodicRowMuon has registered (they
    are overwritten). dx is None with need_dx=False.
    """
    d, f = _ffn_check(x, w_gate, w_up, w_down, act)
    if dy.shape != x.shape or dy.dtype != x.dtype or dy.device != x.device:
        raise ValueError("dy must have x's shape, type and device")
    with _on(x.device, stream) as handle:
        x2, ldx = _rows16(x, d, "x")
        dy2, lddy = _rows16(dy, d, "dy")
        tokens = x2.shape[0]
        n_saved, _, n_ws = _ffn_sizes(tokens, d, f)
        if saved.tokens != tokens or saved.buffer.numel() != n_saved:
            raise ValueError("saved does not belong to this x")
        if grads is None:
            grads = (torch.empty_like(w_gate), torch.empty_like(w_up), torch.empty_like(w_down))
        else:
            for g, w in zip(grads, (w_gate, w_up, w_down)):
                if g.shape != w.shape or g.dtype != w.dtype or g.device != w.device or not g.is_contiguous():
                    raise ValueError("grads must be three contiguous tensors of the weights' shapes and type")
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if need_dx else None
        ws = torch.empty(n_ws, dtype=torch.uint8, device=x.device)
        N.check(N.load().prm_gated_ffn_backward(dy2.data_ptr(), lddy, x2.data_ptr(), ldx, w_gate.data_ptr(),
                                                w_up.data_ptr(), w_down.data_ptr(), saved.buffer.data_ptr(),
                                                _ptr(dx), grads[0].data_ptr(), grads[1].data_ptr(),
                                                grads[2].data_ptr(), ws.data_ptr(), n_ws, tokens, d, f, _ACT[act],
                                                _DTYPE[x.dtype], handle), "prm_gated_ffn_backward")
    return dx, grads[0], grads[1], grads[2]


# --------------------------------------------------------- norms of a block
class BlockNormGrads(NamedTuple):
    """Gradients of block_norm; None for what was not given or not asked for."""
    dx: Optional[torch.Tensor]
    dz: Optional[torch.Tensor]
    dpost_weight: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dpre_weight: Optional[torch.Tensor]
    dscale: Optional[torch.Tensor]
    dshift: Optional[torch.Tensor]


def _norm_desc(ref, block_dtype, kind, alpha, eps, post_weight, gate, pre_weight, scale, shift):
    """Descriptor for rows shaped like `ref` (the residual stream)."""
    if kind not in _KIND:
        raise ValueError(f"kind must be one of {sorted(_KIND)}")
    if ref.dtype not in _DTYPE or block_dtype not in _DTYPE:
        raise ValueError("tensors must be float32, bfloat16 or float16")
    if ref.dtype != torch.float32 and ref.dtype != block_dtype:
        raise ValueError("a 16-bit residual stream needs a block of the same type")
    d = ref.shape[-1]
    rows = ref.numel() // d if d else 0
    samples = 0
    for w in (post_weight, pre_weight):
        if w is not None and (w.shape != (d,) or w.dtype != torch.float32 or w.device != ref.device
                              or not w.is_contiguous()):
            raise ValueError("post_weight and pre_weight must be contiguous float32 tensors of d elements")
    for m in (gate, scale, shift):
        if m is None:
            continue
        if m.dim() != 2 or m.shape[1] != d or m.dtype != block_dtype or m.device != ref.device or m.stride(1) != 1 \
                or (m.shape[0] > 1 and m.stride(0) < d):
            raise ValueError("gate, scale and shift must be samples x d of the block's type with unit column stride")
        if samples and m.shape[0] != samples:
            raise ValueError("gate, scale and shift must have the same number of samples")
        samples = m.shape[0]
        if samples == 0 or rows % samples:
            raise ValueError("the samples must divide the rows")
    lds = [0 if m is None else max(m.stride(0), d) for m in (gate, scale, shift)]
    desc = N.prm_block_norm_desc(rows, max(1, rows // samples if samples else rows), d, _KIND[kind],
                                 _DTYPE[ref.dtype], _DTYPE[block_dtype], alpha, eps, 0, _ptr(post_weight),
                                 _ptr(pre_weight), _ptr(gate), _ptr(scale), _ptr(shift), *lds)
    return desc, rows


def _norm_rows(t, like, dtype, name):
    if t.shape != like.shape or t.dtype != dtype or t.device != like.device:
        raise ValueError(f"{name} must have the residual stream's shape and device and be {dtype}")
    return t if t.is_contiguous() else t.contiguous()


def block_norm(x: torch.Tensor, z: Optional[torch.Tensor] = None, kind: str = "rms", alpha: float = 1.0,
               post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
               pre_weight: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
               shift: Optional[torch.Tensor] = None, eps: float = 1e-6, dtype: Optional[torch.dtype] = None,
               join_only: bool = False, stream: Optional[torch.cuda.Stream] = None):
    """Norms around a block, fused with its gate and residual scale:

      r = alpha x + gate_b * (N(z) post_weight, or z without post_weight)
      y = N(r) pre_weight (1 + scale_b) + shift_b

    x: residual stream [..., d], fp32, bf16 or fp16; z: the block's output, of
    x's shape, fp32 only with an fp32 stream, else x's type or a 16-bit type
    under an fp32 stream. post_weight, pre_weight: [d] fp32; gate, scale,
    shift: [samples, d] of the block's type, consecutive rows of x sharing a
    sample (rows may be strided: slices of one modulation tensor). kind: "rms"
    or "layer". z None: r is x, y is its norm (`dtype` picks y's type).
    join_only: no norm follows; y is None.

    Returns (r, y, stats), stats for block_norm_backward.
    """
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    block = z.dtype if z is not None else (dtype if dtype is not None else x.dtype)
    if dtype is not None and dtype != block:
        raise ValueError("dtype must be z's")
    if z is None and (join_only or alpha != 1.0 or gate is not None or post_weight is not None):
        raise ValueError("alpha, gate, post_weight and join_only need z")
    if join_only and (pre_weight is not None or scale is not None or shift is not None):
        raise ValueError("pre_weight, scale and shift belong to the norm that join_only leaves out")
    with _on(x.device, stream) as handle:
        x = x if x.is_contiguous() else x.contiguous()
        if z is not None:
            z = _norm_rows(z, x, block, "z")
        desc, rows = _norm_desc(x, block, kind, alpha, eps, post_weight, gate, pre_weight, scale, shift)
        r = torch.empty_like(x) if z is not None else x
        y = None if join_only else torch.empty(x.shape, dtype=block, device=x.device)
        stats = torch.empty(rows, 4, dtype=torch.float32, device=x.device)
        N.check(N.load().prm_block_norm_forward(desc, x.data_ptr(), _ptr(z), r.data_ptr(), _ptr(y), stats.data_ptr(),
                                                handle), "prm_block_norm_forward")
    return r, y, stats


def block_norm_backward(dy: Optional[torch.Tensor], dr: Optional[torch.Tensor], r: torch.Tensor,
                        z: Optional[torch.Tensor], stats: torch.Tensor, kind: str = "rms", alpha: float = 1.0,
                        post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                        pre_weight: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                        shift: Optional[torch.Tensor] = None, need_dx: bool = True,
                        stream: Optional[torch.cuda.Stream] = None) -> BlockNormGrads:
    """Gradients of block_norm from dy (of y; None after join_only) and dr (of
    r, from its later uses; None for none), with the r and stats that it
    returned and the same z and parameters. dpost_weight and dpre_weight are
    fp32, the others of their tensor's type."""
    if dy is None and dr is None:
        raise ValueError("dy and dr are both None")
    if not r.is_cuda:
        raise ValueError("r must be a CUDA tensor")
    block = z.dtype if z is not None else dy.dtype if dy is not None else r.dtype
    with _on(r.device, stream) as handle:
        desc, rows = _norm_desc(r, block, kind, alpha, 0.0, post_weight, gate, pre_weight, scale, shift)
        r = r if r.is_contiguous() else r.contiguous()
        dy = None if dy is None else _norm_rows(dy, r, block, "dy")
        dr = None if dr is None else _norm_rows(dr, r, r.dtype, "dr")
        z = None if z is None else _norm_rows(z, r, block, "z")
        if stats.shape != (rows, 4) or stats.dtype != torch.float32 or stats.device != r.device \
                or not stats.is_contiguous():
            raise ValueError("stats must be the tensor block_norm returned")
        d = r.shape[-1]

        def vec(w):
            return None if w is None else torch.empty(d, dtype=torch.float32, device=r.device)

        def mod(m):
            return None if m is None else torch.empty(m.shape, dtype=block, device=r.device)

        out = BlockNormGrads(torch.empty_like(r) if need_dx else None, None if z is None else torch.empty_like(z),
                             vec(post_weight), mod(gate), vec(pre_weight), mod(scale), mod(shift))
        if rows == 0:
            for t in out[2:]:
                if t is not None:
                    t.zero_()
            return out
        n = ctypes.c_size_t()
        N.check(N.load().prm_block_norm_workspace(desc, n), "prm_block_norm_workspace")
        ws = torch.empty(n.value, dtype=torch.uint8, device=r.device) if n.value else None
        N.check(N.load().prm_block_norm_backward(desc, _ptr(dy), _ptr(dr), r.data_ptr(), _ptr(z), stats.data_ptr(),
                                                 *(_ptr(t) for t in out), _ptr(ws), n.value, handle),
                "prm_block_norm_backward")
    return out


# ---------------------------------------------------------------- embedding
def _tokens(tokens: torch.Tensor) -> torch.Tensor:
    if tokens.dtype not in (torch.int64, torch.int32) or not tokens.is_cuda:
        raise ValueError("tokens must be an int64 or int32 CUDA tensor")
    return tokens if tokens.is_contiguous() else tokens.contiguous()


def embedding(tokens: torch.Tensor, table: torch.Tensor, scale: float = 1.0, dtype: Optional[torch.dtype] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """scale * table[tokens], as `dtype` (default: the table's). table: [vocab,
    d] fp32, bf16 or fp16. A token outside [0, vocab) is padding: a zero row."""
    dtype = table.dtype if dtype is None else dtype
    if table.dim() != 2 or table.dtype not in _DTYPE or dtype not in _DTYPE or not table.is_contiguous() \
            or not table.is_cuda or table.device != tokens.device:
        raise ValueError("table must be a contiguous vocab x d CUDA tensor of float32, bfloat16 or float16")
    with _on(table.device, stream) as handle:
        tok = _tokens(tokens)
        vocab, d = table.shape
        out = torch.empty(*tokens.shape, d, dtype=dtype, device=table.device)
        N.check(N.load().prm_embedding_forward(tok.data_ptr(), tok.element_size(), table.data_ptr(),
                                               _DTYPE[table.dtype], out.data_ptr(), _DTYPE[dtype], tok.numel(), vocab,
                                               d, scale, handle), "prm_embedding_forward")
    return out


def embedding_backward(dout: torch.Tensor, tokens: torch.Tensor, vocab: int, scale: float = 1.0,
                       dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                       accumulate: bool = False, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Gradient of embedding's table [vocab, d] as `dtype`: the sum of dout's
    rows per token, in the order of the tokens (deterministic), times scale;
    rows without tokens are zero. out: a tensor to write it into (of `dtype`'s
    place); accumulate=True adds to what out holds, e.g. the output layer's
    gradient of a tied table."""
    if dout.dtype not in _DTYPE or not dout.is_cuda or dout.shape[:-1] != tokens.shape or dout.device != tokens.device:
        raise ValueError("dout must be tokens' shape x d, float32, bfloat16 or float16, on the tokens' device")
    d = dout.shape[-1]
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if out is not None and (out.shape != (vocab, d) or out.dtype not in _DTYPE or out.device != dout.device
                            or not out.is_contiguous()):
        raise ValueError("out must be a contiguous vocab x d tensor of float32, bfloat16 or float16")
    if out is None and dtype not in _DTYPE:
        raise ValueError("dtype must be float32, bfloat16 or float16")
    with _on(dout.device, stream) as handle:
        tok = _tokens(tokens)
        dout = dout if dout.is_contiguous() else dout.contiguous()
        grad = torch.empty(vocab, d, dtype=dtype, device=dout.device) if out is None else out
        n = ctypes.c_size_t()
        N.check(N.load().prm_embedding_backward_workspace(tok.numel(), vocab, d, n),
                "prm_embedding_backward_workspace")
        ws = torch.empty(n.value, dtype=torch.uint8, device=dout.device)
        N.check(N.load().prm_embedding_backward(dout.data_ptr(), _DTYPE[dout.dtype], tok.data_ptr(),
                                                tok.element_size(), grad.data_ptr(), _DTYPE[grad.dtype],
                                                1 if accumulate else 0, tok.numel(), vocab, d, scale, ws.data_ptr(),
                                                n.value, handle), "prm_embedding_backward")
    return grad
