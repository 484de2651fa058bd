"""torch glue over include/prm_blocks.h: the operators of a transformer block
whose parameters the optimizer updates. Each operator is a forward and a
backward call on tensors; PyTorch supplies memory and the stream, every
arithmetic step runs in libprm. The calls are outside autograd: what they
return has no graph, whether or not the inputs require gradients, and the
backward calls are the caller's to make. Outputs and workspaces are allocated
on the stream the call runs on (`stream`, or the current one of the tensors'
device). Work that a call depends on and that runs on another stream is the
caller's to order, as with any torch operation."""
from __future__ import annotations

import contextlib
import ctypes
import functools
import struct
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import native as N

_DTYPE = {torch.float32: N.PRM_FP32, torch.bfloat16: N.PRM_BF16, torch.float16: N.PRM_FP16}
_HALF = (torch.bfloat16, torch.float16)
_DESC = struct.Struct("=3q3i2fi5Q3q")  # prm_block_norm_desc
assert _DESC.size == ctypes.sizeof(N.prm_block_norm_desc)
_ACT = {"silu": N.PRM_ACT_SILU, "gelu": N.PRM_ACT_GELU, "gelu_tanh": N.PRM_ACT_GELU_TANH}
_KIND = {"rms": N.PRM_NORM_RMS, "layer": N.PRM_NORM_LAYER}


_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


@contextlib.contextmanager
def _elsewhere(device: int, stream: Optional[torch.cuda.Stream], *tensors: Optional[torch.Tensor]):
    """Makes the tensors' device and the given stream the current ones, so
    that what a call allocates belongs to the stream it runs on, and tells the
    allocator that the given stream uses the call's tensors: their memory is
    not handed out again before its work is done."""
    with torch.cuda.device(device), torch.cuda.stream(stream):  # (a None stream changes nothing)
        yield
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _is_elsewhere(device: int, stream) -> bool:
    if stream is not None and stream.device.index != device:
        raise ValueError("stream must be one of the tensors' device")
    return stream is not None or device != _current_device()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def blocks_sync_status(stream: Optional[torch.cuda.Stream] = None) -> None:
    """Waits for the stream and raises if a device-side wait of a block
    operator gave up on the stream's device."""
    s = stream if stream is not None else torch.cuda.current_stream()
    with torch.cuda.device(s.device):  # the error word is the current device's
        N.check(N.load().prm_blocks_sync_status(s.cuda_stream), "prm_blocks_sync_status")


# ---------------------------------------------------------------- gated FFN
class FfnSaved(NamedTuple):
    """What gated_ffn leaves for gated_ffn_backward: h, g and u of one pass
    (8 bytes per token and feature), in the library's own layout, and the
    features, activation and type it was made with."""
    buffer: torch.Tensor
    tokens: int
    features: Optional[int] = None
    act: Optional[str] = None
    dtype: Optional[torch.dtype] = None


def _rows16(t: torch.Tensor, d: int) -> Tuple[torch.Tensor, int]:
    """t as rows of d elements with a pitch TMA can read: (tensor, pitch).
    Other layouts are copied."""
    if t.dim() != 2:
        t = t.reshape(-1, d)
    pitch, unit = t.stride()
    if unit != 1 or pitch < d or pitch % 8 or t.data_ptr() % 16:
        t = t.clone(memory_format=torch.contiguous_format)
        pitch = d
    return t, pitch


def _ffn_check(x, w_gate, w_up, w_down, act):
    dt, device = x.dtype, x.get_device()
    if act not in _ACT:
        raise ValueError(f"act must be one of {sorted(_ACT)}")
    if dt not in _HALF or device < 0:
        raise ValueError("x must be a bfloat16 or float16 CUDA tensor")
    shape = w_gate.shape
    d = x.shape[-1]
    if len(shape) != 2 or shape[1] != d or w_up.shape != shape or w_down.shape != (d, shape[0]):
        raise ValueError("w_gate and w_up must be f x d and w_down d x f, d the last extent of x")
    for w in (w_gate, w_up, w_down):
        if w.dtype is not dt or w.get_device() != device or not w.is_contiguous():
            raise ValueError("weights must be contiguous, of x's type and on its device")
    if d % 8 or shape[0] % 8:
        raise ValueError("d and f must be multiples of 8")
    return d, shape[0], device


@functools.lru_cache(maxsize=256)
def _ffn_sizes(tokens, d, f):
    saved, forward, backward = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    N.check(N.load().prm_gated_ffn_sizes(tokens, d, f, saved, forward, backward), "prm_gated_ffn_sizes")
    return saved.value, forward.value, backward.value


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, act: str = "silu",
              save: bool = False, stream: Optional[torch.cuda.Stream] = None):
    """Gated feed-forward block, y = (act(x w_gate^T) * (x w_up^T)) w_down^T.

    x: [..., d] bf16 or fp16; w_gate, w_up: [f, d]; w_down: [d, f], all of x's
    type; d and f multiples of 8. act: "silu", "gelu" (erf) or "gelu_tanh".
    Returns y, or (y, saved) with save=True, saved for gated_ffn_backward
    (autograd does not see the call).
    """
    d, f, device = _ffn_check(x, w_gate, w_up, w_down, act)
    if _is_elsewhere(device, stream):
        with _elsewhere(device, stream, x, w_gate, w_up, w_down):
            return gated_ffn(x, w_gate, w_up, w_down, act, save)
    x2, ldx = _rows16(x, d)
    tokens = x2.shape[0]
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    n_saved, n_ws, _ = _ffn_sizes(tokens, d, f)
    saved = x.new_empty(n_saved, dtype=torch.uint8) if save else None
    ws = x.new_empty(n_ws, dtype=torch.uint8)
    rc = N.load().prm_gated_ffn_forward(x2.data_ptr(), ldx, w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
                                        y.data_ptr(), saved.data_ptr() if save else None, ws.data_ptr(), n_ws, tokens,
                                        d, f, _ACT[act], _DTYPE[x.dtype], _raw_stream(device))
    if rc:
        N.check(rc, "prm_gated_ffn_forward")
    return (y, FfnSaved(saved, tokens, f, act, x.dtype)) if save else y


def gated_ffn_backward(dy: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                       w_down: torch.Tensor, saved: FfnSaved, act: str = "silu", need_dx: bool = True,
                       grads: Optional[Sequence[torch.Tensor]] = None,
                       stream: Optional[torch.cuda.Stream] = None):
    """Gradients of gated_ffn: (dx, dw_gate, dw_up, dw_down), all of x's type.

    grads: three tensors of the weights' shapes and type to write the weight
    gradients into (they are overwritten), e.g. the buffers that PeriodicRowMuon
    has registered where the weights are bf16; it takes no fp16 gradients, which
    the caller converts. act and the weights are those of the pass that made
    `saved`. dx is None with need_dx=False.
    """
    d, f, device = _ffn_check(x, w_gate, w_up, w_down, act)
    if dy.shape != x.shape or dy.dtype is not x.dtype or dy.get_device() != device:
        raise ValueError("dy must have x's shape, type and device")
    if saved.features not in (None, f) or saved.act not in (None, act) or saved.dtype not in (None, x.dtype):
        raise ValueError("saved comes from a pass with other weights, another act or another type")
    if _is_elsewhere(device, stream):
        with _elsewhere(device, stream, dy, x, w_gate, w_up, w_down, saved.buffer, *(grads or ())):
            return gated_ffn_backward(dy, x, w_gate, w_up, w_down, saved, act, need_dx, grads)
    x2, ldx = _rows16(x, d)
    dy2, lddy = _rows16(dy, d)
    tokens = x2.shape[0]
    n_saved, _, n_ws = _ffn_sizes(tokens, d, f)
    if saved.tokens != tokens or saved.buffer.numel() != n_saved:
        raise ValueError("saved does not belong to this x")
    if grads is None:
        dg, du, dd = torch.empty_like(w_gate), torch.empty_like(w_up), torch.empty_like(w_down)
    else:
        dg, du, dd = grads
        for g, w in ((dg, w_gate), (du, w_up), (dd, w_down)):
            if g.shape != w.shape or g.dtype is not w.dtype or g.get_device() != device or not g.is_contiguous():
                raise ValueError("grads must be three contiguous tensors of the weights' shapes and type")
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if need_dx else None
    ws = x.new_empty(n_ws, dtype=torch.uint8)
    rc = N.load().prm_gated_ffn_backward(dy2.data_ptr(), lddy, x2.data_ptr(), ldx, w_gate.data_ptr(),
                                         w_up.data_ptr(), w_down.data_ptr(), saved.buffer.data_ptr(), _ptr(dx),
                                         dg.data_ptr(), du.data_ptr(), dd.data_ptr(), ws.data_ptr(), n_ws, tokens, d,
                                         f, _ACT[act], _DTYPE[x.dtype], _raw_stream(device))
    if rc:
        N.check(rc, "prm_gated_ffn_backward")
    return dx, dg, du, dd


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
    dt, device = ref.dtype, ref.get_device()
    if kind not in _KIND:
        raise ValueError(f"kind must be one of {sorted(_KIND)}")
    if dt not in _DTYPE or block_dtype not in _DTYPE:
        raise ValueError("tensors must be float32, bfloat16 or float16")
    if dt is not torch.float32 and dt is not block_dtype:
        raise ValueError("a 16-bit residual stream needs a block of the same type")
    d = ref.shape[-1]
    rows = ref.numel() // d if d else 0
    for w in (post_weight, pre_weight):
        if w is not None and (w.dtype is not torch.float32 or w.get_device() != device or w.shape != (d,)
                              or not w.is_contiguous()):
            raise ValueError("post_weight and pre_weight must be contiguous float32 tensors of d elements")
    samples = 0
    ptrs, lds = [0, 0, 0], [0, 0, 0]
    for k, m in enumerate((gate, scale, shift)):
        if m is None:
            continue
        shape = m.shape
        if len(shape) != 2 or shape[1] != d or m.dtype is not block_dtype or m.get_device() != device:
            raise ValueError("gate, scale and shift must be samples x d tensors of the block's type")
        pitch, unit = m.stride()
        if unit != 1 or (shape[0] > 1 and pitch < d):
            raise ValueError("gate, scale and shift must have unit column stride")
        if samples and shape[0] != samples:
            raise ValueError("gate, scale and shift must have the same number of samples")
        samples = shape[0]
        if samples == 0 or rows % samples:
            raise ValueError("the samples must divide the rows")
        ptrs[k] = m.data_ptr()
        lds[k] = pitch if pitch > d else d
    packed = _DESC.pack(rows, (rows // samples if samples else rows) or 1, d, _KIND[kind], _DTYPE[dt],
                        _DTYPE[block_dtype], alpha, eps, 0, 0 if post_weight is None else post_weight.data_ptr(),
                        0 if pre_weight is None else pre_weight.data_ptr(), *ptrs, *lds)
    return N.prm_block_norm_desc.from_buffer_copy(packed), rows


def _norm_rows(t, like, dtype, name):
    if t.dtype is not dtype or t.shape != like.shape or t.get_device() != like.get_device():
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

    Returns (r, y, stats), stats for block_norm_backward (autograd does not
    see the call).
    """
    device = x.get_device()
    if device < 0:
        raise ValueError("x must be a CUDA tensor")
    block = z.dtype if z is not None else (dtype if dtype is not None else x.dtype)
    if dtype is not None and dtype is not block:
        raise ValueError("dtype must be z's")
    if z is None and (join_only or alpha != 1.0 or gate is not None or post_weight is not None):
        raise ValueError("alpha, gate, post_weight and join_only need z")
    if join_only and (pre_weight is not None or scale is not None or shift is not None):
        raise ValueError("pre_weight, scale and shift belong to the norm that join_only leaves out")
    if _is_elsewhere(device, stream):
        with _elsewhere(device, stream, x, z, post_weight, gate, pre_weight, scale, shift):
            return block_norm(x, z, kind, alpha, post_weight, gate, pre_weight, scale, shift, eps, dtype, join_only)
    if not x.is_contiguous():
        x = x.contiguous()
    if z is not None:
        z = _norm_rows(z, x, block, "z")
    desc, rows = _norm_desc(x, block, kind, alpha, eps, post_weight, gate, pre_weight, scale, shift)
    r = torch.empty_like(x) if z is not None else x
    y = None if join_only else torch.empty_like(x, dtype=block)
    stats = x.new_empty((rows, 4), dtype=torch.float32)
    rc = N.load().prm_block_norm_forward(desc, x.data_ptr(), _ptr(z), r.data_ptr(), _ptr(y), stats.data_ptr(),
                                         _raw_stream(device))
    if rc:
        N.check(rc, "prm_block_norm_forward")
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
    device = r.get_device()
    if device < 0:
        raise ValueError("r must be a CUDA tensor")
    if _is_elsewhere(device, stream):
        with _elsewhere(device, stream, dy, dr, r, z, stats, post_weight, gate, pre_weight, scale, shift):
            return block_norm_backward(dy, dr, r, z, stats, kind, alpha, post_weight, gate, pre_weight, scale, shift,
                                       need_dx)
    block = z.dtype if z is not None else dy.dtype if dy is not None else r.dtype
    desc, rows = _norm_desc(r, block, kind, alpha, 0.0, post_weight, gate, pre_weight, scale, shift)
    if not r.is_contiguous():
        r = r.contiguous()
    if dy is not None:
        dy = _norm_rows(dy, r, block, "dy")
    if dr is not None:
        dr = _norm_rows(dr, r, r.dtype, "dr")
    if z is not None:
        z = _norm_rows(z, r, block, "z")
    if stats.shape != (rows, 4) or stats.dtype is not torch.float32 or stats.get_device() != device \
            or not stats.is_contiguous():
        raise ValueError("stats must be the tensor block_norm returned")
    out = BlockNormGrads(torch.empty_like(r) if need_dx else None, None if z is None else torch.empty_like(z),
                         *(None if p is None else torch.empty(p.shape, dtype=p.dtype, device=p.device)
                           for p in (post_weight, gate, pre_weight, scale, shift)))
    if rows == 0:
        for t in out[2:]:
            if t is not None:
                t.zero_()
        return out
    lib = N.load()
    n = ctypes.c_size_t()
    rc = lib.prm_block_norm_workspace(desc, n)
    if rc:
        N.check(rc, "prm_block_norm_workspace")
    ws = r.new_empty(n.value, dtype=torch.uint8) if n.value else None
    rc = lib.prm_block_norm_backward(desc, _ptr(dy), _ptr(dr), r.data_ptr(), _ptr(z), stats.data_ptr(),
                                     *(None if t is None else t.data_ptr() for t in out), _ptr(ws), n.value,
                                     _raw_stream(device))
    if rc:
        N.check(rc, "prm_block_norm_backward")
    return out


# ---------------------------------------------------------------- embedding
def _tokens(tokens: torch.Tensor) -> torch.Tensor:
    if tokens.dtype is not torch.int64 and tokens.dtype is not torch.int32:
        raise ValueError("tokens must be an int64 or int32 CUDA tensor")
    return tokens if tokens.is_contiguous() else tokens.contiguous()


def embedding(tokens: torch.Tensor, table: torch.Tensor, scale: float = 1.0, dtype: Optional[torch.dtype] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """scale * table[tokens], as `dtype` (default: the table's). table: [vocab,
    d] fp32, bf16 or fp16. A token outside [0, vocab) is padding: a zero row.
    Autograd does not see the call: embedding_backward gives table's gradient."""
    device = table.get_device()
    if dtype is None:
        dtype = table.dtype
    if device < 0 or table.dim() != 2 or table.dtype not in _DTYPE or dtype not in _DTYPE \
            or not table.is_contiguous() or tokens.get_device() != device:
        raise ValueError("table must be a contiguous vocab x d CUDA tensor of float32, bfloat16 or float16")
    if _is_elsewhere(device, stream):
        with _elsewhere(device, stream, tokens, table):
            return embedding(tokens, table, scale, dtype)
    tok = _tokens(tokens)
    vocab, d = table.shape
    out = table.new_empty((*tokens.shape, d), dtype=dtype)
    rc = N.load().prm_embedding_forward(tok.data_ptr(), tok.element_size(), table.data_ptr(), _DTYPE[table.dtype],
                                        out.data_ptr(), _DTYPE[dtype], tok.numel(), vocab, d, scale,
                                        _raw_stream(device))
    if rc:
        N.check(rc, "prm_embedding_forward")
    return out


@functools.lru_cache(maxsize=256)
def _embedding_workspace(tokens, vocab, d):
    n = ctypes.c_size_t()
    N.check(N.load().prm_embedding_backward_workspace(tokens, vocab, d, n), "prm_embedding_backward_workspace")
    return n.value


def embedding_backward(dout: torch.Tensor, tokens: torch.Tensor, vocab: int, scale: float = 1.0,
                       dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                       accumulate: bool = False, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Gradient of embedding's table [vocab, d] as `dtype`: the sum of dout's
    rows per token, in the order of the tokens (deterministic), times scale;
    rows without tokens are zero. out: a tensor to write it into (its type
    takes `dtype`'s place); accumulate=True adds to what out holds, e.g. the
    output layer's gradient of a tied table."""
    device = dout.get_device()
    if device < 0 or dout.dtype not in _DTYPE or dout.shape[:-1] != tokens.shape or tokens.get_device() != device:
        raise ValueError("dout must be tokens' shape x d, float32, bfloat16 or float16, on the tokens' device")
    d = dout.shape[-1]
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        if dtype not in _DTYPE:
            raise ValueError("dtype must be float32, bfloat16 or float16")
    elif out.shape != (vocab, d) or out.dtype not in _DTYPE or out.get_device() != device or not out.is_contiguous():
        raise ValueError("out must be a contiguous vocab x d tensor of float32, bfloat16 or float16")
    if _is_elsewhere(device, stream):
        with _elsewhere(device, stream, dout, tokens, out):
            return embedding_backward(dout, tokens, vocab, scale, dtype, out, accumulate)
    tok = _tokens(tokens)
    if not dout.is_contiguous():
        dout = dout.contiguous()
    grad = dout.new_empty((vocab, d), dtype=dtype) if out is None else out
    n_tokens = tok.numel()
    n_ws = _embedding_workspace(n_tokens, vocab, d)
    ws = dout.new_empty(n_ws, dtype=torch.uint8)
    rc = N.load().prm_embedding_backward(dout.data_ptr(), _DTYPE[dout.dtype], tok.data_ptr(), tok.element_size(),
                                         grad.data_ptr(), _DTYPE[grad.dtype], 1 if accumulate else 0, n_tokens, vocab,
                                         d, scale, ws.data_ptr(), n_ws, _raw_stream(device))
    if rc:
        N.check(rc, "prm_embedding_backward")
    return grad
