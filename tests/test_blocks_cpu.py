"""CPU checks of the transformer-block operators: every gradient of the fp64
oracle against central differences of its forward function, the C ABI's
declarations and argument refusals (none reaches the device), and the tensor
API's refusals."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from matrix_aware_optimizer_gb300 import blocks, build, native as N
from oracle import blocks as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return N.load()


# ------------------------------------------------------------- differences
def _differences(f, args, which, weight, h=1e-5):
    """d(sum(weight * f(*args))) / d args[which] by central differences."""
    a = args[which]
    out = np.zeros_like(a)
    for i in np.ndindex(*a.shape):
        keep = a[i]
        a[i] = keep + h
        up = (f(*args) * weight).sum()
        a[i] = keep - h
        down = (f(*args) * weight).sum()
        a[i] = keep
        out[i] = (up - down) / (2 * h)
    return out


def _close(a, b):
    # truncation h^2 f''' / 6 ~ 1e-10 and cancellation 2^-53 |f| / h ~ 1e-10, with a margin of 100
    assert np.abs(a - b).max() <= 1e-8 * max(1.0, np.abs(b).max())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_ffn_gradient_against_differences(act):
    rng = np.random.default_rng(1)
    x, wg, wu, wd, dy = (rng.standard_normal(s) for s in ((3, 4), (5, 4), (5, 4), (4, 5), (3, 4)))
    got = O.gated_ffn_backward(dy, x, wg, wu, wd, act)
    for k, g in enumerate(got):
        _close(g, _differences(lambda *a: O.gated_ffn(*a, act), [x, wg, wu, wd], k, dy))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("post,gate,pre,mod", [(0, 0, 0, 0), (1, 0, 1, 0), (0, 1, 0, 1), (1, 1, 1, 1)])
def test_norm_gradient_against_differences(kind, post, gate, pre, mod):
    rng = np.random.default_rng(2)
    B, L, d, alpha, eps = 2, 3, 5, 0.7, 1e-3
    x, z, dy, dr = (rng.standard_normal((B, L, d)) for _ in range(4))
    w_post, w_pre = (rng.standard_normal(d) if on else None for on in (post, pre))
    g = rng.standard_normal((B, d)) if gate else None
    sc, sh = ((rng.standard_normal((B, d)) for _ in range(2)) if mod else (None, None))
    r = O.block_join(x, z, kind, alpha, eps, w_post, g)
    got = O.block_backward(dy, dr, r, z, kind, alpha, eps, w_post, g, w_pre, sc, sh)

    def whole(x, z, w_post, g, w_pre, sc, sh):
        r = O.block_join(x, z, kind, alpha, eps, w_post, g)
        return np.stack([r, O.block_next(r, kind, eps, w_pre, sc, sh)])

    args = [x, z, w_post, g, w_pre, sc, sh]
    for k, name in enumerate(("dx", "dz", "dpost", "dgate", "dpre", "dscale", "dshift")):
        if args[k] is None:
            assert got[name] is None
        else:
            _close(got[name], _differences(whole, args, k, np.stack([dr, dy])))


def test_embedding_gradient_against_differences():
    rng = np.random.default_rng(3)
    tok = np.array([2, 0, 2, -1, 7, 3, 2])
    table, dout = rng.standard_normal((4, 3)), rng.standard_normal((7, 3))
    _close(O.embedding_backward(dout, tok, 4, 1.5),
           _differences(lambda t: O.embedding(tok, t, 1.5), [table], 0, dout))


# --------------------------------------------------------------------- ABI
def test_every_declared_symbol_is_exported_and_bound(lib):
    with open(os.path.join(ROOT, "include", "prm_blocks.h")) as f:
        text = f.read()
    names = sorted(set(re.findall(r"PRM_API\s+[\w\s\*]+?\b(prm_\w+)\s*\(", text)))
    assert len(names) == 10
    for name in names:
        assert hasattr(lib, name) and name in N.SIGNATURES, name


def test_norm_descriptor_layout():
    # 3 int64, 3 int32, 2 float, 1 int32, 5 pointers, 3 int64
    assert ctypes.sizeof(N.prm_block_norm_desc) == 24 + 24 + 40 + 24
    assert N.prm_block_norm_desc.post_weight.offset == 48


def _ffn(lib, x=256, ldx=64, wg=256, wu=256, wd=256, y=256, saved=256, ws=256, n=1 << 30, T=4, d=64, f=64,
         act=0, dtype=N.PRM_BF16):
    return lib.prm_gated_ffn_forward(x, ldx, wg, wu, wd, y, saved, ws, n, T, d, f, act, dtype, None)


def test_ffn_refusals(lib):
    assert _ffn(lib, T=0) == N.PRM_OK
    assert _ffn(lib, T=-1) == N.PRM_ERR_INVALID_ARG
    assert _ffn(lib, act=3) == N.PRM_ERR_INVALID_ARG
    assert _ffn(lib, dtype=N.PRM_FP32) == N.PRM_ERR_INVALID_ARG
    assert _ffn(lib, d=0) == N.PRM_ERR_INVALID_ARG
    assert _ffn(lib, d=12) == N.PRM_ERR_ALIGNMENT
    assert _ffn(lib, f=65) == N.PRM_ERR_ALIGNMENT
    assert _ffn(lib, ldx=56) == N.PRM_ERR_INVALID_ARG
    assert _ffn(lib, ldx=68) == N.PRM_ERR_ALIGNMENT
    assert _ffn(lib, x=264) == N.PRM_ERR_ALIGNMENT
    assert _ffn(lib, saved=272) == N.PRM_ERR_ALIGNMENT
    assert _ffn(lib, wu=None) == N.PRM_ERR_INVALID_ARG
    assert _ffn(lib, ws=None) == N.PRM_ERR_WORKSPACE
    assert _ffn(lib, n=10) == N.PRM_ERR_WORKSPACE
    assert _ffn(lib, T=1 << 31) == N.PRM_ERR_UNSUPPORTED
    assert _ffn(lib, T=1 << 30, f=1 << 23) == N.PRM_ERR_UNSUPPORTED   # more tiles than 32 bits count

    def back(dy=256, lddy=64, saved=256, dx=256, dg=256, du=256, dd=256, n=1 << 30, T=4):
        return lib.prm_gated_ffn_backward(dy, lddy, 256, 64, 256, 256, 256, saved, dx, dg, du, dd, 256, n, T, 64, 64,
                                          0, N.PRM_BF16, None)
    assert back(du=None) == N.PRM_ERR_INVALID_ARG       # some but not all weight gradients
    assert back(saved=None) == N.PRM_ERR_INVALID_ARG
    assert back(lddy=60) == N.PRM_ERR_INVALID_ARG
    assert back(dx=264) == N.PRM_ERR_ALIGNMENT
    assert back(n=5) == N.PRM_ERR_WORKSPACE
    assert back(dx=None, dg=None, du=None, dd=None) == N.PRM_OK  # nothing is wanted
    n = ctypes.c_size_t()
    assert lib.prm_gated_ffn_sizes(4, 64, 63, n, n, n) == N.PRM_ERR_ALIGNMENT
    assert lib.prm_gated_ffn_sizes(4, 64, 64, n, None, n) == N.PRM_ERR_INVALID_ARG


def test_ffn_saved_size(lib):
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.prm_gated_ffn_sizes(8192, 2048, 8192, a, b, c) == N.PRM_OK
    assert a.value == 8 * 8192 * 8192      # 2 bytes of h, 6 of g and u
    assert lib.prm_gated_ffn_sizes(0, 64, 64, a, b, c) == N.PRM_OK
    assert a.value == 0 and c.value == 0


def _desc(**kw):
    v = dict(rows=8, rows_per_sample=4, d=64, kind=0, stream_dtype=N.PRM_FP32, block_dtype=N.PRM_BF16, alpha=1.0,
             eps=1e-6, reserved=0, post_weight=None, pre_weight=None, gate=None, scale=None, shift=None, gate_ld=0,
             scale_ld=0, shift_ld=0)
    v.update(kw)
    return N.prm_block_norm_desc(*(v[k] for k, _ in N.prm_block_norm_desc._fields_))


def test_norm_refusals(lib):
    def fwd(x=16, z=16, r=16, y=16, stats=16, **kw):
        return lib.prm_block_norm_forward(_desc(**kw), x, z, r, y, stats, None)
    assert fwd(rows=0) == N.PRM_OK
    assert fwd(kind=2) == N.PRM_ERR_INVALID_ARG
    assert fwd(reserved=1) == N.PRM_ERR_INVALID_ARG
    assert fwd(alpha=float("nan")) == N.PRM_ERR_INVALID_ARG
    assert fwd(eps=-1.0) == N.PRM_ERR_INVALID_ARG
    assert fwd(stream_dtype=N.PRM_BF16, block_dtype=N.PRM_FP16) == N.PRM_ERR_INVALID_ARG
    assert fwd(stream_dtype=N.PRM_BF16, block_dtype=N.PRM_FP32) == N.PRM_ERR_INVALID_ARG
    assert fwd(rows_per_sample=3) == N.PRM_ERR_SHAPE
    assert fwd(d=0) == N.PRM_ERR_SHAPE
    assert fwd(d=8193) == N.PRM_ERR_UNSUPPORTED
    assert fwd(rows=1 << 32, rows_per_sample=1 << 31) == N.PRM_ERR_UNSUPPORTED
    assert fwd(gate=16, gate_ld=63) == N.PRM_ERR_SHAPE
    assert fwd(x=None) == N.PRM_ERR_INVALID_ARG
    assert fwd(r=None) == N.PRM_ERR_INVALID_ARG
    assert fwd(z=None, y=None) == N.PRM_ERR_INVALID_ARG
    assert fwd(z=None, alpha=0.5) == N.PRM_ERR_INVALID_ARG
    assert fwd(z=None, gate=16, gate_ld=64) == N.PRM_ERR_INVALID_ARG
    assert fwd(y=None, pre_weight=16) == N.PRM_ERR_INVALID_ARG
    assert fwd(stats=8) == N.PRM_ERR_ALIGNMENT
    assert lib.prm_block_norm_forward(None, 16, 16, 16, 16, 16, None) == N.PRM_ERR_INVALID_ARG

    def back(dy=16, dr=16, r=16, z=16, stats=16, dx=16, dz=16, dpost=None, dgate=None, dpre=None, ws=None, n=0, **kw):
        return lib.prm_block_norm_backward(_desc(**kw), dy, dr, r, z, stats, dx, dz, dpost, dgate, dpre, None, None,
                                           ws, n, None)
    assert back(rows=0) == N.PRM_OK
    assert back(dy=None, dr=None) == N.PRM_ERR_INVALID_ARG
    assert back(r=None) == N.PRM_ERR_INVALID_ARG
    assert back(z=None) == N.PRM_ERR_INVALID_ARG            # dz without z
    assert back(pre_weight=16) == N.PRM_ERR_INVALID_ARG     # no place for its gradient
    assert back(gate=16, gate_ld=64) == N.PRM_ERR_INVALID_ARG
    assert back(pre_weight=16, dpre=16) == N.PRM_ERR_WORKSPACE
    assert back(pre_weight=16, dpre=16, ws=8, n=1 << 20) == N.PRM_ERR_ALIGNMENT
    n = ctypes.c_size_t(3)
    assert lib.prm_block_norm_workspace(_desc(), n) == N.PRM_OK and n.value == 0
    assert lib.prm_block_norm_workspace(_desc(pre_weight=16), n) == N.PRM_OK and n.value > 0
    assert lib.prm_block_norm_workspace(_desc(), None) == N.PRM_ERR_INVALID_ARG


def test_embedding_refusals(lib):
    def fwd(tok=16, nb=8, table=16, td=0, out=16, od=0, T=4, V=10, d=8, scale=1.0):
        return lib.prm_embedding_forward(tok, nb, table, td, out, od, T, V, d, scale, None)
    assert fwd(T=0) == N.PRM_OK
    assert fwd(nb=2) == N.PRM_ERR_INVALID_ARG
    assert fwd(td=5) == N.PRM_ERR_INVALID_ARG
    assert fwd(V=0) == N.PRM_ERR_INVALID_ARG
    assert fwd(d=0) == N.PRM_ERR_INVALID_ARG
    assert fwd(T=-1) == N.PRM_ERR_INVALID_ARG
    assert fwd(scale=float("inf")) == N.PRM_ERR_INVALID_ARG
    assert fwd(table=None) == N.PRM_ERR_INVALID_ARG
    assert fwd(T=1 << 31) == N.PRM_ERR_UNSUPPORTED

    def back(dout=16, grad=16, ws=256, n=1 << 30, T=4, V=10, d=8, dd=0, gd=0):
        return lib.prm_embedding_backward(dout, dd, 16, 8, grad, gd, 1, T, V, d, 1.0, ws, n, None)
    assert back(T=0) == N.PRM_OK    # accumulating nothing
    assert back(grad=None) == N.PRM_ERR_INVALID_ARG
    assert back(dout=None) == N.PRM_ERR_INVALID_ARG
    assert back(gd=7) == N.PRM_ERR_INVALID_ARG
    assert back(n=1) == N.PRM_ERR_WORKSPACE
    assert back(ws=264) == N.PRM_ERR_ALIGNMENT
    assert back(V=1 << 31) == N.PRM_ERR_UNSUPPORTED
    n = ctypes.c_size_t()
    assert lib.prm_embedding_backward_workspace(4, 10, 8, None) == N.PRM_ERR_INVALID_ARG
    assert lib.prm_embedding_backward_workspace(0, 10, 8, n) == N.PRM_OK and n.value == 0


def test_tensor_api_refuses_cpu_tensors_and_wrong_shapes():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w, wd = torch.zeros(32, 64, dtype=torch.bfloat16), torch.zeros(64, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        blocks.gated_ffn(x, w, w, wd)
    with pytest.raises(ValueError):
        blocks.gated_ffn(x, w, w, wd, act="relu")
    with pytest.raises(ValueError):
        blocks.embedding(torch.zeros(3, dtype=torch.int64), torch.zeros(5, 8))
    with pytest.raises(ValueError):
        blocks.embedding_backward(torch.zeros(3, 8), torch.zeros(3, dtype=torch.int64), 5, accumulate=True)
    with pytest.raises(ValueError):
        blocks.block_norm(x, alpha=0.5)
    with pytest.raises(ValueError):
        blocks.block_norm(x, x)
    with pytest.raises(ValueError):
        blocks.block_norm_backward(x, None, x, x, torch.zeros(4, 4))
    with pytest.raises(ValueError):
        blocks.block_norm_backward(None, None, x, x, torch.zeros(4, 4))
