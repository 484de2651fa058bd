"""Numerics of the linear layer against the fp64 oracle, at the sizes, layouts
and values where its kernels change path or could go wrong.

Tolerances. U is the largest relative error of one rounding to a type (2^-8
for bf16, 2^-11 for fp16, 2^-24 for fp32)."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_gb300 as prm
from matrix_aware_optimizer_gb300 import native as N
from oracle import attention as O

from .gpu_helpers import ensure_built, host64

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, FP32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()
    N.load()
    yield
    prm.blocks_sync_status()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(gen, *shape, dtype=FP32, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).cuda()


def _linear_inputs(T, k, n, dtype=BF16, seed=0):
    g = _gen(seed + T + 3 * k + 5 * n)
    return (_rand(g, T, k, dtype=dtype), _rand(g, n, k, dtype=dtype, scale=k ** -0.5), _rand(g, n, scale=0.3),
            _rand(g, T, n), _rand(g, T, n))


def _check_linear(x, w, b, res, dy, act, calls=None):
    """res: None or of the type y has; dy of y's type. Compares element by
    element: a sum of n products in fp32 is off by n + 1 steps of 2^-24 of the
    sum of the products' sizes; the activations' slopes are below 1.13 and those
    of their derivatives below 0.8, with 8 and 12 steps for the functions. dg is
    rounded once as an operand (u), so are the results; the bias' gradient is an
    fp32 sum of fp32 terms."""
    u, e, yt = U[x.dtype], 2.0 ** -24, dy.dtype
    if calls is None:
        y, saved = prm.linear(x, w, b, act=act, residual=res, save=True)
        calls = (y,) + prm.linear_backward(dy, x, w, saved, act=act)
        assert torch.equal(prm.linear(x, w, b, act=act, residual=res), y)
    T, k, n = x.shape[0], x.shape[1], w.shape[0]
    hx, hw, hd = host64(x), host64(w), host64(dy)
    hb = None if b is None else host64(b)
    hr = None if res is None else host64(res)
    g = hx @ hw.T + (0.0 if b is None else hb)
    g_off = (k + 2) * e * (np.abs(hx) @ np.abs(hw).T + (0.0 if b is None else np.abs(hb)))
    tiny = 2.0 ** -25 if x.dtype is FP16 else 2.0 ** -126
    slope, curve = (1.0, 0.0) if act is None else (1.13, 0.8)
    want = O.linear(hx, hw, hb, act, hr)
    y_off = slope * g_off + (0.0 if act is None else 8 * e * (1.0 + np.abs(g)))
    y_off = y_off + 2 * e * (np.abs(want) + (0.0 if hr is None else np.abs(hr)))
    dx, dw, db = O.linear_backward(hd, hx, hw, hb, act)
    dg = hd if act is None else hd * O.activation(g, act)[1]
    dg_off = np.abs(hd) * (curve * g_off + (0.0 if act is None else 12 * e))
    dg_all = dg_off + (u if act is not None or yt is not x.dtype else 0.0) * (np.abs(dg) + dg_off) + tiny
    size = np.abs(dg) + dg_all
    for name, got, ref, bound, last in (
            ("y", calls[0], want, y_off, U[yt]),
            ("dx", calls[1], dx, dg_all @ np.abs(hw) + (n + 2) * e * (size @ np.abs(hw)), u),
            ("dw", calls[2], dw, dg_all.T @ np.abs(hx) + (T + 2) * e * (size.T @ np.abs(hx)), u),
            ("db", calls[3], db, dg_off.sum(0) + (T + 2) * e * size.sum(0), U[FP32])):
        got = host64(got)
        assert np.isfinite(got).all(), name
        err = np.abs(got - ref) - (bound + last * (np.abs(ref) + bound) + tiny)
        assert (err <= 0).all(), (name, err.max())
    return calls


# one token and the few that run on CUDA cores, row and column tiles and their edges, the shortest rows, sums shorter
# than one slice, sums split over CTA pairs
LINEAR_SHAPES = [(1, 64, 256), (1, 8, 8), (2, 2048, 1024), (3, 264, 72), (4, 512, 4096), (5, 72, 40), (8, 1032, 2064),
                 (9, 64, 96), (33, 520, 24), (64, 2048, 64), (127, 256, 128), (129, 264, 520), (255, 8, 1000),
                 (256, 256, 256), (257, 200, 328), (300, 1000, 2664), (513, 512, 264), (1030, 64, 64),
                 (700, 4104, 72), (2049, 72, 2568)]


@pytest.mark.parametrize("T,k,n", LINEAR_SHAPES)
def test_linear_shapes(T, k, n):
    x, w, b, _, dy = _linear_inputs(T, k, n)
    _check_linear(x, w, b, None, dy.to(BF16), None)


@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("act", [None, "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("residual", [None, "same", "fp32"])
def test_linear_epilogues(T, act, dtype, residual):
    x, w, b, res, dy = _linear_inputs(T, 136, 264, dtype)
    yt = FP32 if residual == "fp32" else dtype
    res, dy = None if residual is None else res.to(yt), dy.to(yt)
    _check_linear(x, w, b, res, dy, act)
    _check_linear(x, w, None, res, dy, act)


@pytest.mark.parametrize("T,k,n", [(64, 4096, 256), (300, 2048, 512), (600, 5000, 264), (520, 512, 1024)])
@pytest.mark.parametrize("act", [None, "gelu"])
def test_linear_in_parts(T, k, n, act):
    x, w, b, res, dy = _linear_inputs(T, k, n)
    _check_linear(x, w, b, res, dy, act)
    _check_linear(x, w, b, res.to(BF16), dy.to(BF16), act)


# enough tokens for the 256 x 256 tiles, ragged ones, with and without tiles of a last round in parts
@pytest.mark.parametrize("T,k,n", [(5120, 512, 4096), (4099, 72, 4104)])
@pytest.mark.parametrize("act", [None, "gelu_tanh"])
def test_linear_large_tiles(T, k, n, act):
    x, w, b, res, dy = _linear_inputs(T, k, n)
    _check_linear(x, w, b, None, dy.to(BF16), act)
    _check_linear(x, w, b, res.to(BF16), dy.to(BF16), act)
    _check_linear(x, w, b, res, dy, act)


def test_linear_layouts():
    x, w, b, res, dy = _linear_inputs(60, 128, 192)
    res, dy = res.to(BF16), dy.to(BF16)
    want = _check_linear(x, w, b, res, dy, "silu")

    def same(x, res, dy):
        y, saved = prm.linear(x, w, b, act="silu", residual=res, save=True)
        assert y.shape == dy.shape
        for a, c in zip((y,) + prm.linear_backward(dy, x, w, saved, act="silu"), want):
            assert torch.equal(a.reshape(c.shape), c)

    same(x.view(3, 20, 128), res.view(3, 20, 192), dy.view(3, 20, 192))
    wide = torch.zeros(60, 520, dtype=BF16, device="cuda")
    wide[:, 8:136], wide[:, 136:328], wide[:, 328:] = x, res, dy
    same(wide[:, 8:136], wide[:, 136:328], wide[:, 328:])
    same(x.t().contiguous().t(), res.t().contiguous().t(), dy.t().contiguous().t())
    odd = torch.zeros(60 * 128 + 1, dtype=BF16, device="cuda")[1:].view(60, 128)
    odd.copy_(x)
    same(odd, res, dy)
    # a broadcast loss; a gradient into a given buffer; parts that are not wanted
    y, saved = prm.linear(x, w, b, act="silu", residual=res, save=True)
    flat = torch.full((1,), 0.5, dtype=BF16, device="cuda").expand(60, 192)
    for a, c in zip(prm.linear_backward(flat, x, w, saved, act="silu"),
                    prm.linear_backward(flat.contiguous(), x, w, saved, act="silu")):
        assert torch.equal(a, c)
    held = torch.full_like(w, float("nan"))
    got = prm.linear_backward(dy, x, w, saved, act="silu", need_dx=False, need_dbias=False, grad=held)
    assert got[0] is None and got[2] is None and got[1] is held and torch.equal(held, want[2])
    # a slice of a fused weight, one row of many
    fused = torch.cat([w, w])
    assert torch.equal(prm.linear(x, fused[192:], b, act="silu", residual=res), want[0])
    one = prm.linear(wide[:1, 8:136], w, b, act="silu", residual=wide[:1, 136:328])
    assert torch.equal(one, prm.linear(x[:1], w, b, act="silu", residual=res[:1]))


def test_linear_without_tokens():
    x, w, b, res, dy = _linear_inputs(4, 64, 32)
    y, saved = prm.linear(x[:0], w, b, act="gelu", save=True)
    assert y.shape == (0, 32)
    dx, dw, db = prm.linear_backward(dy[:0].to(BF16), x[:0], w, saved, act="gelu")
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


@pytest.mark.parametrize("T,k,n", [(70, 1024, 512), (1500, 512, 1536)])
def test_linear_is_reproducible_and_leaves_its_inputs(T, k, n):
    x, w, b, res, dy = _linear_inputs(T, k, n)
    before = [t.clone() for t in (x, w, b, res, dy)]
    runs = []
    for _ in range(4):
        y, saved = prm.linear(x, w, b, act="gelu", residual=res, save=True)
        runs.append((y,) + prm.linear_backward(dy, x, w, saved, act="gelu"))
    for r in runs[1:]:
        for a, c in zip(r, runs[0]):
            assert torch.equal(a, c)
    for a, c in zip((x, w, b, res, dy), before):
        assert torch.equal(a, c)


def test_linear_refuses():
    x, w, b, res, dy = _linear_inputs(6, 64, 32)
    for bad in (dict(x=x.float()), dict(weight=w.half()), dict(weight=w.t()), dict(weight=w[:, :32]),
                dict(weight=w[:30].contiguous()), dict(bias=b.to(BF16)), dict(bias=b[:16]), dict(bias=b.cpu()),
                dict(residual=res[:3]), dict(residual=res.half()), dict(act="relu"),
                dict(bias=torch.zeros(33, device="cuda")[1:])):
        args = dict(x=x, weight=w, bias=b)
        args.update(bad)
        with pytest.raises(ValueError):
            prm.linear(**args)
    y, saved = prm.linear(x, w, b, act="silu", save=True)
    for bad in (dict(act=None), dict(act="gelu"), dict(x=x[:3], dy=dy[:3].to(BF16)), dict(dy=dy.half()),
                dict(weight=w[:16]), dict(grad=w[:16]), dict(grad=w.half()), dict(grad=w.t())):
        args = dict(dy=dy.to(BF16), x=x, weight=w, saved=saved, act="silu")
        args.update(bad)
        with pytest.raises(ValueError):
            prm.linear_backward(**args)
