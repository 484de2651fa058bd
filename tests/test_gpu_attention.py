"""Numerics of the operators of a block's attention half against the fp64
oracle, at the sizes, layouts and values where their kernels change path or
could go wrong.

Tolerances. U is the largest relative error of one rounding to a type: half a
step, 2^-9 of the value's power of two, so at most 2^-8 of the value for bf16
(2^-11 for fp16, 2^-24 for fp32). fp32 arithmetic adds its own steps of 2^-24,
counted where they matter."""
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


# --------------------------------------------------------- rotary positions
def _inv_freq(dim, base=10000.0):
    return [base ** (-2.0 * i / dim) for i in range(dim // 2)]


def _check_rotary(x, pos, dim, layout, amplitude=1.0, y=None, inverse=False):
    """x: 4-D; y: what the call gave (made here if not given)."""
    plan = prm.rotary_plan(dim, layout=layout, amplitude=amplitude)
    if y is None:
        y = (prm.rotary_backward if inverse else prm.rotary)(x, pos, plan)
    p = pos.expand(x.shape[:2]).cpu().numpy()
    host = host64(x)
    want = O.rotary(host, p, _inv_freq(dim), layout, amplitude, inverse)
    # both of a pair bound the error that the angle's leaves: sine and cosine are taken of an angle rounded to
    # fp32 (pi 2^-24), are themselves off by 2 2^-24 at most, and three products and sums follow; the plan's
    # fraction is off by 2^-65 of a turn per position
    half = dim // 2
    size = np.abs(host)
    a, b = (size[..., :half], size[..., half:dim]) if layout == "half" else (size[..., 0:dim:2], size[..., 1:dim:2])
    pair = np.zeros_like(host)
    far = np.abs(p.astype(np.float64))[:, :, None, None] * 2.0 ** -62
    both = (10 * 2.0 ** -24 + far) * amplitude * (a + b)
    if layout == "half":
        pair[..., :half] = pair[..., half:dim] = both
    else:
        pair[..., 0:dim:2] = pair[..., 1:dim:2] = both
    got = host64(y)
    assert (np.abs(got - want) <= U[x.dtype] * np.abs(want) + pair).all()
    assert np.array_equal(got[..., dim:], host[..., dim:])
    return y


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("D,dim", [(128, 128), (64, 32), (72, 72), (40, 20), (2, 2), (7, 4), (20, 12), (24, 6)])
def test_rotary_heads(layout, dtype, D, dim):
    g = _gen(D + dim)
    x = _rand(g, 2, 5, 3, D, dtype=dtype)
    pos = torch.randint(0, 5000, (2, 5), generator=g).cuda()
    _check_rotary(x, pos, dim, layout, amplitude=1.25)
    _check_rotary(x, pos, dim, layout, amplitude=1.25, inverse=True)


@pytest.mark.parametrize("B,L,H", [(1, 1, 1), (1, 1, 40), (3, 1, 2), (1, 70, 1), (2, 33, 17), (5, 200, 2), (1, 3, 130)])
def test_rotary_shapes(B, L, H):
    g = _gen(B * L * H)
    _check_rotary(_rand(g, B, L, H, 16, dtype=BF16), torch.arange(L, device="cuda"), 16, "half")


def test_rotary_many_tokens_share_a_block():
    g = _gen(3)
    x = _rand(g, 3, 70000, 1, 8, dtype=BF16)
    pos = torch.arange(70000, device="cuda", dtype=torch.int32)
    y = prm.rotary(x, pos, prm.rotary_plan(8))
    for at in (0, 69990):
        _check_rotary(x[:, at:at + 10], pos[at:at + 10], 8, "half", y=y[:, at:at + 10])


def test_rotary_far_and_negative_positions():
    g = _gen(4)
    x = _rand(g, 1, 6, 2, 32, dtype=FP32)
    pos = torch.tensor([[0, -1, 2 ** 31 + 5, -(2 ** 33), 2 ** 36 + 1, 999999937]], device="cuda")
    _check_rotary(x, pos, 32, "half")
    _check_rotary(x, pos[:, -1:].int(), 32, "interleaved")


def test_rotary_strides_and_in_place():
    g = _gen(5)
    qkv = _rand(g, 2, 9, 3 * 4, 64, dtype=BF16)
    pos = torch.arange(100, 109, device="cuda")
    plan = prm.rotary_plan(48)
    want = prm.rotary(qkv.contiguous(), pos, plan)
    # queries and keys of a fused projection, turned in place; the values stay
    fused = qkv.clone()
    out = prm.rotary(fused[:, :, :8], pos, plan, out=fused[:, :, :8])
    assert out.data_ptr() == fused.data_ptr() and torch.equal(fused[:, :, :8], want[:, :, :8])
    assert torch.equal(fused[:, :, 8:], qkv[:, :, 8:])
    # heads before tokens, odd pitches, elements that do not follow each other, no samples
    x = qkv.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(prm.rotary(x, pos, plan), want)
    wide = torch.zeros(2, 9, 12, 67, dtype=BF16, device="cuda")
    wide[..., 1:65] = qkv
    assert torch.equal(prm.rotary(wide[..., 1:65], pos, plan), want)
    held = torch.full_like(wide, 7.0)
    prm.rotary(qkv, pos, plan, out=held[..., 2:66])
    assert torch.equal(held[..., 2:66], want) and (held[..., :2] == 7).all() and (held[..., 66:] == 7).all()
    turned = qkv.transpose(2, 3).contiguous().transpose(2, 3)
    assert torch.equal(prm.rotary(turned, pos, plan), want)
    assert torch.equal(prm.rotary(qkv[1], pos, plan), want[1])
    assert torch.equal(prm.rotary(qkv[:, :1].expand(2, 9, 12, 64), pos, plan)[:, :1], want[:, :1])
    # one position for all tokens of a sample
    one = torch.tensor([[3], [4]], device="cuda")
    assert torch.equal(prm.rotary(qkv, one, plan), prm.rotary(qkv, one.expand(2, 9).contiguous(), plan))


def test_rotary_refuses():
    x, pos, plan = torch.zeros(2, 3, 4, 8, device="cuda"), torch.arange(3, device="cuda"), prm.rotary_plan(8)
    for bad in (dict(positions=pos.float()), dict(positions=torch.arange(4, device="cuda")),
                dict(positions=torch.zeros(3, 3, device="cuda", dtype=torch.int64)),
                dict(positions=torch.zeros(1, 2, 3, device="cuda", dtype=torch.int64)), dict(positions=pos.cpu()),
                dict(plan=prm.rotary_plan(10)), dict(plan=prm.rotary_plan(8, device="cpu")), dict(x=x[0, 0]),
                dict(x=x.double()), dict(out=x[:1]), dict(out=x.half()), dict(out=x[:, :1].expand(2, 3, 4, 8))):
        args = dict(x=x, positions=pos, plan=plan)
        args.update(bad)
        with pytest.raises(ValueError):
            prm.rotary(**args)
    assert prm.rotary(x[:, :0], pos[:0], plan).shape == (2, 0, 4, 8)


# ------------------------------------------------------------------ dropout
def _check_dropout(x, p, seed, offset=0, residual=None):
    y = prm.dropout(x, p, seed, offset, residual=residual)
    want = O.dropout(host64(x), p, seed, offset, None if residual is None else host64(residual))
    # x / (1 - p) is a product with the rounded reciprocal: two steps of fp32, then the sum's and the output's
    size = np.abs(host64(x)) / max(1.0 - p, 2.0 ** -32)
    assert (np.abs(host64(y) - want) <= U[y.dtype] * np.abs(want) + 3 * 2.0 ** -24 * (size + np.abs(want))).all()
    return y


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("n", [1, 3, 4, 7, 8, 9, 2047, 2048, 2051, 10000])
def test_dropout_sizes(dtype, n):
    g = _gen(n)
    x, res = _rand(g, n, dtype=dtype), _rand(g, n, dtype=dtype)
    y = _check_dropout(x, 0.3, 2 ** 63 + n, offset=2 ** 32 - 1)
    assert torch.equal(prm.dropout_backward(x, 0.3, 2 ** 63 + n, offset=2 ** 32 - 1), y)
    _check_dropout(x, 0.3, n, residual=res)
    _check_dropout(x, 0.3, n, residual=res.float())


@pytest.mark.parametrize("p", [0.0, 2.0 ** -33, 0.1, 0.5, 1.0 - 2.0 ** -20, 1.0])
def test_dropout_probabilities(p):
    g = _gen(8)
    x = _rand(g, 60, 50)
    y = _check_dropout(x, p, 5)
    if p == 0.0:
        assert torch.equal(y, x)
    if p == 1.0:
        assert not y.any()


def test_dropout_leaves_out_what_it_drops():
    bad = torch.full((4096,), float("nan"), device="cuda")
    keep = torch.from_numpy(O.kept(4096, 0.5, 3)).cuda()
    x = torch.where(keep, torch.ones_like(bad), bad)
    assert torch.isfinite(prm.dropout(x, 0.5, 3)).all()
    assert torch.isfinite(prm.dropout(x, 0.5, 3, residual=torch.ones_like(x))).all()
    assert not prm.dropout(bad, 1.0, 3).any()


def test_dropout_layouts_types_and_seeds():
    g = _gen(9)
    x, res = _rand(g, 40, 24, dtype=BF16), _rand(g, 40, 24)
    y = _check_dropout(x, 0.2, -5, offset=11, residual=res)
    assert y.dtype is FP32
    # its gradient comes in fp32 and goes back to 16 bits
    dx = prm.dropout_backward(res, 0.2, -5, offset=11, dtype=BF16)
    assert dx.dtype is BF16 and torch.equal(dx, prm.dropout_backward(res, 0.2, -5, offset=11).to(BF16))
    # the mask goes by the element's index, whatever the memory
    assert torch.equal(prm.dropout(x.t().contiguous().t(), 0.2, -5, offset=11, residual=res), y)
    odd = torch.zeros(40 * 24 + 1, dtype=BF16, device="cuda")[1:].view(40, 24)
    odd.copy_(x)
    assert torch.equal(prm.dropout(odd, 0.2, -5, offset=11, residual=res), y)
    # the next call's offset: fresh words, and those of a part are those of the whole
    assert torch.equal(prm.dropout(x[8:], 0.2, -5, offset=11 + 8 * 24 // 4, residual=res[8:]), y[8:])
    # a seed that is read on the device
    seed = torch.tensor([-5], device="cuda")
    assert torch.equal(prm.dropout(x, 0.2, seed, offset=11, residual=res), y)
    assert prm.dropout(x[:0], 0.2, 1).shape == (0, 24)


def test_dropout_in_a_graph_draws_again():
    g = _gen(10)
    x, seed = _rand(g, 5000), torch.tensor([1], device="cuda")
    prm.dropout(x, 0.4, seed)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = prm.dropout(x, 0.4, seed)
        seed += 1
    for k in range(1, 4):
        graph.replay()
        assert torch.equal(y, prm.dropout(x, 0.4, k))


def test_dropout_refuses():
    x = torch.zeros(4, 4, device="cuda")
    for bad in (dict(p=-0.1), dict(p=1.1), dict(residual=x[:2]), dict(residual=x.half()), dict(residual=x.cpu()),
                dict(seed=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(seed=torch.zeros(1, device="cuda")),
                dict(seed=torch.zeros(1, dtype=torch.int64)), dict(x=x.double())):
        args = dict(x=x, p=0.5, seed=1)
        args.update(bad)
        with pytest.raises(ValueError):
            prm.dropout(**args)
