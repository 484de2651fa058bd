"""Numerics of the operators of a block's attention half against the fp64
oracle, at the sizes, layouts and values where their kernels change path or
could go wrong.

Tolerances. U is the largest relative error of one rounding to a type: half a
step, 2^-9 of the value's power of two, so at most 2^-8 of the value for bf16
(2^-11 for fp16, 2^-24 for fp32). fp32 arithmetic adds its own steps of 2^-24,
counted where they matter."""
import math

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


# ---------------------------------------------------------- cross attention
def _attention_inputs(B, Lq, Lk, H, Hkv, D, dtype=BF16, seed=0, size=1.5):
    g = _gen(seed + B + Lq + 3 * Lk + 5 * H + 7 * Hkv + 11 * D)
    return (_rand(g, B, Lq, H, D, dtype=dtype, scale=size), _rand(g, B, Lk, Hkv, D, dtype=dtype),
            _rand(g, B, Lk, Hkv, D, dtype=dtype), _rand(g, B, Lq, H, D, dtype=dtype))


def _tiny(u):
    return 2.0 ** -25 if u == U[FP16] else 2.0 ** -126


def _attention_bounds(do, q, k, v, lengths, scale, u):
    """What o, dq, dk and dv may be off by, element by element, from the roundings that the header names and fp32
    steps of 2^-24. S is off by (head + 3) steps of sum |q| |k|, 2^x by 2 steps more, and the row's sum and
    maximum leave P relatively exact to that; P is rounded to 16 bits (u) as an operand, and sums over n terms in
    fp32 add n steps. o is rounded once more (u), and delta is formed from it; dS is rounded (u). Gradients are
    rounded once at the end (u). What lies below a type's normal range is off by half of its smallest step (fp16
    2^-25), or left out (2^x below 2^-126)."""
    e, tiny = 2.0 ** -24, _tiny(u)
    out = [np.zeros(t.shape) for t in (q, q, k, v)]
    heads, kv_heads, head = q.shape[2], k.shape[2], q.shape[3]
    for b, n in enumerate(lengths):
        if n <= 0:
            continue
        kk, vv = (np.repeat(t[b, :n], heads // kv_heads, axis=1) for t in (k, v))
        p = O.attention_probabilities(q[b], k[b, :n], scale)
        s_off = scale * (head + 3) * e * np.einsum("qhd,khd->hqk", np.abs(q[b]), np.abs(kk)).max(-1, keepdims=True)
        off = 2 * s_off + (n + 40) * e                      # relative error of a normalised, unrounded P
        pv = np.einsum("hqk,khd->qhd", p, np.abs(vv))
        o_abs = np.abs(np.einsum("hqk,khd->qhd", p, vv))
        off_q = off[..., 0].T[..., None]                    # [queries, heads, 1]
        out[0][b] = (u + off_q) * pv * (1 + u) + u * o_abs + tiny * np.abs(vv).sum(0)[None]
        dp_abs = np.einsum("qhd,khd->hqk", np.abs(do[b]), np.abs(vv))
        delta_off = (np.abs(do[b]) * (out[0][b] + head * e * (o_abs + out[0][b]))).sum(-1).T[..., None]
        dp = np.einsum("qhd,khd->hqk", do[b], vv)
        ds = np.abs(p * (dp - (p * dp).sum(-1, keepdims=True)))
        ds_off = ((u + off + 4 * e) * ds + p * (1 + off) * (head * e * dp_abs + delta_off)) * (1 + u) + tiny
        terms = n * e
        out[1][b] = scale * (np.einsum("hqk,khd->qhd", ds_off + terms * ds, np.abs(kk)))
        for at, w, w_off, t in ((2, scale * ds, scale * ds_off, q[b]), (3, p, (u + off) * p + tiny, do[b])):
            terms = heads // kv_heads * q.shape[1] * e
            g = np.einsum("hqk,qhd->khd", w_off + terms * (w + w_off), np.abs(t))
            out[at][b, :n] = g.reshape(n, kv_heads, heads // kv_heads, head).sum(2)
    return out


def _check_attention(q, k, v, do, lengths=None, scale=None, calls=None):
    """Runs both passes and compares them; calls: (o, dq, dk, dv) made elsewhere."""
    u = U[q.dtype]
    n = None if lengths is None else torch.tensor(lengths, device="cuda")
    if calls is None:
        o, saved = prm.cross_attention(q, k, v, n, scale=scale, save=True)
        calls = (o,) + tuple(prm.cross_attention_backward(do, q, k, v, o, saved, n, scale=scale))
        assert torch.equal(prm.cross_attention(q, k, v, n, scale=scale), o)
    cut = [k.shape[1]] * k.shape[0] if lengths is None else [max(0, min(x, k.shape[1])) for x in lengths]
    scale = q.shape[3] ** -0.5 if scale is None else scale
    host = [host64(t) for t in (do, q, k, v)]
    for t in host[2:]:
        for b, x in enumerate(cut):
            t[b, x:] = 0.0
    want = (O.cross_attention(*host[1:], cut, scale),) + O.cross_attention_backward(*host, cut, scale)
    bounds = _attention_bounds(*host, cut, scale, u)
    for name, got, ref, bound in zip(("o", "dq", "dk", "dv"), calls, want, bounds):
        got = host64(got)
        assert np.isfinite(got).all(), name
        err = np.abs(got - ref) - (bound + u * np.abs(ref) + _tiny(u))  # (the output's own rounding)
        assert (err <= 0).all(), (name, err.max(), np.abs(ref).max())
    return calls


# one of everything, edges of the query and key tiles, one and two tiles and more on both axes
ATTENTION_SHAPES = [(1, 1, 1, 1, 1), (1, 2, 3, 1, 1), (2, 127, 129, 2, 2), (1, 128, 128, 1, 1), (1, 129, 127, 3, 3),
                    (1, 256, 256, 2, 2), (1, 257, 130, 1, 1), (2, 300, 77, 2, 2), (1, 5, 1000, 2, 2),
                    (1, 600, 385, 2, 1), (1, 513, 513, 1, 1)]


@pytest.mark.parametrize("B,Lq,Lk,H,Hkv", ATTENTION_SHAPES)
@pytest.mark.parametrize("D", [64, 128])
def test_attention_shapes(B, Lq, Lk, H, Hkv, D):
    _check_attention(*_attention_inputs(B, Lq, Lk, H, Hkv, D))


@pytest.mark.parametrize("D", [8, 16, 24, 40, 56, 72, 80, 104, 120])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_attention_heads(D, dtype):
    _check_attention(*_attention_inputs(2, 150, 140, 3, 3, D, dtype=dtype), lengths=[140, 133])


@pytest.mark.parametrize("H,Hkv", [(2, 1), (4, 1), (8, 2), (6, 2), (12, 1), (32, 1), (64, 1), (7, 1), (40, 8)])
@pytest.mark.parametrize("Lq", [1, 3, 70])
def test_attention_shared_heads(H, Hkv, Lq):
    _check_attention(*_attention_inputs(2, Lq, 200, H, Hkv, 64), lengths=[200, 65])


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_attention_lengths(dtype):
    lengths = [0, 1, 63, 64, 65, 127, 128, 129, 191, 200, 300, -3]
    _check_attention(*_attention_inputs(12, 40, 200, 2, 1, 64, dtype=dtype), lengths=lengths)
    _check_attention(*_attention_inputs(12, 140, 200, 2, 1, 128, dtype=dtype), lengths=lengths)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("Lq", [1, 150])
def test_attention_ignores_what_lies_behind_the_last_key(bad, Lq):
    q, k, v, do = _attention_inputs(3, Lq, 300, 2, 2, 72)
    lengths = [299, 130, 0]
    want = _check_attention(q, k, v, do, lengths)
    k, v = k.clone(), v.clone()
    for b, n in enumerate(lengths):
        k[b, n:] = bad
        v[b, n:] = bad
    for a, b in zip(_check_attention(q, k, v, do, lengths), want):
        assert torch.equal(a, b)


# long keys for few queries and long queries for few keys: ranges on different CTAs, some without work
@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D,lengths", [(1, 9, 3000, 1, 1, 64, None), (2, 100, 2500, 2, 1, 128, [2500, 300]),
                                                     (1, 2500, 60, 1, 1, 128, None), (2, 1500, 130, 4, 2, 64, [130, 0]),
                                                     (1, 1200, 1300, 1, 1, 72, [1201])])
def test_attention_in_parts(B, Lq, Lk, H, Hkv, D, lengths):
    _check_attention(*_attention_inputs(B, Lq, Lk, H, Hkv, D), lengths=lengths)


# more tiles than SMs, and a last round of them that leaves SMs idle: its tiles in parts, the others whole
@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,lengths", [(1, 1030, 1100, 40, 40, None), (2, 1030, 1100, 40, 20, [1100, 700]),
                                                   (3, 1030, 100, 60, 60, [100, 0, 37])])
def test_attention_last_round_in_parts(B, Lq, Lk, H, Hkv, lengths):
    _check_attention(*_attention_inputs(B, Lq, Lk, H, Hkv, 16), lengths=lengths)


def test_attention_large_and_growing_scores():
    # maxima that grow from tile to tile by more than the exponent's slack, and fall again
    q, k, v, do = _attention_inputs(1, 200, 700, 2, 2, 64)
    steps = torch.tensor([0.2, 3.0, 0.5, 8.0, 20.0, 1.0], device="cuda").repeat_interleave(128)[:700]
    k = (k.float() * steps[None, :, None, None]).to(BF16)
    _check_attention(q, k, v, do)
    _check_attention(q, k, v, do, scale=2.0)
    _check_attention(q, k, v, do, scale=1e-6)


def test_attention_layouts():
    B, Lq, Lk, H, D = 2, 90, 140, 4, 64
    q, k, v, do = _attention_inputs(B, Lq, Lk, H, 2, D)
    want = _check_attention(q, k, v, do, [140, 100])
    n = torch.tensor([140, 100], device="cuda", dtype=torch.int32)

    def same(q, k, v, do, n=n, **kw):
        o, saved = prm.cross_attention(q, k, v, n, save=True, **kw)
        got = (o,) + tuple(prm.cross_attention_backward(do, q, k, v, o, saved, n))
        for a, b in zip(got, want):
            assert torch.equal(a, b)

    kv = torch.stack([k, v], 2)                                      # one projection of the states
    same(q, kv[:, :, 0], kv[:, :, 1], do)
    qs = q.transpose(1, 2).contiguous().transpose(1, 2)              # heads before tokens
    same(qs, k.transpose(1, 2).contiguous().transpose(1, 2), v, do.transpose(1, 2).contiguous().transpose(1, 2))
    same(q.transpose(2, 3).contiguous().transpose(2, 3), k, v, do)   # elements apart: copied
    wide = torch.zeros(B, Lq, H, 67, dtype=BF16, device="cuda")
    wide[..., 1:65] = q
    same(wide[..., 1:65], k, v, do)                                  # an odd start: copied
    same(q, k, v, do, torch.tensor([140, 7, 100, 9], device="cuda")[::2])
    held = torch.full((B, Lq, 3 * H, D), 3.0, dtype=BF16, device="cuda")
    same(q, k, v, do, out=held[:, :, H:2 * H])
    assert torch.equal(held[:, :, H:2 * H], want[0]) and (held[:, :, :H] == 3).all() and (held[:, :, 2 * H:] == 3).all()
    # gradients into the halves of a fused projection's gradient; a gradient that is broadcast
    o, saved = prm.cross_attention(q, k, v, n, save=True)
    dkv, dq = torch.full_like(kv, float("nan")), torch.full_like(q, float("nan"))
    got = prm.cross_attention_backward(do, q, k, v, o, saved, n, grads=(dq, dkv[:, :, 0], dkv[:, :, 1]))
    assert got[0] is dq and torch.equal(dq, want[1])
    assert torch.equal(dkv[:, :, 0], want[2]) and torch.equal(dkv[:, :, 1], want[3])
    flat = torch.full((1,), 0.5, dtype=BF16, device="cuda").expand(B, Lq, H, D)
    for a, b in zip(prm.cross_attention_backward(flat, q, k, v, o, saved, n),
                    prm.cross_attention_backward(flat.contiguous(), q, k, v, o, saved, n)):
        assert torch.equal(a, b)


def test_attention_is_reproducible_and_leaves_its_inputs():
    q, k, v, do = _attention_inputs(2, 700, 900, 4, 2, 128)
    before = [t.clone() for t in (q, k, v, do)]
    runs = []
    for _ in range(4):
        o, saved = prm.cross_attention(q, k, v, save=True)
        runs.append((o,) + tuple(prm.cross_attention_backward(do, q, k, v, o, saved)) + (saved.lse,))
    for r in runs[1:]:
        for a, b in zip(r, runs[0]):
            assert torch.equal(a, b)
    for a, b in zip((q, k, v, do), before):
        assert torch.equal(a, b)


def test_attention_without_keys_or_queries():
    q, k, v, do = _attention_inputs(2, 5, 7, 2, 2, 16)
    o, saved = prm.cross_attention(q, k[:, :0], v[:, :0], save=True)
    assert not o.any() and torch.isneginf(saved.lse).all()
    dq, dk, dv = prm.cross_attention_backward(do, q, k[:, :0], v[:, :0], o, saved)
    assert not dq.any() and dk.shape == (2, 0, 2, 16)
    o, saved = prm.cross_attention(q[:, :0], k, v, save=True)
    assert o.shape == (2, 0, 2, 16)
    dq, dk, dv = prm.cross_attention_backward(do[:, :0], q[:, :0], k, v, o, saved)
    assert not dk.any() and not dv.any() and dk.shape == k.shape
    assert prm.cross_attention(q[:0], k[:0], v[:0]).shape == (0, 5, 2, 16)


def test_attention_refuses():
    q, k, v, do = _attention_inputs(2, 5, 7, 4, 2, 16)
    n = torch.tensor([7, 3], device="cuda")
    for bad in (dict(q=q.float()), dict(k=k.half()), dict(v=v[:, :6]), dict(q=q[:1]), dict(q=q[..., :12]),
                dict(k=k[:, :, :1].expand(2, 7, 3, 16), v=v[:, :, :1].expand(2, 7, 3, 16)), dict(key_lengths=n[:1]),
                dict(key_lengths=n.float()), dict(key_lengths=n.cpu()), dict(scale=0.0), dict(scale=-1.0),
                dict(out=q[:1]), dict(out=q.half()), dict(out=q[:, :1].expand(2, 5, 4, 16)), dict(q=q[0])):
        args = dict(q=q, k=k, v=v)
        args.update(bad)
        with pytest.raises(ValueError):
            prm.cross_attention(**args)
    o, saved = prm.cross_attention(q, k, v, save=True)
    for bad in (dict(do=do[:1]), dict(o=o.half()), dict(saved=saved._replace(lse=saved.lse[:, :, :1])),
                dict(scale=0.5), dict(k=k[:, :6], v=v[:, :6]), dict(grads=(q, k)), dict(grads=(q, k, v[:, :1]))):
        args = dict(do=do, q=q, k=k, v=v, o=o, saved=saved)
        args.update(bad)
        with pytest.raises(ValueError):
            prm.cross_attention_backward(**args)


def test_scales_beyond_fp32_are_refused():
    q, k, v = (torch.zeros(1, n, 1, 8, dtype=torch.bfloat16, device="cuda") for n in (2, 3, 3))
    for scale in (0.0, -1.0, 1e-50, 3.5e38, 1e300, math.inf, math.nan):
        with pytest.raises(ValueError):
            prm.cross_attention(q, k, v, scale=scale)


def test_attention_gradients_of_one_key():
    # softmax of one score is one: o is v, dv the sum of do, dq and dk zero but for delta's rounding
    q, k, v, do = _attention_inputs(3, 70, 1, 4, 2, 64)
    o, saved = prm.cross_attention(q, k, v, save=True)
    assert torch.equal(o, v.repeat_interleave(2, 2).expand_as(o))
    dq, dk, dv = prm.cross_attention_backward(do, q, k, v, o, saved)
    want = do.double().sum(1, keepdim=True).unflatten(2, (2, 2)).sum(3)
    # 140 additions in fp32 and the rounding to bf16
    size = do.double().abs().sum(1, keepdim=True).unflatten(2, (2, 2)).sum(3)
    assert ((dv.double() - want).abs() <= 2.0 ** -8 * want.abs() + 140 * 2.0 ** -23 * size).all()
    # do . v is summed twice, in two orders: 64 additions each, of products of up to 16 sizes (P is one to 2^-22)
    off = 2 * 65 * 2.0 ** -23 * (do.double().abs() * v.repeat_interleave(2, 2).double().abs()).sum(3)
    scale = 64 ** -0.5
    assert (dq.double().abs() <= 1.01 * scale * off[..., None] * k.repeat_interleave(2, 2).double().abs() + 1e-30).all()
    bound = (off[..., None] * q.double().abs()).sum(1, keepdim=True).unflatten(2, (2, 2)).sum(3)
    assert (dk.double().abs() <= 1.01 * scale * bound + 1e-30).all()


@pytest.mark.parametrize("dtype", [BF16, torch.float16])
@pytest.mark.parametrize("Lk, Hkv, D", [(1, 2, 64), (2, 4, 128), (3, 1, 32), (4, 2, 72), (5, 4, 128), (300, 2, 64)])
def test_attention_gradients_of_few_keys(Lk, Hkv, D, dtype):
    """With up to four keys delta has no rounding of o in it: what is left are dS'
    rounding, a half step of each of its values, and the result's own."""
    q, k, v, do = _attention_inputs(5, 130, Lk, 4, Hkv, D, dtype)
    lengths = torch.tensor([Lk, min(Lk, 2), 1, min(Lk, 4), 0], device="cuda")
    o, saved = prm.cross_attention(q, k, v, lengths, save=True)
    dq, dk, dv = prm.cross_attention_backward(do, q, k, v, o, saved, lengths)
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps  # the least step
    scale = D ** -0.5
    for b, n in enumerate(lengths.tolist()):
        if n == 0 or n > 4:
            continue
        Q, G = (t[b].double().transpose(0, 1) for t in (q, do))
        K, V = (t[b, :n].double().transpose(0, 1).repeat_interleave(4 // Hkv, 0) for t in (k, v))
        P = (scale * Q @ K.transpose(1, 2)).softmax(-1)
        dP = G @ V.transpose(1, 2)
        dS = P * (dP - (P * dP).sum(-1, keepdim=True))
        # fp32: P to 2^-20 of its value (scores below 100, their logarithm's rounding), sums of up to 128 products
        small = 2.0 ** -14 * P * (G.abs() @ V.abs().transpose(1, 2)).amax(-1, keepdim=True)
        off = half * dS.abs() + small + tiny
        want, bound = scale * dS @ K, scale * off @ K.abs()
        err = (dq[b].double().transpose(0, 1) - want).abs()
        assert (err <= 1.01 * (bound + half * (want.abs() + bound)) + tiny).all()
        want = (scale * dS.transpose(1, 2) @ Q).unflatten(0, (Hkv, 4 // Hkv)).sum(1)
        bound = (scale * off.transpose(1, 2) @ Q.abs()).unflatten(0, (Hkv, 4 // Hkv)).sum(1)
        err = (dk[b, :n].double().transpose(0, 1) - want).abs()
        assert (err <= 1.01 * (bound + half * (want.abs() + bound)) + tiny).all()
