"""Numerics of the transformer-block operators against the fp64 oracle, at
the sizes, layouts and values where their kernels change path or could go
wrong.

Tolerances. u is the unit roundoff of a 16-bit type (2^-8 for bf16, 2^-11 for
fp16). A result that is rounded once from fp32 is at most u off in relative
norm. The feed-forward block rounds h (and dg, du) to 16 bits before the next
product, so its outputs carry two independent roundings: 2 u. fp32 arithmetic
adds about (terms of a sum) 2^-24, stated where it is the bound."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_gb300 as prm
from matrix_aware_optimizer_gb300 import native as N
from oracle import blocks as O

from .gpu_helpers import ensure_built, host64, rel_frob

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, FP32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()
    N.load()
    yield
    prm.blocks_sync_status()


def _rand(gen, *shape, dtype=FP32, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).cuda()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------- gated FFN
def _ffn_inputs(T, d, f, dtype, seed=0):
    g = _gen(seed)
    x = _rand(g, T, d, dtype=dtype)
    ws = [_rand(g, f, d, dtype=dtype, scale=d ** -0.5), _rand(g, f, d, dtype=dtype, scale=d ** -0.5),
          _rand(g, d, f, dtype=dtype, scale=f ** -0.5)]
    return x, ws, _rand(g, T, d, dtype=dtype)


def _check_ffn(x, ws, dy, act):
    u = U[x.dtype]
    y, saved = prm.gated_ffn(x, *ws, act=act, save=True)
    grads = prm.gated_ffn_backward(dy, x, *ws, saved, act=act)
    host = [host64(t).reshape(-1, t.shape[-1]) for t in (x, *ws, dy)]
    ref = (O.gated_ffn(*host[:4], act),) + O.gated_ffn_backward(host[4], *host[:4], act)
    for name, got, want in zip(("y", "dx", "dw_gate", "dw_up", "dw_down"), (y,) + tuple(grads), ref):
        got = host64(got).reshape(want.shape)
        assert np.isfinite(got).all(), name
        assert rel_frob(got, want) <= 2 * u, (name, rel_frob(got, want))
    # the pass without saving gives the same y
    assert torch.equal(prm.gated_ffn(x, *ws, act=act), y)
    return y, saved, grads


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_ffn_activations_and_types(act, dtype):
    _check_ffn(*_ffn_inputs(130, 136, 264, dtype), act)


# one token, row tiles and their edges, column tiles and their edges, the
# shortest rows, sums shorter than one slice, sums split over CTA pairs
FFN_SHAPES = [(1, 64, 256), (2, 8, 8), (5, 2048, 1024), (31, 72, 40), (32, 64, 96), (33, 520, 24), (127, 256, 128),
              (128, 128, 128), (129, 264, 520), (255, 8, 1000), (256, 256, 256), (257, 200, 328), (300, 1000, 2664),
              (1, 512, 4096), (9, 1024, 2048), (16, 768, 2048), (17, 768, 2048), (64, 320, 8192), (1030, 64, 64)]


@pytest.mark.parametrize("T,d,f", FFN_SHAPES)
def test_ffn_shapes(T, d, f):
    _check_ffn(*_ffn_inputs(T, d, f, BF16, seed=T + d + f), "silu")


# enough output tiles for clusters of two CTA pairs (one of them without a tile
# at the end of a row), in the first products, in all of them, in the down
# projection; few tokens with wide weights
FFN_LARGE_SHAPES = [(300, 64, 9224), (1100, 72, 9224), (2100, 4104, 72), (2049, 2056, 2568), (6, 1032, 2064),
                    (8, 2056, 1032)]


@pytest.mark.parametrize("T,d,f", FFN_LARGE_SHAPES)
def test_ffn_large_shapes(T, d, f):
    _check_ffn(*_ffn_inputs(T, d, f, BF16, seed=T + d + f), "silu")


@pytest.mark.parametrize("T", list(range(1, 17)))
def test_ffn_few_tokens(T):
    _check_ffn(*_ffn_inputs(T, 264, 1032, FP16 if T % 2 else BF16, seed=T), "gelu_tanh")


def test_ffn_layouts():
    x, ws, dy = _ffn_inputs(60, 128, 192, BF16)
    y, saved, grads = _check_ffn(x, ws, dy, "silu")
    # leading dimensions, row-strided and column-strided inputs, both halves of one fused weight
    wide = torch.zeros(60, 200, dtype=BF16, device="cuda")
    wide[:, 8:136] = x
    turned = x.t().contiguous().t()
    odd = torch.zeros(60 * 128 + 1, dtype=BF16, device="cuda")[1:].view(60, 128)
    odd.copy_(x)
    fused = torch.cat([ws[0], ws[1]])
    for xx in (x.view(3, 20, 128), wide[:, 8:136], turned, odd):
        dyy = dy.view(xx.shape)
        y2, s2 = prm.gated_ffn(xx, fused[:192], fused[192:], ws[2], save=True)
        assert y2.shape == xx.shape and torch.equal(y2.reshape(60, 128), y)
        g2 = prm.gated_ffn_backward(dyy, xx, fused[:192], fused[192:], ws[2], s2)
        for a, b in zip(g2, grads):
            assert torch.equal(a.reshape(b.shape), b)
    # gradients of a broadcast loss arrive with stride 0
    flat = torch.full((1,), 0.5, dtype=BF16, device="cuda").expand(60, 128)
    a = prm.gated_ffn_backward(flat, x, *ws, saved)
    b = prm.gated_ffn_backward(flat.contiguous(), x, *ws, saved)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_ffn_gradients_into_given_buffers():
    x, ws, dy = _ffn_inputs(50, 64, 128, BF16)
    _, saved, grads = _check_ffn(x, ws, dy, "silu")
    out = [torch.full_like(w, float("nan")) for w in ws]
    got = prm.gated_ffn_backward(dy, x, *ws, saved, grads=out, need_dx=False)
    assert got[0] is None
    for o, g, r in zip(out, got[1:], grads[1:]):
        assert o is g and torch.equal(o, r)


def test_ffn_is_reproducible_and_leaves_its_inputs():
    x, ws, dy = _ffn_inputs(70, 1024, 512, BF16)
    before = [t.clone() for t in (x, *ws, dy)]
    y, saved, grads = _check_ffn(x, ws, dy, "gelu")
    for _ in range(3):
        y2, s2 = prm.gated_ffn(x, *ws, act="gelu", save=True)
        assert torch.equal(y, y2)
        for a, b in zip(prm.gated_ffn_backward(dy, x, *ws, s2, act="gelu"), grads):
            assert torch.equal(a, b)
    for a, b in zip(before, (x, *ws, dy)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [4, 40, 300])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_ffn_large_values_and_non_finite_rows(T, act):
    """Saturated gates (|g| up to several hundred) stay exact; a row with an
    infinity or a NaN spoils its own outputs only."""
    x, ws, dy = _ffn_inputs(T, 64, 128, BF16, seed=7)
    x = x * 100
    _check_ffn(x, ws, dy, act)
    y = prm.gated_ffn(x, *ws, act=act)
    x2 = x.clone()
    x2[1, 3] = float("nan")
    x2[3, 5] = float("inf")
    y2, saved = prm.gated_ffn(x2, *ws, act=act, save=True)
    keep = [i for i in range(T) if i not in (1, 3)]
    assert torch.equal(y2[keep], y[keep])
    assert torch.isnan(y2[1]).all()
    dx = prm.gated_ffn_backward(dy, x2, *ws, saved, act=act)[0]
    dx0 = prm.gated_ffn_backward(dy, x, *ws, prm.gated_ffn(x, *ws, act=act, save=True)[1], act=act)[0]
    assert torch.equal(dx[keep], dx0[keep])
    assert torch.isnan(dx[1]).all()


@pytest.mark.parametrize("T", [3, 40])
def test_ffn_keeps_an_infinite_projection(T):
    """u = inf in one place: the gradient of that feature's gate is infinite
    of a definite sign, not a NaN, and the other features' gradients stay finite."""
    x, (w_gate, w_up, w_down), dy = _ffn_inputs(T, 16, 64, BF16, seed=11)
    x[:, 0] = 0.0
    x[1, 0] = 3e38
    w_gate[:, 0] = 0.0
    w_up[:, 0] = 0.0
    w_up[9, 0] = 3e38
    y, saved = prm.gated_ffn(x, w_gate, w_up, w_down, save=True)
    assert torch.isinf(y[1]).all() and torch.isfinite(y[[0] + list(range(2, T))]).all()
    _, dw_gate, _, _ = prm.gated_ffn_backward(dy, x, w_gate, w_up, w_down, saved)
    g = x.double() @ w_gate.double().t()
    s = torch.sigmoid(g[1, 9])
    dg = (dy[1].double() @ w_down[:, 9].double()) * (s + g[1, 9] * s * (1 - s))
    assert torch.isinf(dw_gate[9]).all()
    assert torch.equal(torch.sign(dw_gate[9].double()), torch.sign(dg * x[1].double()))
    rest = [j for j in range(64) if j != 9]
    assert torch.isfinite(dw_gate[rest, 1:]).all()


def test_ffn_without_tokens():
    x, ws, dy = _ffn_inputs(0, 64, 128, BF16)
    y, saved = prm.gated_ffn(x, *ws, save=True)
    assert y.shape == (0, 64)
    out = [torch.full_like(w, 3.0) for w in ws]
    dx, *g = prm.gated_ffn_backward(dy, x, *ws, saved, grads=out)
    assert dx.shape == (0, 64) and all((t == 0).all() for t in g)


def test_ffn_on_another_stream():
    x, ws, dy = _ffn_inputs(200, 512, 1024, BF16)
    y, saved, grads = _check_ffn(x, ws, dy, "silu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2, saved2 = prm.gated_ffn(x, *ws, save=True, stream=s)
    g2 = prm.gated_ffn_backward(dy, x, *ws, saved2, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, y2)
    for a, b in zip(g2, grads):
        assert torch.equal(a, b)


def test_ffn_inputs_freed_while_another_stream_reads_them():
    """The memory of an input that dies right after a call on another stream
    is not handed out while that stream still has to read it."""
    x, ws, _ = _ffn_inputs(4096, 512, 1024, BF16)
    want = prm.gated_ffn(x, *ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        busy = torch.zeros(1 << 28, device="cuda")
        for _ in range(20):
            busy.add_(1.0)      # keeps the stream from starting the call at once
    mine = x.clone()
    torch.cuda.current_stream().synchronize()
    y = prm.gated_ffn(mine, *ws, stream=s)
    del mine
    junk = torch.full_like(x, float("nan"))   # would take the freed block
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.isnan(junk).all()


def test_ffn_in_a_graph():
    x, ws, dy = _ffn_inputs(90, 256, 512, BF16)
    _check_ffn(x, ws, dy, "silu")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, saved = prm.gated_ffn(x, *ws, save=True)
        grads = prm.gated_ffn_backward(dy, x, *ws, saved)
    x2, _, dy2 = _ffn_inputs(90, 256, 512, BF16, seed=5)
    x.copy_(x2)
    dy.copy_(dy2)
    g.replay()
    torch.cuda.synchronize()
    y1, s1 = prm.gated_ffn(x, *ws, save=True)
    assert torch.equal(y, y1)
    for a, b in zip(grads, prm.gated_ffn_backward(dy, x, *ws, s1)):
        assert torch.equal(a, b)


def test_ffn_offsets_past_32_bits():
    """tokens x f beyond 2^31: the last rows of y and dx, and a weight
    gradient that only the last rows feed."""
    T, d, f = 140001, 64, 16384
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, d, generator=g, device="cuda").to(BF16)
    _, ws, _ = _ffn_inputs(1, d, f, BF16)
    dy = torch.zeros(T, d, dtype=BF16, device="cuda")
    dy[-40:] = torch.randn(40, d, generator=g, device="cuda").to(BF16)
    y, saved = prm.gated_ffn(x, *ws, save=True)
    grads = prm.gated_ffn_backward(dy, x, *ws, saved)
    host = [host64(t) for t in (x[-40:], *ws, dy[-40:])]
    ref = (O.gated_ffn(*host[:4], "silu"),) + O.gated_ffn_backward(host[4], *host[:4], "silu")
    for got, want in zip((y[-40:], grads[0][-40:]) + tuple(grads[1:]), ref):
        assert rel_frob(host64(got), want) <= 2 * U[BF16]
    assert (grads[0][:-40] == 0).all()


def test_ffn_refusals():
    x, ws, dy = _ffn_inputs(8, 64, 128, BF16)
    y, saved = prm.gated_ffn(x, *ws, save=True)
    for bad in ((x.float(), *ws), (x, ws[0].half(), ws[1], ws[2]), (x, ws[0], ws[1], ws[2].t()),
                (x[:, :60], ws[0][:, :60].contiguous(), ws[1][:, :60].contiguous(), ws[2][:60])):
        with pytest.raises(ValueError):
            prm.gated_ffn(*bad)
    with pytest.raises(ValueError):
        prm.gated_ffn_backward(dy[:4], x[:4], *ws, saved)
    with pytest.raises(ValueError):
        prm.gated_ffn_backward(dy.half(), x, *ws, saved)
    with pytest.raises(ValueError):
        prm.gated_ffn_backward(dy, x, *ws, saved, grads=[w.float() for w in ws])


# --------------------------------------------------------- norms of a block
NORM_TYPES = [(FP32, FP32), (FP32, BF16), (FP32, FP16), (BF16, BF16), (FP16, FP16)]


def _norm_case(B, L, d, kind, st, bt, post, gate, pre, mod, alpha=0.75, eps=1e-6, seed=0, scale=1.0, mean=0.3):
    g = _gen(seed + d + L)
    x = _rand(g, B, L, d, dtype=st, scale=scale) + torch.tensor(mean, dtype=st)
    z = (_rand(g, B, L, d, scale=scale) + mean).to(bt)
    m = _rand(g, B, 4 * d + 3, dtype=bt, scale=0.5)     # modulation rows with an odd pitch, or below a tidy one
    if d % 8 == 0:
        m = m[:, :4 * d].contiguous()
    par = dict(post_weight=_rand(g, d) + 1 if post else None, gate=m[:, :d] if gate else None,
               pre_weight=_rand(g, d) + 1 if pre else None, scale=m[:, d:2 * d] if mod else None,
               shift=m[:, 2 * d:3 * d] if mod else None)
    dy, dr = _rand(g, B, L, d, dtype=bt), _rand(g, B, L, d, dtype=st)
    return x, z, par, dy, dr, dict(kind=kind, alpha=alpha), eps


def _check_norm(x, z, par, dy, dr, kw, eps):
    st, bt = x.dtype, (z if z is not None else dy).dtype
    h = {k: None if v is None else host64(v) for k, v in par.items()}
    p = dict(post=h["post_weight"], gate=h["gate"])
    q = dict(pre=h["pre_weight"], scale=h["scale"], shift=h["shift"])
    r, y, stats = prm.block_norm(x, z, eps=eps, **kw, **par, **({} if z is not None else dict(dtype=bt)))
    d = x.shape[-1]
    # an element's fp32 arithmetic (about 16 roundings) and sums over a row by a tree: below 2^-19
    fp = 2.0 ** -19
    if z is not None:
        want = O.block_join(host64(x), host64(z), kw["kind"], kw["alpha"], eps, **p)
        assert rel_frob(host64(r), want) <= (U[st] if st != FP32 else 0) + fp
    else:
        assert r is x
    rh = host64(r)
    if y is not None:
        want = O.block_next(rh, kw["kind"], eps, **q)
        assert rel_frob(host64(y), want) <= (U[bt] if bt != FP32 else 0) + fp
    got = prm.block_norm_backward(dy, dr, r, z, stats, **kw, **par)
    ref = O.block_backward(None if dy is None else host64(dy), None if dr is None else host64(dr), rh,
                           None if z is None else host64(z), kw["kind"], kw["alpha"], eps, **p, **q)
    rows = x.numel() // d
    for name, t in got._asdict().items():
        want = ref[name.replace("_weight", "")]
        assert (t is None) == (want is None), name
        if t is None:
            continue
        out = U[t.dtype] if t.dtype != FP32 else 0
        # a column sum of `rows` terms of either sign: relative to its result the terms weigh sqrt(rows)
        tol = fp * max(1.0, np.sqrt(rows) if name not in ("dx", "dz") else 1.0) + out
        if d <= 2 and kw["kind"] == "layer":
            # the norm of one or two elements has (almost) no gradient: compare against what cancels
            assert np.abs(host64(t) - want).max() <= 1e-2 * max(1.0, np.abs(want).max()), name
        else:
            assert rel_frob(host64(t), want) <= tol, (name, rel_frob(host64(t), want), tol)
    return r, y, stats, got


@pytest.mark.parametrize("st,bt", NORM_TYPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_types_with_everything(st, bt, kind):
    _check_norm(*_norm_case(3, 37, 264, kind, st, bt, 1, 1, 1, 1))
    _check_norm(*_norm_case(2, 9, 1000, kind, st, bt, 1, 1, 1, 1))


@pytest.mark.parametrize("post,gate,pre,mod", [(a, b, c, e) for a in (0, 1) for b in (0, 1) for c in (0, 1)
                                               for e in (0, 1)])
def test_norm_option_sets(post, gate, pre, mod):
    _check_norm(*_norm_case(2, 21, 96, "rms", FP32, BF16, post, gate, pre, mod))
    _check_norm(*_norm_case(2, 5, 2048, "layer", BF16, BF16, post, gate, pre, mod))


@pytest.mark.parametrize("d", [1, 2, 3, 7, 8, 15, 16, 17, 31, 64, 100, 255, 256, 257, 264, 511, 512, 513, 520, 1001,
                               1024, 1032, 2040, 2049, 4096, 4104, 5120, 8191, 8192])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_widths(d, kind):
    _check_norm(*_norm_case(2, 7, d, kind, FP32, BF16 if d % 3 else FP32, 1, 1, 1, 1, eps=1e-3 if d <= 2 else 1e-6))


@pytest.mark.parametrize("st,bt", [(FP32, FP32), (FP32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("d", [2040, 5112, 5128, 8184, 8192])
def test_norm_long_rows_by_option(d, st, bt):
    """Rows of which two may not fit in shared memory beside the option's
    column arrays."""
    for opts in ((1, 0, 1, 0), (0, 1, 0, 1), (0, 0, 0, 0), (1, 1, 1, 1)):
        _check_norm(*_norm_case(2, 9, d, "layer", st, bt, *opts))


@pytest.mark.parametrize("st,bt", [(FP32, FP32), (FP32, FP16), (BF16, BF16)])
@pytest.mark.parametrize("d", [17, 253, 1001, 2047, 2049, 3001, 5119, 5121, 7003, 8191])
def test_norm_odd_rows_by_option(d, st, bt):
    """Widths that are no multiple of 8, with every set of column sums."""
    for opts in ((1, 0, 1, 0), (0, 1, 0, 1), (0, 0, 0, 0), (1, 1, 1, 1)):
        _check_norm(*_norm_case(2, 9, d, "layer", st, bt, *opts))


@pytest.mark.parametrize("B,L", [(1, 1), (1, 2), (5, 1), (1300, 1), (1300, 3), (1, 5000), (7, 700), (40, 31)])
@pytest.mark.parametrize("mod", [0, 1])
def test_norm_row_counts(B, L, mod):
    _check_norm(*_norm_case(B, L, 48, "rms", FP32, FP32, 1, mod, 1, mod))
    _check_norm(*_norm_case(B, L, 520 if B * L < 2000 else 264, "layer", FP32, BF16, 1, mod, 1, mod))


def test_norm_misaligned_and_strided_inputs():
    x, z, par, dy, dr, kw, eps = _norm_case(2, 6, 256, "rms", BF16, BF16, 1, 1, 1, 1)
    r, y, stats, got = _check_norm(x, z, par, dy, dr, kw, eps)

    def off(t):
        o = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        return o.copy_(t)

    par2 = {k: None if v is None else off(v) for k, v in par.items()}
    _check_norm(off(x), off(z), par2, off(dy), off(dr), kw, eps)
    turned = z.transpose(0, 1).contiguous().transpose(0, 1)
    r3, y3, _ = prm.block_norm(x, turned, eps=eps, **kw, **par)
    assert torch.equal(r, r3) and torch.equal(y, y3)


def test_norm_first_and_last_of_a_stack():
    x, z, par, dy, dr, kw, eps = _norm_case(2, 11, 320, "layer", FP32, BF16, 0, 0, 1, 1, alpha=1.0)
    _check_norm(x, None, par, dy, dr, kw, eps)
    _check_norm(x, None, par, dy, None, kw, eps)
    x, z, par, dy, dr, kw, eps = _norm_case(2, 11, 320, "rms", FP32, BF16, 1, 1, 0, 0)
    r, y, stats = prm.block_norm(x, z, eps=eps, join_only=True, **kw, **par)
    assert y is None
    want = O.block_join(host64(x), host64(z), "rms", kw["alpha"], eps, host64(par["post_weight"]),
                        host64(par["gate"]))
    assert rel_frob(host64(r), want) <= 2.0 ** -19
    got = prm.block_norm_backward(None, dr, r, z, stats, **kw, **par)
    ref = O.block_backward(None, host64(dr), host64(r), host64(z), "rms", kw["alpha"], eps,
                           post=host64(par["post_weight"]), gate=host64(par["gate"]))
    for name in ("dx", "dz", "dgate"):
        assert rel_frob(host64(getattr(got, name)), ref[name]) <= U[BF16] + 2.0 ** -16, name
    assert got.dpre_weight is None and got.dscale is None


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("d", [64, 2048])
def test_norm_hard_rows(kind, d):
    """Rows of zeros, constant rows, rows with a mean far above their
    deviation, tiny and huge rows; a NaN row spoils itself only."""
    x, z, par, dy, dr, kw, eps = _norm_case(1, 8, d, kind, FP32, FP32, 1, 0, 1, 0, alpha=1.0)
    base = z.clone()
    z[0, 0] = 0
    z[0, 1] = 3.0
    z[0, 2] = base[0, 2] * 1e-3 + 50.0
    z[0, 3] *= 1e-18
    z[0, 4] *= 1e15
    x[0, 5] = 0
    z[0, 5] = 0
    r, y, stats = prm.block_norm(x, z, eps=eps, **kw, **par)
    m = (host64(z) - host64(z).mean(-1, keepdims=True)) if kind == "layer" else host64(z)
    want = host64(x) + m / np.sqrt((m * m).mean(-1, keepdims=True) + eps) * host64(par["post_weight"])
    # row 2 keeps 50 2^-24 / 1e-3 of its digits in fp32 input already: compared at that level
    err = np.abs(host64(r) - want).max(-1)[0]
    bound = np.full(8, 2.0 ** -18)
    bound[2] = 50 * 2.0 ** -22 / 1e-3 if kind == "layer" else 2.0 ** -18
    assert (err <= bound * np.abs(want).max(-1)[0]).all(), err
    wy = O.block_next(host64(r), kind, eps, pre=host64(par["pre_weight"]))
    assert np.abs(host64(y) - wy).max() <= 2.0 ** -17 * np.abs(wy).max()
    assert (y[0, 5] == 0).all()
    good = prm.block_norm_backward(dy, dr, r, z, stats, **kw, **par)
    assert all(torch.isfinite(t).all() for t in good if t is not None)
    z2 = z.clone()
    z2[0, 6, 1] = float("nan")
    r2, y2, _ = prm.block_norm(x, z2, eps=eps, **kw, **par)
    keep = [0, 1, 2, 3, 4, 5, 7]
    assert torch.equal(r2[0, keep], r[0, keep]) and torch.equal(y2[0, keep], y[0, keep])
    assert torch.isnan(y2[0, 6]).all()


def test_norm_repeats_bit_for_bit_and_on_another_stream():
    case = _norm_case(4, 300, 1024, "layer", FP32, BF16, 1, 1, 1, 1)
    x, z, par, dy, dr, kw, eps = case
    r, y, stats, got = _check_norm(*case)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s):
        r2, y2, st2 = prm.block_norm(x, z, eps=eps, stream=stream, **kw, **par)
        g2 = prm.block_norm_backward(dy, dr, r2, z, st2, stream=stream, **kw, **par)
        torch.cuda.synchronize()
        assert torch.equal(r, r2) and torch.equal(y, y2)
        for a, b in zip(got, g2):
            assert torch.equal(a, b)


def test_norm_no_rows():
    x = torch.zeros(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    r, y, stats = prm.block_norm(x, x.clone(), pre_weight=w)
    assert r.shape == y.shape == (0, 64)
    got = prm.block_norm_backward(x, None, r, x, stats, pre_weight=w)
    assert (got.dpre_weight == 0).all()


def test_norm_offsets_past_32_bits():
    d, rows = 8192, 262150   # rows x d beyond 2^31
    x = torch.zeros(rows, d, dtype=BF16, device="cuda")
    z = torch.zeros(rows, d, dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x[-9:] = torch.randn(9, d, generator=g, device="cuda").to(BF16)
    z[-9:] = torch.randn(9, d, generator=g, device="cuda").to(BF16)
    r, y, stats = prm.block_norm(x, z)
    want = O.block_next(host64(r[-9:]), "rms", 1e-6)
    assert rel_frob(host64(r[-9:]), host64(x[-9:]) + host64(z[-9:])) <= U[BF16]
    assert rel_frob(host64(y[-9:]), want) <= U[BF16] + 2.0 ** -19
    del x
    dy = torch.zeros(rows, d, dtype=BF16, device="cuda")
    dy[-9:] = 1.0
    got = prm.block_norm_backward(dy, None, r, z, stats)
    ref = O.block_backward(np.ones((1, 9, d)), None, host64(r[-9:])[None], host64(z[-9:])[None], "rms", 1.0, 1e-6)
    assert rel_frob(host64(got.dx[-9:]), ref["dx"][0]) <= U[BF16] + 2.0 ** -19


def test_norm_refusals():
    x = torch.zeros(4, 64, device="cuda")
    z = x.clone()
    for kw in (dict(kind="batch"), dict(pre_weight=torch.ones(64, device="cuda", dtype=BF16)),
               dict(pre_weight=torch.ones(63, device="cuda")), dict(gate=torch.ones(3, 64, device="cuda")),
               dict(gate=torch.ones(2, 64, device="cuda", dtype=BF16)),
               dict(gate=torch.ones(2, 64, device="cuda"), scale=torch.ones(4, 64, device="cuda")),
               dict(join_only=True, shift=torch.ones(2, 64, device="cuda"))):
        with pytest.raises(ValueError):
            prm.block_norm(x, z, **kw)
    with pytest.raises(ValueError):
        prm.block_norm(x.bfloat16(), z)     # fp32 block under a 16-bit stream
    with pytest.raises(ValueError):
        prm.block_norm(x, z[:2])
    with pytest.raises(N.PrmError):
        big = torch.zeros(1, 8200, device="cuda")
        prm.block_norm(big, big.clone())
    r, y, stats = prm.block_norm(x, z)
    with pytest.raises(ValueError):
        prm.block_norm_backward(y, None, r, z, stats[:3])


# ---------------------------------------------------------------- embedding
def _token_set(T, V, gen, pattern):
    if pattern == "uniform":
        return torch.randint(0, V, (T,), generator=gen)
    if pattern == "one":
        return torch.full((T,), V - 1, dtype=torch.int64)
    if pattern == "padding":
        return torch.full((T,), -1, dtype=torch.int64)
    if pattern == "ordered":
        return torch.arange(T) % V
    # a few long runs, many short ones, padding of both kinds
    t = (torch.rand(T, generator=gen) ** 4 * V).long().clamp_(0, V - 1)
    t[torch.rand(T, generator=gen) < 0.1] = -100
    t[torch.rand(T, generator=gen) < 0.05] = V
    t[torch.rand(T, generator=gen) < 0.02] = 2 ** 40
    return t


@pytest.mark.parametrize("T", [1, 2, 31, 33, 500])
@pytest.mark.parametrize("d", [1, 7, 8, 64, 100, 1001, 2048, 2056, 5120])
def test_embedding_lookup_is_exact(T, d):
    g = _gen(T + d)
    V = 211
    tok = _token_set(T, V, g, "mixed").cuda()
    for tt, ot in ((FP32, BF16), (FP32, FP32), (BF16, BF16), (BF16, FP32), (FP16, FP16), (FP32, FP16)):
        table = _rand(g, V, d, dtype=tt)
        got = prm.embedding(tok, table, scale=1.5, dtype=ot)
        ok = (tok >= 0) & (tok < V)
        want = torch.where(ok[:, None], table[tok.clamp(0, V - 1)].float() * 1.5, torch.zeros(1, device="cuda")).to(ot)
        assert torch.equal(got, want), (tt, ot)


def _check_embedding_grad(tok, V, d, dt, gt, scale=0.75, accumulate=False, seed=0):
    g = _gen(seed)
    dout = _rand(g, *tok.shape, d, dtype=dt)
    out = _rand(g, V, d, dtype=gt) if accumulate else None
    old = host64(out) if accumulate else 0.0
    got = prm.embedding_backward(dout, tok, V, scale=scale, dtype=gt, out=out.clone() if accumulate else None,
                                 accumulate=accumulate)
    assert got.dtype == gt and got.shape == (V, d)
    tok_h, dout_h = tok.cpu().numpy().reshape(-1), host64(dout).reshape(-1, d)
    ok = (tok_h >= 0) & (tok_h < V)
    want, mag, count = np.zeros((V, d)), np.zeros((V, d)), np.zeros(V)
    np.add.at(want, tok_h[ok], dout_h[ok])
    np.add.at(mag, tok_h[ok], np.abs(dout_h[ok]))
    np.add.at(count, tok_h[ok], 1)
    want = want * scale + old
    # n fp32 additions, the scaling, the addition to what was there and the final rounding
    bound = ((count + 2)[:, None] * mag * scale + np.abs(old)) * 2.0 ** -24 + U[gt] * np.abs(want) + 2.0 ** -25 * (gt == FP16)
    assert (np.abs(host64(got) - want) <= bound).all()
    again = prm.embedding_backward(dout, tok, V, scale=scale, dtype=gt, out=out.clone() if accumulate else None,
                                   accumulate=accumulate)
    assert torch.equal(got, again)
    return got


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 65, 1000, 2048, 2049, 5000, 20000])
@pytest.mark.parametrize("pattern", ["uniform", "one", "padding", "ordered", "mixed"])
def test_embedding_gradient_runs(T, pattern):
    g = _gen(T)
    for V in (1, 2, 300, 511, 513, 70001):
        tok = _token_set(T, V, g, pattern).cuda()
        _check_embedding_grad(tok, V, 16 if V > 1000 else 40, BF16, FP32)


@pytest.mark.parametrize("T", [16400, 65536, 65537, 140000])
@pytest.mark.parametrize("pattern", ["uniform", "one", "mixed"])
def test_embedding_gradient_many_tokens(T, pattern):
    """Above and below what one cluster sorts; runs over many blocks of pieces."""
    g = _gen(T)
    for V in (3, 1000, 300007):     # 300007: three passes over the digits
        tok = _token_set(T, V, g, pattern).cuda()
        _check_embedding_grad(tok, V, 12, BF16, FP32)
        _check_embedding_grad(tok, V, 8, FP32, FP32, accumulate=True)


def test_embedding_gradient_run_ends():
    """Runs that start and end at every place around the edges of a piece and
    of a block of pieces (16 entries, 16 pieces), up to the last entry."""
    T = 17000
    g = _gen(8)
    for first in (0, 1, 15, 16, 17, 239, 255, 256, 257, 511, 512, 513, 529):
        for length in (1, 15, 16, 17, 240, 256, 272, 497, 512, 1024, 1040, 5000, T - first):
            tok = torch.arange(T) + 10
            tok[first:first + length] = 5 + first     # sorted: below entries that come later, above those before
            tok[:first] = torch.arange(first) % 5
            tok = tok[torch.randperm(T, generator=g)].cuda()
            _check_embedding_grad(tok, T + 10, 4, BF16, FP32)


def test_embedding_gradient_off_16_bytes():
    """dout or the gradient's buffer off 16 bytes: rows read from memory, or written element by element."""
    g = _gen(9)
    tok = _token_set(700, 90, g, "mixed").cuda()
    for d in (64, 1001, 2056):
        dout = _rand(g, 700, d, dtype=BF16)
        want = prm.embedding_backward(dout, tok, 90)
        odd = torch.zeros(700 * d + 1, dtype=BF16, device="cuda")[1:].view(700, d)
        odd.copy_(dout)
        assert torch.equal(prm.embedding_backward(odd, tok, 90), want)
        out = torch.full((90 * d + 1,), float("nan"), device="cuda")[1:].view(90, d)
        assert prm.embedding_backward(dout, tok, 90, out=out) is out
        assert torch.equal(out, want)
        table = torch.randn(90 * d + 1, device="cuda")[1:].view(90, d)
        assert torch.equal(prm.embedding(tok, table, dtype=BF16), prm.embedding(tok, table.clone(), dtype=BF16))


@pytest.mark.parametrize("d", [8, 64, 1001, 2048, 4104])
def test_embedding_lookup_of_many_tokens(d):
    g = _gen(d)
    T = 20001 if d > 512 else 320003      # enough for several rows per thread, with a rest
    tok = _token_set(T, 500, g, "mixed").cuda()
    table = _rand(g, 500, d)
    got = prm.embedding(tok, table, scale=0.5, dtype=BF16)
    ok = (tok >= 0) & (tok < 500)
    want = torch.where(ok[:, None], table[tok.clamp(0, 499)] * 0.5, torch.zeros(1, device="cuda")).to(BF16)
    assert torch.equal(got, want)


@pytest.mark.parametrize("d", [1, 5, 8, 100, 1001, 2048, 2056, 5120])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_gradient_widths_and_types(d, accumulate):
    g = _gen(d)
    tok = _token_set(900, 333, g, "mixed").cuda()
    for dt, gt in ((BF16, FP32), (BF16, BF16), (FP32, FP32), (FP16, FP16), (FP32, BF16)):
        _check_embedding_grad(tok, 333, d, dt, gt, accumulate=accumulate)


def test_embedding_token_layouts():
    g = _gen(4)
    table = _rand(g, 50, 24)
    tok = _token_set(60, 50, g, "mixed").cuda()
    dout = _rand(g, 60, 24)
    a, ga = prm.embedding(tok, table), prm.embedding_backward(dout, tok, 50)
    grid = tok.view(6, 10)
    turned = grid.t().contiguous().t()
    small = tok.clone()
    small[small > 2 ** 31 - 1] = 50
    for t in (grid, turned, small.int().view(6, 10)):
        assert torch.equal(prm.embedding(t, table).view(60, 24), a)
        assert torch.equal(prm.embedding_backward(dout.view(6, 10, 24), t, 50), ga)
    wide = torch.zeros(60, 30, device="cuda")
    wide[:, 3:27] = dout
    assert torch.equal(prm.embedding_backward(wide[:, 3:27], tok, 50), ga)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gs = prm.embedding_backward(dout, tok, 50, stream=s)
    es = prm.embedding(tok, table, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(gs, ga) and torch.equal(es, a)


def test_embedding_no_tokens():
    tok = torch.zeros(0, dtype=torch.int64, device="cuda")
    assert prm.embedding(tok, torch.ones(5, 8, device="cuda")).shape == (0, 8)
    assert (prm.embedding_backward(torch.zeros(0, 8, device="cuda"), tok, 5) == 0).all()


def test_embedding_offsets_past_32_bits():
    V, d = 600000, 4096
    table = torch.zeros(V, d, dtype=BF16, device="cuda")
    table[-3:] = 2.0
    tok = torch.tensor([V - 1, 0, V - 3, V - 1], device="cuda")
    out = prm.embedding(tok, table)
    assert (out[[0, 2, 3]] == 2).all() and (out[1] == 0).all()
    del table
    grad = prm.embedding_backward(torch.ones(4, d, dtype=BF16, device="cuda"), tok, V, dtype=BF16)
    assert (grad[V - 1] == 2).all() and (grad[V - 3] == 1).all() and (grad[0] == 1).all()
    assert grad[1:V - 3].abs().max() == 0 and (grad[V - 2] == 0).all()


def test_embedding_refusals():
    tok = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        prm.embedding(tok.float(), torch.zeros(4, 8, device="cuda"))
    with pytest.raises(ValueError):
        prm.embedding(tok, torch.zeros(4, 8, device="cuda").t())
    with pytest.raises(ValueError):
        prm.embedding_backward(torch.zeros(3, 8, device="cuda"), tok, 5)
    with pytest.raises(ValueError):
        prm.embedding_backward(torch.zeros(4, 8, device="cuda"), tok, 5, out=torch.zeros(5, 9, device="cuda"))
