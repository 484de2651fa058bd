"""CPU checks of the operators of a block's attention half: the fp64 oracle
against known values and differences, the C ABI's declarations and refusals
(none reaches the device), and the tensor API's refusals."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from matrix_aware_optimizer_gb300 import attention, build, native as N
from oracle import attention as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return N.load()


def test_every_declared_symbol_is_exported_and_bound(lib):
    with open(os.path.join(ROOT, "include", "prm_attention.h")) as f:
        text = f.read()
    names = sorted(set(re.findall(r"PRM_API\s+[\w\s\*]+?\b(prm_\w+)\s*\(", text)))
    assert {"prm_rotary", "prm_dropout"} <= set(names)
    for name in names:
        assert hasattr(lib, name) and name in N.SIGNATURES, name


# --------------------------------------------------------- rotary positions
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_oracle_turns_back_and_keeps_distances(layout):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 5, 3, 10))
    pos = rng.integers(0, 1000, (2, 5))
    f = [1.0, 0.1, 0.01]
    y = O.rotary(x, pos, f, layout, amplitude=2.0)
    assert np.abs(O.rotary(y, pos, f, layout, amplitude=0.5, inverse=True) - x).max() < 1e-14
    assert np.array_equal(y[..., 6:], x[..., 6:])
    # a product of two turned heads depends on the distance of their positions alone
    a, b = rng.standard_normal((2, 1, 1, 1, 6))
    first = [(O.rotary(a, np.array([[p]]), f, layout) * O.rotary(b, np.array([[p + 7]]), f, layout)).sum()
             for p in (0, 13, 500)]
    assert np.ptp(first) < 1e-12
    # the transpose of the turn is what the gradient takes
    dy = rng.standard_normal(x.shape)
    left = (y * dy).sum()
    right = (x * O.rotary(dy, pos, f, layout, amplitude=2.0, inverse=True)).sum()
    assert abs(left - right) < 1e-11


def test_rotary_plan_frequencies():
    def turns(*a, **k):
        plan = attention.rotary_plan(*a, device="cpu", **k)
        return (plan.turns.numpy().astype(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * math.pi), plan
    f, plan = turns(8)
    assert np.allclose(f, 10000.0 ** (-np.arange(4) / 4), rtol=1e-14) and plan.amplitude == 1.0
    g, _ = turns(8, scaling="linear", factor=4.0)
    assert np.allclose(g, f / 4, rtol=1e-14)
    g, _ = turns(8, scaling="base", factor=4.0)
    assert np.isclose(g[0], f[0]) and np.isclose(g[-1], f[-1] / 4)
    g, plan = turns(64, scaling="ramp", factor=4.0, trained_length=8192)
    f, _ = turns(64)
    rounds = 8192 * f / (2 * math.pi)
    assert np.allclose(g[rounds > 32], f[rounds > 32]) and np.allclose(g[rounds < 1], f[rounds < 1] / 4)
    assert (np.diff(g) < 0).all() and np.isclose(plan.amplitude, 0.1 * math.log(4.0) + 1.0)
    # a frequency of a whole turn and more keeps its fraction
    g, _ = turns(2, base=1.0)
    assert np.isclose(g[0], 1.0)
    for bad in (dict(dim=7), dict(dim=0), dict(dim=8, layout="pairs"), dict(dim=8, scaling="double"),
                dict(dim=8, base=0.0), dict(dim=8, factor=float("inf")), dict(dim=8, scaling="ramp", fast=1.0),
                dict(dim=8, amplitude=float("nan"))):
        with pytest.raises(ValueError):
            attention.rotary_plan(**bad, device="cpu")


def _rotary(**kw):
    v = dict(samples=2, tokens=3, heads=4, head=16, dim=8, x_sample=192, x_token=64, x_head=16, y_sample=192,
             y_token=64, y_head=16, position_sample=3, position_token=1, position_bytes=8, layout=0, dtype=0,
             inverse=0, amplitude=1.0, reserved=0)
    v.update(kw)
    return N.prm_rotary_desc(*(v[k] for k, _ in N.prm_rotary_desc._fields_))


def test_amplitudes_beyond_fp32_are_refused():
    assert attention.rotary_plan(8, amplitude=3.4e38, device="cpu").amplitude == 3.4e38
    for amplitude in (3.5e38, -1e300, float("inf")):
        with pytest.raises(ValueError):
            attention.rotary_plan(8, amplitude=amplitude, device="cpu")



def test_rotary_refusals(lib):
    def call(x=16, pos=16, turns=16, y=32, **kw):
        return lib.prm_rotary(_rotary(**kw), x, pos, turns, y, None)
    for zero in ("samples", "tokens", "heads"):
        assert call(None, None, None, None, **{zero: 0}) == N.PRM_OK
        assert call(**{zero: -1}) == N.PRM_ERR_INVALID_ARG
    for bad in (dict(reserved=1), dict(dtype=3), dict(layout=2), dict(position_bytes=2),
                dict(amplitude=float("inf")), dict(amplitude=float("nan"))):
        assert call(**bad) == N.PRM_ERR_INVALID_ARG, bad
    for bad in (dict(dim=0), dict(dim=7), dict(dim=18), dict(head=0)):
        assert call(**bad) == N.PRM_ERR_SHAPE, bad
    for missing in ("x", "pos", "turns", "y"):
        assert call(**{missing: None}) == N.PRM_ERR_INVALID_ARG
    for bad in (dict(head=1 << 17, dim=8), dict(heads=(1 << 14) + 1), dict(tokens=1 << 31), dict(samples=1 << 41),
                dict(samples=1 << 30, tokens=1 << 30), dict(head=8192, dim=8192)):
        assert call(**bad) == N.PRM_ERR_UNSUPPORTED, bad
    assert call(x=16, y=16, y_token=128) == N.PRM_ERR_INVALID_ARG    # in place with other strides
    assert lib.prm_rotary(None, 16, 16, 16, 16, None) == N.PRM_ERR_INVALID_ARG


# ------------------------------------------------------------------ dropout
def test_philox_known_answers():
    # the published test vectors of the generator (zero counter and key; all ones, whose upper counter half
    # is not reachable here, is left out)
    assert O.philox(0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    words = np.array([O.philox(i, 12345) for i in range(4000)], dtype=np.float64) / 2.0 ** 32
    assert abs(words.mean() - 0.5) < 5 / math.sqrt(12 * words.size)


def test_dropout_oracle_keeps_its_share_and_is_linear():
    n, p = 20000, 0.3
    k = O.kept(n, p, 99, 5)
    assert abs(k.mean() - 0.7) < 5 * math.sqrt(p * (1 - p) / n)
    assert np.array_equal(O.kept(n - 8, p, 99, 7), k[8:])       # the offset counts blocks of four
    x = np.arange(12.0)
    assert np.array_equal(O.dropout(x, 0.0, 1), x) and not O.dropout(x, 1.0, 1).any()
    assert np.array_equal(O.dropout(x, 0.5, 1, residual=x) - x, O.dropout(x, 0.5, 1))


def test_dropout_refusals(lib):
    def call(x=16, t=0, res=None, y=16, yt=0, n=8, p=0.1):
        return lib.prm_dropout(x, t, res, y, yt, n, p, 1, None, 0, None)
    assert call(None, y=None, n=0) == N.PRM_OK
    for bad in (dict(t=3), dict(yt=9), dict(n=-1), dict(p=-0.1), dict(p=1.5), dict(p=float("nan")), dict(x=None),
                dict(y=None), dict(t=N.PRM_BF16, yt=N.PRM_FP16), dict(t=N.PRM_BF16, yt=N.PRM_FP32),
                dict(t=N.PRM_FP32, yt=N.PRM_BF16, res=16), dict(t=N.PRM_BF16, yt=N.PRM_FP16, res=16)):
        assert call(**bad) == N.PRM_ERR_INVALID_ARG, bad
    assert call(n=(1 << 41) + 1) == N.PRM_ERR_UNSUPPORTED


def test_tensor_api_refuses_cpu_tensors_and_wrong_arguments():
    x, plan = torch.zeros(2, 3, 4, 8), attention.rotary_plan(8, device="cpu")
    with pytest.raises(ValueError):
        attention.rotary(x, torch.zeros(3, dtype=torch.int64), plan)
    with pytest.raises(ValueError):
        attention.dropout(x, 0.1, 1)
    with pytest.raises(ValueError):
        attention.dropout_backward(x, 0.1, 1, dtype=torch.float64)
    with pytest.raises(ValueError):
        attention.dropout_backward(x.bfloat16(), 0.1, 1, dtype=torch.float32)


def test_distinct():
    t = torch.zeros(4, 6, 8)
    assert attention._distinct(t) and attention._distinct(t.transpose(0, 2)) and attention._distinct(t[:, ::2, 1:5])
    assert not attention._distinct(t.as_strided((2, 3), (1, 1))) and not attention._distinct(t[:1].expand(3, 6, 8))


# ---------------------------------------------------------- cross attention
def test_attention_gradient_against_differences():
    rng = np.random.default_rng(5)
    q, do = rng.standard_normal((2, 3, 3, 4, 2))
    k, v = rng.standard_normal((2, 3, 5, 2, 2))
    lengths, scale, h = [5, 2, 0], 0.7, 1e-5
    got = O.cross_attention_backward(do, q, k, v, lengths, scale)
    for grad, a in zip(got, (q, k, v)):
        for i in np.ndindex(*a.shape):
            keep = a[i]
            a[i] = keep + h
            up = (O.cross_attention(q, k, v, lengths, scale) * do).sum()
            a[i] = keep - h
            down = (O.cross_attention(q, k, v, lengths, scale) * do).sum()
            a[i] = keep
            # truncation h^2 f''' / 6 ~ 1e-10 and cancellation 2^-53 |f| / h ~ 1e-10, with a margin of 100
            assert abs(grad[i] - (up - down) / (2 * h)) <= 1e-8
    assert not got[0][2].any() and not got[1][1, 2:].any() and not got[2][2].any()


def _attn(strides=None, **kw):
    v = dict(batch=2, queries=3, keys=5, heads=4, kv_heads=2, head=16, key_lengths=None, length_bytes=0,
             dtype=N.PRM_BF16, scale=0.25, reserved=0)
    v.update(kw)
    names = ("q", "k", "v", "o", "grad_o", "dq", "dk", "dv")
    rows = {n: (5, 2) if n in ("k", "v", "dk", "dv") else (3, 4) for n in names}
    lay = {n: N.prm_attention_strides(t * h * 16, h * 16, 16) for n, (t, h) in rows.items()}
    lay.update({n: N.prm_attention_strides(*s) for n, s in (strides or {}).items()})
    return N.prm_attention_desc(**v, **lay)


def test_attention_refusals(lib):
    def fwd(q=16, k=16, v=16, o=16, lse=16, ws=None, n=0, **kw):
        return lib.prm_attention_forward(_attn(**kw), q, k, v, o, lse, ws, n, None)

    def back(g=16, q=16, k=16, v=16, o=16, lse=16, dq=16, dk=16, dv=16, ws=256, n=1 << 30, **kw):
        return lib.prm_attention_backward(_attn(**kw), g, q, k, v, o, lse, dq, dk, dv, ws, n, None)

    def sizes(**kw):
        a, b = ctypes.c_size_t(7), ctypes.c_size_t(7)
        rc = lib.prm_attention_workspace(_attn(**kw), a, b)
        return rc if rc else (a.value, b.value)

    for call in (fwd, back, sizes):
        for bad in (dict(reserved=1), dict(dtype=N.PRM_FP32), dict(batch=-1), dict(queries=-1), dict(keys=-1),
                    dict(heads=-1), dict(kv_heads=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                    dict(scale=float("inf")), dict(key_lengths=16, length_bytes=2)):
            assert call(**bad) == N.PRM_ERR_INVALID_ARG, bad
        for bad in (dict(head=0), dict(head=12), dict(kv_heads=3), dict(kv_heads=0)):
            assert call(**bad) == N.PRM_ERR_SHAPE, bad
        for bad in (dict(head=136), dict(queries=1 << 31), dict(keys=1 << 31), dict(heads=1 << 17, kv_heads=1 << 17),
                    dict(batch=1 << 21), dict(batch=1 << 20, heads=1 << 12),
                    dict(batch=1 << 12, heads=1 << 12, queries=1 << 17)):
            assert call(**bad) == N.PRM_ERR_UNSUPPORTED, bad
    for call in (fwd, back):
        for t in ("q", "k", "v", "o"):
            assert call(**{t: None}) == N.PRM_ERR_INVALID_ARG, t
            assert call(**{t: 8}) == N.PRM_ERR_ALIGNMENT, t
        for t in ("q", "k", "v", "o") + (("grad_o", "dq", "dk", "dv") if call is back else ()):
            assert call(strides={t: (640, 64, 12)}) == N.PRM_ERR_SHAPE, t      # heads overlap
            assert call(strides={t: (640, 64, 20)}) == N.PRM_ERR_ALIGNMENT, t
            assert call(strides={t: (1 << 38, 64, 16)}) == N.PRM_ERR_UNSUPPORTED, t
        assert call(lse=2) == N.PRM_ERR_ALIGNMENT
        assert call(ws=128, n=1 << 30) == N.PRM_ERR_ALIGNMENT
        assert call(batch=0) == N.PRM_OK and call(heads=0, kv_heads=0) == N.PRM_OK
    for t in ("g", "lse", "dq", "dk", "dv"):
        assert back(**{t: None}) == N.PRM_ERR_INVALID_ARG, t
    assert back(n=100) == N.PRM_ERR_WORKSPACE and back(ws=None) == N.PRM_ERR_WORKSPACE
    assert fwd(queries=0) == N.PRM_OK
    # a long key axis for few queries is split over CTAs, whose parts need room
    forward, backward = sizes(batch=1, heads=1, kv_heads=1, queries=300, keys=100000)
    assert forward > 0 and backward > 0
    lay = {t: (1 << 30, 16, 16) for t in ("q", "k", "v", "o")}
    assert fwd(batch=1, heads=1, kv_heads=1, queries=300, keys=100000, strides=lay) == N.PRM_ERR_WORKSPACE
    assert sizes(queries=0) == (0, 0) and sizes(keys=0) == (0, 0) and sizes(batch=0) == (0, 0)
    assert lib.prm_attention_workspace(_attn(), None, None) == N.PRM_ERR_INVALID_ARG
    assert lib.prm_attention_forward(None, 16, 16, 16, 16, None, None, 0, None) == N.PRM_ERR_INVALID_ARG


def test_attention_tensor_api_refuses():
    q, k = torch.zeros(2, 3, 4, 16, dtype=torch.bfloat16), torch.zeros(2, 5, 2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        attention.cross_attention(q, k, k)
    with pytest.raises(ValueError):
        attention.cross_attention_backward(q, q, k, k, q, attention.AttentionSaved(torch.zeros(2, 4, 3), 0.25, 5))
    assert attention._usable(q[:, :, 1:3]) and attention._usable(q.transpose(1, 2))
    assert not attention._usable(q[..., 1:9]) and not attention._usable(q.transpose(2, 3))
    assert not attention._usable(q[:, :1].expand(2, 3, 4, 16)) and not attention._usable(q[..., ::2])
