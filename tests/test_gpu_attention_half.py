"""The attention half of a block as its operators are used together: projected
queries, keys and values in one tensor, turned in place, attended to, projected
back and joined into an fp32 residual stream through dropout, and the way back
into the buffers that the optimizer would own. Every step is compared with the
fp64 oracle on what that step was given. Then the same on other streams, at the
same time, and in a captured graph."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_gb300 as prm
from matrix_aware_optimizer_gb300 import native as N
from oracle import attention as O

from .gpu_helpers import ensure_built, host64
from .test_gpu_attention import _check_attention, _check_rotary
from .test_gpu_linear import _check_linear

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()
    N.load()
    yield
    prm.blocks_sync_status()


class Half:
    """Sizes, parameters and the two passes."""

    def __init__(self, B, L, H, Hkv, D, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.L, self.H, self.Hkv, self.D = B, L, H, Hkv, D
        self.d, self.n = H * D, (H + 2 * Hkv) * D

        def randn(*shape, std=1.0, dtype=BF16):
            return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()

        self.w_qkv, self.b_qkv = randn(self.n, self.d, std=self.d ** -0.5), randn(self.n, std=0.1, dtype=FP32)
        self.w_out, self.b_out = randn(self.d, self.d, std=self.d ** -0.5), randn(self.d, std=0.1, dtype=FP32)
        self.y, self.r = randn(B, L, self.d), randn(B, L, self.d, dtype=FP32)
        self.dr = randn(B, L, self.d, dtype=FP32)
        self.positions = torch.arange(50, 50 + L, device="cuda")
        self.plan = prm.rotary_plan(D // 2 // 2 * 2)
        self.lengths = torch.tensor([L - 3 * b for b in range(B)], device="cuda", dtype=torch.int32)
        self.grads = [torch.empty_like(self.w_qkv), torch.empty_like(self.w_out)]

    def run(self, stream=None, seed=7):
        """Everything the two passes compute, by name."""
        B, L, H, Hkv, D = self.B, self.L, self.H, self.Hkv, self.D
        kw = dict(stream=stream)
        qkv, s_qkv = prm.linear(self.y, self.w_qkv, self.b_qkv, save=True, **kw)
        heads = qkv.view(B, L, H + 2 * Hkv, D)
        plain = None if stream is not None else heads.clone()
        prm.rotary(heads[:, :, :H + Hkv], self.positions, self.plan, out=heads[:, :, :H + Hkv], **kw)
        q, k, v = heads.split([H, Hkv, Hkv], dim=2)
        o, s_o = prm.cross_attention(q, k, v, self.lengths, save=True, **kw)
        z, s_z = prm.linear(o.view(B, L, self.d), self.w_out, self.b_out, save=True, **kw)
        r = prm.dropout(z, 0.2, seed, residual=self.r, **kw)
        dz = prm.dropout_backward(self.dr, 0.2, seed, dtype=BF16, **kw)
        do, _, db_out = prm.linear_backward(dz, o.view(B, L, self.d), self.w_out, s_z, grad=self.grads[1], **kw)
        d_heads = torch.empty_like(heads)
        dq, dk, dv = d_heads.split([H, Hkv, Hkv], dim=2)
        prm.cross_attention_backward(do.view(B, L, H, D), q, k, v, o, s_o, self.lengths, grads=(dq, dk, dv), **kw)
        turned = None if stream is not None else d_heads.clone()
        prm.rotary_backward(d_heads[:, :, :H + Hkv], self.positions, self.plan, out=d_heads[:, :, :H + Hkv], **kw)
        dy, _, db_qkv = prm.linear_backward(d_heads.view(B, L, self.n), self.y, self.w_qkv, s_qkv, grad=self.grads[0],
                                            **kw)
        return dict(plain=plain, heads=heads, o=o, z=z, r=r, dz=dz, do=do, db_out=db_out, turned=turned,
                    d_heads=d_heads, dy=dy, db_qkv=db_qkv, dw_qkv=self.grads[0], dw_out=self.grads[1])


SIZES = [(2, 70, 4, 2, 64), (3, 200, 2, 2, 72), (1, 1, 8, 2, 128)]


@pytest.mark.parametrize("sizes", SIZES)
def test_every_step_of_a_run(sizes):
    m = Half(*sizes)
    B, L, H, Hkv, D = sizes
    x = m.run()
    rows = B * L
    flat = lambda t: t.reshape(rows, -1)  # noqa: E731
    _check_linear(flat(m.y), m.w_qkv, m.b_qkv, None, flat(x["d_heads"]), None,
                  (flat(x["plain"]), flat(x["dy"]), x["dw_qkv"], x["db_qkv"]))
    turning = H + Hkv
    _check_rotary(x["plain"][:, :, :turning].contiguous(), m.positions, m.plan.dim, "half",
                  y=x["heads"][:, :, :turning])
    assert torch.equal(x["heads"][:, :, turning:], x["plain"][:, :, turning:])
    q, k, v = x["heads"].split([H, Hkv, Hkv], dim=2)
    _check_attention(q, k, v, x["do"].view(B, L, H, D), m.lengths.tolist(),
                     calls=(x["o"],) + tuple(x["turned"].split([H, Hkv, Hkv], dim=2)))
    _check_linear(flat(x["o"]), m.w_out, m.b_out, None, flat(x["dz"]), None,
                  (flat(x["z"]), flat(x["do"]), x["dw_out"], x["db_out"]))
    keep = O.kept(rows * m.d, 0.2, 7).reshape(B, L, m.d)
    z, r, dr = host64(x["z"]), host64(m.r), host64(m.dr)
    want = r + np.where(keep, z / 0.8, 0.0)
    assert (np.abs(host64(x["r"]) - want) <= 5 * 2.0 ** -24 * (np.abs(want) + np.abs(z / 0.8))).all()
    want = np.where(keep, dr / 0.8, 0.0)
    assert (np.abs(host64(x["dz"]) - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want)).all()
    _check_rotary(x["turned"][:, :, :turning].contiguous(), m.positions, m.plan.dim, "half", inverse=True,
                  y=x["d_heads"][:, :, :turning])


def _same(a, b):
    for name in a:
        if a[name] is not None and b[name] is not None:
            assert torch.equal(a[name], b[name]), name


def _kept(x):
    return {name: None if t is None else t.clone() for name, t in x.items()}


@pytest.mark.parametrize("sizes", SIZES)
def test_on_another_stream(sizes):
    m = Half(*sizes)
    want = _kept(m.run())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):          # the stream is the current one
        inside = _kept(m.run())
    got = m.run(stream=side)               # and given with the call
    torch.cuda.synchronize()
    _same(inside, want)
    _same(got, want)


def test_two_runs_at_the_same_time():
    models = [Half(2, 300, 4, 2, 64, seed=s) for s in range(2)]
    want = [_kept(m.run()) for m in models]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in models]
    for _ in range(5):
        got = []
        for m, s in zip(models, streams):
            with torch.cuda.stream(s):
                got.append(m.run())
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            _same(g, w)


@pytest.mark.parametrize("sizes", SIZES + [(1, 1500, 3, 3, 128)])
def test_captured_and_replayed(sizes):
    m = Half(*sizes)
    seed = torch.tensor([7], device="cuda")
    m.run(seed=seed)                       # (kernels are set up outside of a capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x = m.run(seed=seed)
    for s in range(3):
        g = torch.Generator().manual_seed(100 + s)
        m.y.copy_((torch.randn(m.y.shape, generator=g)).to(BF16))
        m.dr.copy_(torch.randn(m.dr.shape, generator=g))
        m.lengths.copy_(torch.tensor([max(0, m.L - 40 * s - b) for b in range(m.B)]))
        seed.fill_(1000 + s)
        graph.replay()
        torch.cuda.synchronize()
        got = _kept(x)
        _same(got, m.run(seed=1000 + s))


def test_long_cache_offsets_pass_32_bits():
    """Keys and values whose last rows lie behind 2^32 bytes and 2^31 elements of their start."""
    B, Lk, Hkv, D = 2, 40, 2, 64
    pitch = (1 << 31) // (Lk - 1) // 8 * 8 + 8             # elements from token to token
    store = torch.zeros(pitch * (Lk - 1) + 2 * B * Hkv * D, dtype=BF16, device="cuda")
    kv = store.as_strided((2, B, Lk, Hkv, D), (B * Hkv * D, Hkv * D, pitch, D, 1))
    assert kv[1, 1, -1, -1].data_ptr() - store.data_ptr() > 1 << 32
    g = torch.Generator().manual_seed(3)
    kv.copy_(torch.randn(2, B, Lk, Hkv, D, generator=g).to(BF16))
    for Lq in (1, 30):
        q = torch.randn(B, Lq, 2 * Hkv, D, generator=g).to(BF16).cuda()
        near = kv.contiguous()
        o, saved = prm.cross_attention(q, kv[0], kv[1], save=True)
        want, saved2 = prm.cross_attention(q, near[0], near[1], save=True)
        assert torch.equal(o, want)
        far = torch.empty_like(store).as_strided(kv.shape, kv.stride())
        dq = torch.empty_like(q)
        prm.cross_attention_backward(q, q, kv[0], kv[1], o, saved, grads=(dq, far[0], far[1]))
        a = prm.cross_attention_backward(q, q, near[0], near[1], want, saved2)
        assert torch.equal(dq, a[0]) and torch.equal(far[0], a[1]) and torch.equal(far[1], a[2])
        del far
    pos = torch.arange(Lk, device="cuda")
    plan = prm.rotary_plan(D)
    turned = prm.rotary(near[0], pos, plan)
    prm.rotary(kv[0], pos, plan, out=kv[0])
    assert torch.equal(kv[0], turned)


def test_rows_around_an_output_are_left():
    """Outputs that are slices of larger buffers: nothing around them is written."""
    B, L, H, D = 2, 37, 3, 72
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(B, L, H, D, generator=g).to(BF16).cuda() for _ in range(3))
    o, saved = prm.cross_attention(q, k, v, save=True)
    want = (o,) + prm.cross_attention_backward(q, q, k, v, o, saved)

    def hold():
        big = torch.full((B + 2, L + 4, H + 2, D + 8), 9.0, dtype=BF16, device="cuda")
        return big, big[1:1 + B, 2:2 + L, 1:1 + H, :D]

    held = [hold() for _ in range(4)]
    prm.cross_attention(q, k, v, out=held[0][1])
    prm.cross_attention_backward(q, q, k, v, o, saved, grads=[h[1] for h in held[1:]])
    for (big, part), w in zip(held, want):
        assert torch.equal(part, w)
        part.fill_(9.0)
        assert (big == 9.0).all()


def test_gradients_that_share_memory_are_refused():
    q = torch.zeros(1, 4, 2, 16, dtype=BF16, device="cuda")
    o, saved = prm.cross_attention(q, q, q, save=True)
    d = torch.empty_like(q)
    with pytest.raises(ValueError):
        prm.cross_attention_backward(q, q, q, q, o, saved, grads=(d, torch.empty_like(q), d))
