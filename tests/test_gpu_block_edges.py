"""The block operators where rows, buffers, threads and limits meet their
edges. Comparisons and tolerances are those of test_gpu_blocks.py."""
import ctypes
import threading

import pytest
import torch

import matrix_aware_optimizer_gb300 as prm
from matrix_aware_optimizer_gb300 import native as N

from .gpu_helpers import ensure_built
from .test_gpu_blocks import BF16, FP16, FP32, _check_norm, _norm_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()
    N.load()
    yield
    prm.blocks_sync_status()


# ------------------------------------------- rows narrower than one 16-byte copy
@pytest.mark.parametrize("st,bt", [(FP32, FP32), (FP32, BF16), (BF16, BF16), (FP16, FP16)])
@pytest.mark.parametrize("d", [3, 5, 6, 7])
@pytest.mark.parametrize("B,L", [(2, 1), (5, 1), (6, 1), (7, 1), (10, 1), (14, 1), (40, 1), (9, 2)])
def test_norm_gradient_of_narrow_rows(B, L, d, st, bt):
    """A sample's rows are copied by themselves. Several samples at the end of
    a narrow tensor lie behind its last whole 16 bytes."""
    _check_norm(*_norm_case(B, L, d, "rms", st, bt, 1, 1, 1, 1, eps=1e-3))
    _check_norm(*_norm_case(B, L, d, "rms", st, bt, 0, 0, 0, 1, eps=1e-3))


@pytest.mark.parametrize("d,rows", [(3, 304 * 129 - 1), (3, 304 * 129 - 3), (5, 304 * 129 - 2), (7, 304 * 129)])
def test_norm_gradient_of_narrow_rows_without_samples(d, rows):
    """As many rows as leave one behind the last full step of 128 rows."""
    _check_norm(*_norm_case(1, rows, d, "rms", BF16, BF16, 1, 0, 1, 0, eps=1e-3))


# ------------------------------------------------------ threads of one process
def test_embedding_gradients_of_four_threads():
    """Threads that run gradients of the same types and different widths at
    once do not change each other's launches."""
    lib = N.load()
    T, V, kept, failures = 300, 40, [], []

    def call(d):
        """The library call for one width on a stream of its own, and its check."""
        g = torch.Generator(device="cuda").manual_seed(d)
        tok = torch.randint(0, V, (T,), generator=g, device="cuda")
        dout = torch.randn(T, d, generator=g, device="cuda")
        want = prm.embedding_backward(dout, tok, V)
        n = ctypes.c_size_t()
        assert lib.prm_embedding_backward_workspace(T, V, d, n) == N.PRM_OK
        ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
        out, stream = torch.empty_like(want), torch.cuda.Stream()
        kept.append((tok, dout, ws, stream))
        args = (dout.data_ptr(), N.PRM_FP32, tok.data_ptr(), 8, out.data_ptr(), N.PRM_FP32, 0, T, V, d, 1.0,
                ws.data_ptr(), n.value, stream.cuda_stream)
        return args, out, want

    # rows in whole vectors: 128 and 65 KB of shared memory; element by element: 192 and 112 KB
    calls = [call(d) for d in (2048, 1032, 15, 17)]
    torch.cuda.synchronize()

    def run(args):
        codes = {lib.prm_embedding_backward(*args) for _ in range(3000)}
        if codes != {N.PRM_OK}:
            failures.append((args[9], codes))

    threads = [threading.Thread(target=run, args=(c[0],)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures, failures
    for _, out, want in calls:
        assert torch.equal(out, want)


# ------------------------------------------------- what a forward pass left behind
def test_ffn_backward_refuses_what_another_call_saved():
    def inputs(f, dtype):
        g = torch.Generator(device="cuda").manual_seed(f)
        return [torch.randn(*s, generator=g, device="cuda").to(dtype) for s in ((1, 64), (f, 64), (f, 64), (64, f))]

    x, *ws = inputs(8, BF16)
    y, saved = prm.gated_ffn(x, *ws, act="gelu", save=True)
    prm.gated_ffn_backward(y, x, *ws, saved, act="gelu")
    with pytest.raises(ValueError):
        prm.gated_ffn_backward(y, x, *ws, saved)                      # silu is not what was saved
    with pytest.raises(ValueError):
        prm.gated_ffn_backward(y, x, *inputs(16, BF16)[1:], saved, act="gelu")   # as many bytes, more features
    half = inputs(8, FP16)
    with pytest.raises(ValueError):
        prm.gated_ffn_backward(y.half(), *half, saved, act="gelu")


# ------------------------------------------------------------ buffers in place
@pytest.mark.parametrize("st,bt", [(FP32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("d,off", [(48, 0), (2048, 0), (5120, 0), (8192, 0), (7, 0), (1001, 0), (3001, 0), (1001, 1),
                                   (64, 1)])
def test_norms_in_place(d, off, st, bt):
    """r over x, dx over dr and dz over dy give the bits of separate buffers,
    with whole vectors, odd rows and buffers off 16 bytes."""
    lib, stream = N.load(), torch.cuda.current_stream().cuda_stream
    B, L = 3, 211
    x, z, par, dy, dr, kw, eps = _norm_case(B, L, d, "layer", st, bt, 1, 1, 1, 1)
    code = {FP32: N.PRM_FP32, BF16: N.PRM_BF16}

    def copy(t):
        return torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")[off:].view(t.shape).copy_(t)

    p = {k: v.data_ptr() for k, v in par.items()}
    ld = par["gate"].stride(0)
    desc = N.prm_block_norm_desc(rows=B * L, rows_per_sample=L, d=d, kind=N.PRM_NORM_LAYER, stream_dtype=code[st],
                                 block_dtype=code[bt], alpha=kw["alpha"], eps=eps, gate_ld=ld, scale_ld=ld,
                                 shift_ld=ld, **p)
    n = ctypes.c_size_t()
    assert lib.prm_block_norm_workspace(desc, n) == N.PRM_OK
    ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")

    def forward(src, dst, y, stats):
        assert lib.prm_block_norm_forward(desc, src.data_ptr(), z.data_ptr(), dst.data_ptr(), y.data_ptr(),
                                          stats.data_ptr(), stream) == N.PRM_OK

    def backward(gy, gr, gx, gz, r, stats):
        cols = [torch.empty(d, device="cuda"), torch.empty(B, d, dtype=bt, device="cuda"),
                torch.empty(d, device="cuda"), torch.empty(B, d, dtype=bt, device="cuda"),
                torch.empty(B, d, dtype=bt, device="cuda")]
        assert lib.prm_block_norm_backward(desc, gy.data_ptr(), gr.data_ptr(), r.data_ptr(), z.data_ptr(),
                                           stats.data_ptr(), gx.data_ptr(), gz.data_ptr(),
                                           *(c.data_ptr() for c in cols), ws.data_ptr(), n.value, stream) == N.PRM_OK
        return cols

    x1, x2 = copy(x), copy(x)
    r, y1, y2 = copy(x), copy(z), copy(z)
    s1, s2 = (torch.empty(B * L, 4, device="cuda") for _ in range(2))
    forward(x1, r, y1, s1)
    forward(x2, x2, y2, s2)
    assert torch.equal(r, x2) and torch.equal(y1, y2) and torch.equal(s1, s2)
    gy, gr, gy2, gr2 = copy(dy), copy(dr), copy(dy), copy(dr)
    gx, gz = copy(dr), copy(dy)
    a = backward(gy, gr, gx, gz, r, s1)
    b = backward(gy2, gr2, gr2, gy2, r, s1)
    assert torch.equal(gx, gr2) and torch.equal(gz, gy2)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


# ----------------------------------------------------------------- many rows
def test_norm_of_more_rows_than_31_bits_count():
    rows = (1 << 31) + 77
    x = torch.zeros(rows, 1, dtype=BF16, device="cuda")
    x[-100:, 0] = torch.linspace(-2.0, 2.0, 100, device="cuda")
    y = torch.empty_like(x)
    desc = N.prm_block_norm_desc(rows=rows, rows_per_sample=rows, d=1, kind=N.PRM_NORM_RMS, stream_dtype=N.PRM_BF16,
                                 block_dtype=N.PRM_BF16, alpha=1.0, eps=0.25)
    rc = N.load().prm_block_norm_forward(desc, x.data_ptr(), None, None, y.data_ptr(), None,
                                         torch.cuda.current_stream().cuda_stream)
    assert rc == N.PRM_OK
    v = x[-100:].double()
    want = v / torch.sqrt(v * v + 0.25)
    # one rounding to bf16 and a few in fp32
    assert ((y[-100:].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want.abs()).all()
    assert torch.count_nonzero(y[:-100]) == 0
