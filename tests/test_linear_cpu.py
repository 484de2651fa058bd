"""CPU checks of the linear layer: the fp64 oracle's gradients against
differences, the C ABI's refusals (none reaches the device) and the tensor
API's."""
import ctypes

import numpy as np
import pytest
import torch

from matrix_aware_optimizer_gb300 import attention, build, native as N
from oracle import attention as O


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return N.load()


@pytest.mark.parametrize("act", [None, "silu", "gelu", "gelu_tanh"])
def test_linear_gradient_against_differences(act):
    rng = np.random.default_rng(6)
    x, w, b, dy = (rng.standard_normal(s) for s in ((3, 4), (5, 4), (5,), (3, 5)))
    res, h = rng.standard_normal((3, 5)), 1e-5
    for grad, a in zip(O.linear_backward(dy, x, w, b, act), (x, w, b)):
        for i in np.ndindex(*a.shape):
            keep = a[i]
            a[i] = keep + h
            up = (O.linear(x, w, b, act, res) * dy).sum()
            a[i] = keep - h
            down = (O.linear(x, w, b, act, res) * dy).sum()
            a[i] = keep
            # truncation h^2 f''' / 6 ~ 1e-10 and cancellation 2^-53 |f| / h ~ 1e-10, with a margin of 100
            assert abs(grad[i] - (up - down) / (2 * h)) <= 1e-8


def test_linear_refusals(lib):
    def fwd(x=16, ldx=64, w=16, b=16, r=None, ldr=0, y=16, yt=N.PRM_BF16, pre=None, ws=256, size=1 << 30, T=40, n=64,
            k=64, act=0, dtype=N.PRM_BF16):
        return lib.prm_linear_forward(x, ldx, w, b, r, ldr, y, yt, pre, ws, size, T, n, k, act, dtype, None)

    def back(dy=16, lddy=64, dyt=N.PRM_BF16, x=16, ldx=64, w=16, pre=16, dx=16, dw=16, db=16, ws=256, size=1 << 30,
             T=40, n=64, k=64, act=0, dtype=N.PRM_BF16):
        return lib.prm_linear_backward(dy, lddy, dyt, x, ldx, w, pre, dx, dw, db, ws, size, T, n, k, act, dtype, None)

    for call in (fwd, back):
        for bad in (dict(act=4), dict(act=-1), dict(dtype=N.PRM_FP32), dict(T=-1), dict(n=0), dict(k=0), dict(x=None),
                    dict(w=None), dict(ldx=56)):
            assert call(**bad) == N.PRM_ERR_INVALID_ARG, bad
        for bad in (dict(n=60), dict(k=60), dict(ldx=68), dict(x=8), dict(w=8), dict(pre=8), dict(ws=128)):
            assert call(**bad) == N.PRM_ERR_ALIGNMENT, bad
        for bad in (dict(T=1 << 31), dict(n=1 << 24), dict(k=1 << 24), dict(T=1 << 30, n=1 << 23)):
            assert call(**bad) == N.PRM_ERR_UNSUPPORTED, bad
    assert fwd(T=0, x=None) == N.PRM_OK
    assert fwd(yt=N.PRM_FP32) == N.PRM_ERR_INVALID_ARG                  # fp32 without a residual
    assert fwd(yt=N.PRM_FP16, r=16, ldr=64) == N.PRM_ERR_INVALID_ARG
    assert fwd(r=16, ldr=56) == N.PRM_ERR_INVALID_ARG and fwd(r=16, ldr=68) == N.PRM_ERR_ALIGNMENT
    assert fwd(y=None) == N.PRM_ERR_INVALID_ARG and fwd(b=8) == N.PRM_ERR_ALIGNMENT
    # some tiles behind a full round, split along k
    assert fwd(T=5120, n=4096, k=2048, ldx=2048, size=10) == N.PRM_ERR_WORKSPACE
    assert back(dy=None) == N.PRM_ERR_INVALID_ARG and back(lddy=56) == N.PRM_ERR_INVALID_ARG
    assert back(pre=None) == N.PRM_ERR_INVALID_ARG and back(dyt=N.PRM_FP16) == N.PRM_ERR_INVALID_ARG
    assert back(lddy=68) == N.PRM_ERR_ALIGNMENT and back(dx=8) == N.PRM_ERR_ALIGNMENT
    assert back(dw=8) == N.PRM_ERR_ALIGNMENT and back(db=2) == N.PRM_ERR_ALIGNMENT
    assert back(size=10) == N.PRM_ERR_WORKSPACE and back(ws=None) == N.PRM_ERR_WORKSPACE
    assert back(dx=None, dw=None, db=None) == N.PRM_OK
    n = ctypes.c_size_t()
    assert lib.prm_linear_sizes(4, 64, 63, n, n) == N.PRM_ERR_ALIGNMENT
    assert lib.prm_linear_sizes(4, 64, 64, None, n) == N.PRM_ERR_INVALID_ARG


def test_linear_tensor_api_refuses():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        attention.linear(x, w)
    with pytest.raises(ValueError):
        attention.linear(x, w, act="relu")
    with pytest.raises(ValueError):
        attention.linear_backward(x, x, w, attention.LinearSaved(None, 4, 32, None, torch.bfloat16))
