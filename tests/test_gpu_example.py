"""The block operators and the optimizer together, as the example uses them:
its gradients against autograd's of the same model in fp64, and a short run
whose loss has to fall."""
import math
import os
import sys

import pytest
import torch

from .gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    ensure_built()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_blocks
    finally:
        sys.path.pop(0)
    return train_blocks


def _autograd(model, tokens, targets):
    """Loss and gradients of the same model in fp64 on the CPU."""
    def leaf(t):
        return t.detach().double().cpu().requires_grad_()

    table, first = leaf(model.table), leaf(model.first)
    post, pre = [leaf(v) for v in model.post], [leaf(v) for v in model.pre]
    mats = [leaf(w) for w in model.work]

    def norm(v):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)

    r = table[tokens.cpu()] * model.scale
    y = norm(r) * first
    for k in range(len(post)):
        wg, wu, wd = mats[3 * k:3 * k + 3]
        z = (torch.nn.functional.silu(y @ wg.t()) * (y @ wu.t())) @ wd.t()
        r = r + norm(z) * post[k]
        y = norm(r) * pre[k]
    loss = torch.nn.functional.cross_entropy(y @ table.t(), targets.cpu())
    return loss.detach(), torch.autograd.grad(loss, [table, first] + post + pre + mats)


def test_gradients_of_the_whole_model(example):
    model = example.Model(vocab=100, width=64, hidden=168, layers=3, seed=3)
    tok, target = next(example.batches(100, 333, 4))
    loss, grads = model.loss_and_gradients(tok, target)
    ref_loss, ref = _autograd(model, tok, target)
    # bf16 activations between the operators: every value on the way carries 2^-8 at most, about a dozen of them
    assert abs(loss.item() - ref_loss.item()) <= 12 * 2.0 ** -8 * ref_loss.item()
    for got, want in zip(grads + model.grads, ref):
        err = (got.double().cpu() - want).norm() / want.norm()
        assert err <= 12 * 2.0 ** -8, err


def test_the_loss_falls(example):
    losses = example.main(steps=60, layers=2, width=128, hidden=352, vocab=200, tokens=2048, report=0)
    assert all(math.isfinite(v) for v in losses)
    # untrained, the tied table votes for the token itself: worse than knowing nothing, log(200)
    assert losses[0] > math.log(200)
    assert losses[-1] < 0.5 * math.log(200)
