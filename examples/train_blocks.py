"""A small language model trained with the framework alone: token embedding,
a stack of blocks (norm, gated feed-forward, join into the residual stream),
and the optimizer that owns their parameters -- PR-Muon for the feed-forward
matrices, AdamW for the norms' gains and the token table.

    python examples/train_blocks.py [--steps 60] [--layers 4] [--width 256]

Each block computes, over the residual stream r (fp32) and its input y (bf16):

    z    = gated_ffn(y)
    r, y = block_norm(r, z)        r + N(z) post_weight, then N(r) pre_weight

The output layer is the token table once more (tied), with torch's own matrix
product and cross entropy. The data is a random but fixed next-token map with
noise, so the loss can fall from log(vocab) towards the noise's entropy.

Weights are fp32; the bf16 copies that the products read are refreshed every
step. The backward pass writes the matrices' gradients straight into the
buffers that PeriodicRowMuon has registered.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import matrix_aware_optimizer_gb300 as prm  # noqa: E402

BF16 = torch.bfloat16


class Model:
    """Parameters, optimizer state and the two passes, written out."""

    def __init__(self, vocab, width, hidden, layers, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape, std):
            return torch.randn(*shape, generator=g, device="cuda") * std

        self.scale = math.sqrt(width)  # of the embedding, so that its rows have about unit elements
        self.table = randn(vocab, width, std=1.0 / self.scale)
        self.first = torch.ones(width, device="cuda")
        self.post = [torch.full((width,), 0.5, device="cuda") for _ in range(layers)]
        self.pre = [torch.ones(width, device="cuda") for _ in range(layers)]
        self.matrices = []  # per layer: w_gate, w_up, w_down
        for _ in range(layers):
            self.matrices += [randn(hidden, width, std=width ** -0.5), randn(hidden, width, std=width ** -0.5),
                              randn(width, hidden, std=hidden ** -0.5)]
        self.work = [w.to(BF16) for w in self.matrices]
        self.grads = [torch.empty_like(w) for w in self.work]
        self.muon = prm.PeriodicRowMuon(self.matrices, [torch.zeros_like(w) for w in self.matrices], self.grads)
        self.vectors = [self.table, self.first] + self.post + self.pre
        self.moments = [(torch.zeros_like(v), torch.zeros_like(v)) for v in self.vectors]

    def layer(self, k):
        return self.work[3 * k:3 * k + 3]

    def loss_and_gradients(self, tokens, targets):
        """The loss, and the gradients of `vectors`; the matrices' go to self.grads."""
        layers = len(self.post)
        x = prm.embedding(tokens, self.table, scale=self.scale)
        r, y, stats = prm.block_norm(x, pre_weight=self.first, dtype=BF16)
        saved = [(r, None, stats)]
        inputs = []
        for k in range(layers):
            z, ffn = prm.gated_ffn(y, *self.layer(k), save=True)
            inputs.append((y, ffn))
            r, y, stats = prm.block_norm(r, z, post_weight=self.post[k], pre_weight=self.pre[k])
            saved.append((r, z, stats))

        # output layer and loss, in torch: logits = y table^T
        table = self.table.to(BF16)
        logits = (y @ table.t()).float()
        log_p = torch.log_softmax(logits, dim=-1)
        n = targets.numel()
        loss = -log_p[torch.arange(n, device="cuda"), targets].mean()
        d_logits = log_p.exp_()
        d_logits[torch.arange(n, device="cuda"), targets] -= 1.0
        d_logits = (d_logits / n).to(BF16)
        dy = d_logits @ table
        d_table = (d_logits.t() @ y).float()

        dr, d_post, d_pre = None, [None] * layers, [None] * layers
        for k in reversed(range(layers)):
            r, z, stats = saved[k + 1]
            g = prm.block_norm_backward(dy, dr, r, z, stats, post_weight=self.post[k], pre_weight=self.pre[k])
            dr, d_post[k], d_pre[k] = g.dx, g.dpost_weight, g.dpre_weight
            y_in, ffn = inputs[k]
            dy = prm.gated_ffn_backward(g.dz, y_in, *self.layer(k), ffn, grads=self.grads[3 * k:3 * k + 3])[0]
        r, _, stats = saved[0]
        g = prm.block_norm_backward(dy, dr, r, None, stats, pre_weight=self.first)
        # the lookup's gradient joins the output layer's in the tied table's
        prm.embedding_backward(g.dx, tokens, self.table.shape[0], scale=self.scale, out=d_table, accumulate=True)
        return loss, [d_table, g.dpre_weight] + d_post + d_pre

    def step(self, t, tokens, targets, lr=0.01, lr_vectors=3e-3):
        loss, grads = self.loss_and_gradients(tokens, targets)
        self.muon.step(t, lr=lr, wd=0.0)
        for v, (m, s), g in zip(self.vectors, self.moments, grads):
            prm.adamw_step(v, m, s, g, t + 1, lr=lr_vectors)
        for w, master in zip(self.work, self.matrices):
            w.copy_(master)
        return loss


def batches(vocab, tokens, seed, noise=0.1):
    """Endless (tokens, targets): a fixed random successor for every token,
    replaced by a random one with probability `noise`."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    successor = torch.randperm(vocab, generator=g, device="cuda")
    while True:
        tok = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        target = successor[tok]
        wrong = torch.rand(tokens, generator=g, device="cuda") < noise
        yield tok, torch.where(wrong, torch.randint(0, vocab, (tokens,), generator=g, device="cuda"), target)


def main(steps=60, layers=4, width=256, hidden=704, vocab=1000, tokens=4096, seed=0, report=10):
    model = Model(vocab, width, hidden, layers, seed)
    losses = []
    for t, (tok, target) in zip(range(steps), batches(vocab, tokens, seed + 1)):
        losses.append(model.step(t, tok, target))
        if report and (t % report == 0 or t == steps - 1):
            print(f"step {t:4d}  loss {losses[-1].item():.4f}", flush=True)
    model.muon.sync_status()
    prm.blocks_sync_status()
    return [v.item() for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("steps", 60), ("layers", 4), ("width", 256), ("hidden", 704), ("vocab", 1000),
                        ("tokens", 4096), ("seed", 0)):
        ap.add_argument("--" + name, type=int, default=value)
    main(**vars(ap.parse_args()))
