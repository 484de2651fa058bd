"""fp64 restatement of the transformer-block operators: the gated
feed-forward block, the norms around a block and the token embedding, each
with its gradient written out.

TEST INFRASTRUCTURE ONLY (see the package docstring). Plain numpy from the
formulas in include/prm_blocks.h; tests/test_blocks_cpu.py checks every
gradient here against central differences of the forward function.
"""
from __future__ import annotations

import math

import numpy as np


def _erf(v):
    return np.vectorize(math.erf, otypes=[np.float64])(v)


def activation(g, act):
    """(act(g), act'(g))."""
    g = np.asarray(g, dtype=np.float64)
    if act == "silu":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        c = 0.5 * (1.0 + _erf(g / math.sqrt(2.0)))
        return g * c, c + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = np.tanh(k * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * g * g)
    raise ValueError(act)


def gated_ffn(x, wg, wu, wd, act):
    a, _ = activation(x @ wg.T, act)
    return (a * (x @ wu.T)) @ wd.T


def gated_ffn_backward(dy, x, wg, wu, wd, act):
    """(dx, dwg, dwu, dwd)."""
    g, u = x @ wg.T, x @ wu.T
    a, da = activation(g, act)
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ (a * u)


def _stats(v, kind, eps):
    m = v.mean(-1, keepdims=True) if kind == "layer" else np.zeros_like(v[..., :1])
    return m, 1.0 / np.sqrt(((v - m) ** 2).mean(-1, keepdims=True) + eps)


def _mod(m):
    return 0.0 if m is None else m[:, None, :]


def block_join(x, z, kind, alpha, eps, post=None, gate=None):
    """r of x, z [samples, rows, d]; gate [samples, d]."""
    p = z
    if post is not None:
        m, s = _stats(z, kind, eps)
        p = (z - m) * s * post
    return alpha * x + (p if gate is None else gate[:, None, :] * p)


def block_next(r, kind, eps, pre=None, scale=None, shift=None):
    """y of r."""
    m, s = _stats(r, kind, eps)
    n = (r - m) * s * (1.0 if pre is None else pre)
    return n * (1.0 + _mod(scale)) + _mod(shift)


def _norm_grad(dn, n, s, kind):
    out = dn - n * (dn * n).mean(-1, keepdims=True)
    if kind == "layer":
        out = out - dn.mean(-1, keepdims=True)
    return s * out


def block_backward(dy, dr, r, z, kind, alpha, eps, post=None, gate=None, pre=None, scale=None, shift=None):
    """dict of dx, dz, dpost, dgate, dpre, dscale, dshift (None where absent);
    dy, dr and z may be None."""
    out = dict.fromkeys(("dx", "dz", "dpost", "dgate", "dpre", "dscale", "dshift"))
    D = np.zeros_like(r) if dr is None else dr.copy()
    if dy is not None:
        m, s = _stats(r, kind, eps)
        n = (r - m) * s
        w = 1.0 if pre is None else pre
        dn = dy * (1.0 + _mod(scale))
        if scale is not None:
            out["dscale"] = (dy * n * w).sum(1)
        if shift is not None:
            out["dshift"] = dy.sum(1)
        if pre is not None:
            out["dpre"] = (dn * n).sum((0, 1))
        D = D + _norm_grad(dn * w, n, s, kind)
    out["dx"] = alpha * D
    if z is None:
        return out
    p, q = z, None
    if post is not None:
        m, s = _stats(z, kind, eps)
        q = (z - m) * s
        p = q * post
    dp = D
    if gate is not None:
        out["dgate"] = (D * p).sum(1)
        dp = D * gate[:, None, :]
    if post is not None:
        out["dpost"] = (dp * q).sum((0, 1))
        dp = _norm_grad(dp * post, q, s, kind)
    out["dz"] = dp
    return out


def embedding(tokens, table, scale):
    tokens = np.asarray(tokens)
    ok = (tokens >= 0) & (tokens < table.shape[0])
    out = table[np.where(ok, tokens, 0)] * scale
    out[~ok] = 0.0
    return out


def embedding_backward(dout, tokens, vocab, scale):
    grad = np.zeros((vocab, dout.shape[-1]))
    for t, v in enumerate(np.asarray(tokens).reshape(-1)):
        if 0 <= v < vocab:
            grad[v] += dout.reshape(-1, dout.shape[-1])[t] * scale
    return grad
