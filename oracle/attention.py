"""fp64 restatement of the operators of a block's attention half: the
projection, cross attention, rotary positions and dropout, forward and
backward. Like the rest of this package it shares no code with the library."""
import math
from fractions import Fraction

import numpy as np

from .blocks import activation



# ------------------------------------------------------- rotary positions
def rotary(x, positions, inv_freq, layout, amplitude=1.0, inverse=False):
    """x: [samples, tokens, heads, head]; positions: [samples, tokens] ints;
    inv_freq: radians per position of every pair. Angles are reduced as exact
    rationals, so that far positions lose nothing."""
    out = np.array(x, dtype=np.float64)
    two_pi = 2 * Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    half = len(inv_freq)
    for b in range(x.shape[0]):
        for t in range(x.shape[1]):
            for i, f in enumerate(inv_freq):
                angle = float((int(positions[b, t]) * Fraction(float(f))) % two_pi)
                c, s = amplitude * math.cos(angle), amplitude * math.sin(angle) * (-1.0 if inverse else 1.0)
                p, q = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
                u, v = x[b, t, :, p], x[b, t, :, q]
                out[b, t, :, p] = u * c - v * s
                out[b, t, :, q] = v * c + u * s
    return out


# ---------------------------------------------------------------- dropout
def philox(counter, key):
    """The four words of one block: ten rounds, counter of 64 bits (the upper
    64 zero), key of 64 bits."""
    low = 0xFFFFFFFF
    c = [counter & low, counter >> 32 & low, 0, 0]
    k = [key & low, key >> 32 & low]
    for _ in range(10):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [q >> 32 ^ c[1] ^ k[0], q & low, p >> 32 ^ c[3] ^ k[1], p & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return c


def kept(n, p, seed, offset=0):
    """Which of n elements dropout keeps."""
    words = [w for i in range((n + 3) // 4) for w in philox((offset + i) % 2 ** 64, seed % 2 ** 64)]
    limit = int(math.floor(p * 2 ** 32 + 0.5))
    return np.array([w >= limit for w in words[:n]], dtype=bool)


def dropout(x, p, seed, offset=0, residual=None):
    keep = kept(x.size, p, seed, offset).reshape(x.shape)
    y = np.where(keep, x / (1.0 - p) if p < 1.0 else 0.0, 0.0)
    return y if residual is None else y + residual


# -------------------------------------------------------- cross attention
def _shared(t, heads):
    """[keys, kv_heads, head] with every key head repeated for its query heads."""
    return np.repeat(t, heads // t.shape[1], axis=1)


def attention_probabilities(q, k, scale):
    """P [heads, queries, keys] of one sequence, k cut to its keys."""
    s = np.einsum("qhd,khd->hqk", q, _shared(k, q.shape[1])) * scale
    p = np.exp(s - s.max(-1, keepdims=True))
    return p / p.sum(-1, keepdims=True)


def cross_attention(q, k, v, lengths, scale):
    """q: [batch, queries, heads, head]; k, v: [batch, keys, kv_heads, head];
    lengths: keys of each sequence."""
    o = np.zeros(q.shape)
    for b, n in enumerate(lengths):
        if n > 0:
            p = attention_probabilities(q[b], k[b, :n], scale)
            o[b] = np.einsum("hqk,khd->qhd", p, _shared(v[b, :n], q.shape[2]))
    return o


def cross_attention_backward(do, q, k, v, lengths, scale):
    """(dq, dk, dv)."""
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    heads, kv_heads = q.shape[2], k.shape[2]
    for b, n in enumerate(lengths):
        if n <= 0:
            continue
        p = attention_probabilities(q[b], k[b, :n], scale)
        dp = np.einsum("qhd,khd->hqk", do[b], _shared(v[b, :n], heads))
        ds = p * (dp - (p * dp).sum(-1, keepdims=True)) * scale
        dq[b] = np.einsum("hqk,khd->qhd", ds, _shared(k[b, :n], heads))
        for out, w, t in ((dk, ds, q[b]), (dv, p, do[b])):
            g = np.einsum("hqk,qhd->khd", w, t)
            out[b, :n] = g.reshape(n, kv_heads, heads // kv_heads, -1).sum(2)
    return dq, dk, dv


# ------------------------------------------------------------ linear layer
def linear(x, w, bias, act, residual):
    g = x @ w.T + (0.0 if bias is None else bias)
    a = g if act is None else activation(g, act)[0]
    return a if residual is None else residual + a


def linear_backward(dy, x, w, bias, act):
    """(dx, dw, dbias)."""
    g = x @ w.T + (0.0 if bias is None else bias)
    dg = dy if act is None else dy * activation(g, act)[1]
    return dg @ w, dg.T @ x, dg.sum(0)
