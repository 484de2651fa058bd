"""The operators of a transformer block's attention half as cases to time: the
projection with bias, activation and residual, the attention of tokens to an
encoder's states, the rotary positions and the dropout, forward and backward.

Every case has a plain form (elementary torch operations in 32 bits, rounded
once at the end) and the framework's own call; `own` picks which one `run`
takes. `exact` computes the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

_DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
_LARGEST_FLOPS = 6 * 4096 * 5120 * 15360
_LARGEST_BYTES = 2_000_000_000
_MASK32 = 0xFFFFFFFF


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token through the qkv projection of the d = 2048 model: a sampling step, bound by the weights
        {"name": "linear_one_token", "op": "linear", "T": 1, "k": 2048, "n": 6144, "bias": True, "act": "none",
         "residual": "none", "dtype": "bf16"},
        # the down projection of a ragged evaluation batch, added to an fp32 residual stream
        {"name": "linear_residual_ragged", "op": "linear", "T": 777, "k": 8192, "n": 2048, "bias": True,
         "act": "none", "residual": "fp32", "dtype": "bf16"},
        # the up projection with its activation in one training micro-batch, forward and backward
        {"name": "linear_train_act", "op": "linear_train", "T": 4096, "k": 2048, "n": 8192, "bias": True,
         "act": "gelu_tanh", "residual": "none", "dtype": "bf16"},
        # the qkv projection of the d = 5120 model, forward and backward: the largest
        {"name": "linear_train_wide", "op": "linear_train", "T": 4096, "k": 5120, "n": 15360, "bias": True,
         "act": "none", "residual": "none", "dtype": "bf16"},
        # one new token per sequence against the kept keys and values of long encoder states, shared heads
        {"name": "attention_one_token", "op": "attn", "B": 16, "Lq": 1, "Lk": 4096, "H": 16, "Hkv": 4, "D": 128,
         "ragged": True, "dtype": "bf16"},
        # image tokens to ragged captions, forward
        {"name": "attention_captions", "op": "attn", "B": 16, "Lq": 1024, "Lk": 250, "H": 16, "Hkv": 16, "D": 128,
         "ragged": True, "dtype": "bf16"},
        # the same in training, with heads of 72 elements and captions that were dropped (no keys at all)
        {"name": "attention_train_captions", "op": "attn_train", "B": 32, "Lq": 1024, "Lk": 120, "H": 16, "Hkv": 16,
         "D": 72, "ragged": True, "dtype": "bf16"},
        # long image tokens to long states, forward and backward
        {"name": "attention_train_long", "op": "attn_train", "B": 2, "Lq": 4096, "Lk": 4096, "H": 16, "Hkv": 16,
         "D": 128, "ragged": False, "dtype": "bf16"},
        # a token's queries of every sequence of a batch, part of the head: latency counts
        {"name": "rotary_few_tokens", "op": "rotary", "B": 16, "L": 1, "H": 20, "D": 128, "dim": 64,
         "layout": "interleaved", "scaling": "ramp", "far": 100000, "dtype": "bf16"},
        # queries and keys of a micro-batch and the way back of their gradients
        {"name": "rotary_train", "op": "rotary_train", "B": 4, "L": 4096, "H": 32, "D": 128, "dim": 128,
         "layout": "half", "scaling": "none", "far": 0, "dtype": "bf16"},
        # the residual branch of a small batch: latency counts
        {"name": "dropout_small", "op": "dropout", "T": 77, "d": 256, "p": 0.1, "residual": True, "dtype": "fp32"},
        # a micro-batch joined into the residual stream, and its gradient
        {"name": "dropout_train", "op": "dropout_train", "T": 32768, "d": 2048, "p": 0.1, "residual": True,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear_train", "attn", "attn_train", "attn_train", "rotary", "rotary_train", "dropout",
                     "dropout_train"])
    while True:
        if op in ("linear", "linear_train"):
            c = {"op": op, "T": _log(rng, 1, 8192), "k": 8 * _log(rng, 4, 1024), "n": 8 * _log(rng, 4, 1920),
                 "bias": rng.random() < 0.7, "act": rng.choice(["none", "none", "silu", "gelu", "gelu_tanh"]),
                 "residual": rng.choice(["none", "none", "same", "fp32"]),
                 "dtype": rng.choice(["bf16", "bf16", "fp16"])}
        elif op in ("attn", "attn_train"):
            H = rng.choice([1, 2, 4, 8, 12, 16, 24, 32])
            few = op == "attn" and rng.random() < 0.4
            c = {"op": op, "B": _log(rng, 1, 32), "Lq": rng.choice([1, 1, 2, 4]) if few else _log(rng, 5, 4096),
                 "Lk": _log(rng, 1, 16384 if few else 4096), "H": H,
                 "Hkv": rng.choice([h for h in range(1, H + 1) if H % h == 0]),
                 "D": rng.choice([32, 40, 64, 64, 72, 80, 96, 128, 128]), "ragged": rng.random() < 0.6,
                 "dtype": rng.choice(["bf16", "bf16", "fp16"])}
        elif op in ("rotary", "rotary_train"):
            D = 8 * rng.randint(2, 16)
            c = {"op": op, "B": _log(rng, 1, 32), "L": _log(rng, 1, 16384), "H": _log(rng, 1, 48), "D": D,
                 "dim": D if rng.random() < 0.6 else 2 * rng.randint(1, D // 2),
                 "layout": rng.choice(["half", "interleaved"]),
                 "scaling": rng.choice(["none", "linear", "base", "ramp"]), "far": rng.choice([0, 1000, 500000]),
                 "dtype": rng.choice(["bf16", "fp16", "fp32"])}
        else:
            c = {"op": op, "T": _log(rng, 1, 65536), "d": _log(rng, 8, 8192), "p": rng.choice([0.05, 0.1, 0.1, 0.5]),
                 "residual": rng.random() < 0.6, "dtype": rng.choice(["bf16", "fp16", "fp32"])}
        w = work(c)
        scores = c["B"] * c["H"] * c["Lq"] * c["Lk"] if "Lq" in c else 0
        if w["flops"] <= _LARGEST_FLOPS and w["bytes"] <= _LARGEST_BYTES and scores <= 1 << 29:
            return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    op, dt = c["op"], _DTYPES[c["dtype"]]
    # fp16 trains with a scaled loss, so that its gradients stay clear of the type's lowest values
    grad_scale = 1.0 if c["dtype"] == "fp16" else 1e-2
    if op in ("linear", "linear_train"):
        T, k, n = c["T"], c["k"], c["n"]
        # rows of a normalised stream with uneven channels; a weight that keeps their size
        c["x"] = (_randn(g, T, k) * torch.exp(0.5 * _randn(g, 1, k))).to(dt)
        c["w"] = (_randn(g, n, k) * k ** -0.5).to(dt)
        c["b"] = 0.1 * _randn(g, n) if c["bias"] else None
        rt = {"none": None, "same": dt, "fp32": torch.float32}[c["residual"]]
        c["res"] = None if rt is None else _randn(g, T, n).to(rt)
        if op == "linear_train":
            c["dy"] = (_randn(g, T, n) * grad_scale).to(dt if rt is None else rt)
    elif op in ("attn", "attn_train"):
        B, Lq, Lk, H, Hkv, D = (c[v] for v in ("B", "Lq", "Lk", "H", "Hkv", "D"))
        # queries as a projection leaves them; keys and values side by side, as one projection of the states does
        c["q"] = (1.3 * _randn(g, B, Lq, H, D)).to(dt)
        kv = _randn(g, B, Lk, 2, Hkv, D)
        kv[:, :, 0] += 0.5 * _randn(g, 1, 1, Hkv, D)
        kv = kv.to(dt)
        c["k"], c["v"] = kv[:, :, 0], kv[:, :, 1]
        c["lengths"] = None
        if c["ragged"]:
            n = torch.randint(1, Lk + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            if op == "attn_train":  # some captions are dropped
                n *= (torch.rand(B, generator=g, device="cuda") > 0.1).int()
            c["lengths"] = n
        if op == "attn_train":
            c["do"] = (_randn(g, B, Lq, H, D) * grad_scale).to(dt)
    elif op in ("rotary", "rotary_train"):
        B, L, H, D = c["B"], c["L"], c["H"], c["D"]
        c["x"] = _randn(g, B, L, H, D).to(dt)
        first = torch.randint(0, c["far"] + 1, (B, 1), generator=g, device="cuda")
        c["positions"] = first + torch.arange(L, device="cuda")
        if op == "rotary_train":
            c["dy"] = (_randn(g, B, L, H, D) * grad_scale).to(dt)
        c["inv_freq"] = torch.tensor(_frequencies(c["dim"], c["scaling"]), dtype=torch.float64, device="cuda")
        c["plan"] = _plan(c) if own else None
    else:
        T, d = c["T"], c["d"]
        c["x"] = _randn(g, T, d).to(dt)
        c["res"] = (2.0 * _randn(g, T, d)).to(dt) if c["residual"] else None
        c["dy"] = (_randn(g, T, d) * grad_scale).to(dt) if op == "dropout_train" else None
        c["key"] = int(torch.randint(0, 1 << 62, (1,), generator=torch.Generator().manual_seed(seed)))
        c["offset"] = 1 << 33  # some steps into the run
    return c


# the numbers of a run that extends a context four times
_BASE, _FACTOR, _TRAINED, _FAST, _SLOW = 10000.0, 4.0, 8192, 32.0, 1.0


def _frequencies(dim, scaling):
    """Radians per position of every pair, and how long contexts change them."""
    if scaling == "base":
        base = _BASE * _FACTOR ** (dim / max(dim - 2, 1))
    else:
        base = _BASE
    out = []
    for i in range(dim // 2):
        f = base ** (-2.0 * i / dim)
        if scaling == "linear":
            f /= _FACTOR
        elif scaling == "ramp":
            # pairs that turn more than _FAST times over the trained length stay, those below _SLOW are stretched
            keep = min(max((_TRAINED * f / (2.0 * math.pi) - _SLOW) / (_FAST - _SLOW), 0.0), 1.0)
            f = f * keep + f / _FACTOR * (1.0 - keep)
        out.append(f)
    return out


def _amplitude(scaling):
    return 0.1 * math.log(_FACTOR) + 1.0 if scaling == "ramp" else 1.0


def _plan(c):
    import matrix_aware_optimizer_gb300 as prm
    return prm.rotary_plan(c["dim"], base=_BASE, layout=c["layout"], scaling=c["scaling"], factor=_FACTOR,
                           trained_length=_TRAINED, fast=_FAST, slow=_SLOW, device="cuda")


# --------------------------------------------------------------------- run
def run(s):
    return _own_run(s) if own else _plain_run(s)


def _own_run(s):
    import matrix_aware_optimizer_gb300 as prm
    op = s["op"]
    if op in ("linear", "linear_train"):
        act = None if s["act"] == "none" else s["act"]
        if op == "linear":
            return prm.linear(s["x"], s["w"], s["b"], act=act, residual=s["res"])
        y, saved = prm.linear(s["x"], s["w"], s["b"], act=act, residual=s["res"], save=True)
        return (y,) + tuple(prm.linear_backward(s["dy"], s["x"], s["w"], saved, act=act, need_dbias=s["bias"]))
    if op == "attn":
        return prm.cross_attention(s["q"], s["k"], s["v"], key_lengths=s["lengths"])
    if op == "attn_train":
        o, saved = prm.cross_attention(s["q"], s["k"], s["v"], key_lengths=s["lengths"], save=True)
        return (o,) + tuple(prm.cross_attention_backward(s["do"], s["q"], s["k"], s["v"], o, saved,
                                                         key_lengths=s["lengths"]))
    if op in ("rotary", "rotary_train"):
        plan = s["plan"] if s["plan"] is not None else _plan(s)
        y = prm.rotary(s["x"], s["positions"], plan)
        return y if op == "rotary" else (y, prm.rotary_backward(s["dy"], s["positions"], plan))
    y = prm.dropout(s["x"], s["p"], s["key"], offset=s["offset"], residual=s["res"])
    return y if op == "dropout" else (y, prm.dropout_backward(s["dy"], s["p"], s["key"], offset=s["offset"]))


def _plain_run(s):
    op = s["op"]
    if op in ("linear", "linear_train"):
        return _plain_linear(s)
    if op in ("attn", "attn_train"):
        return _plain_attention(s)
    if op == "rotary":
        return _plain_rotary(s, s["x"], 1.0)
    if op == "rotary_train":
        return _plain_rotary(s, s["x"], 1.0), _plain_rotary(s, s["dy"], -1.0)
    keep = _keep(s)
    y = s["x"].float() * keep
    y = (y if s["res"] is None else s["res"].float() + y).to(s["x"].dtype)
    return y if op == "dropout" else (y, (s["dy"].float() * keep).to(s["dy"].dtype))


def _act(g, act):
    """Activation and its derivative."""
    if act == "none":
        return g, torch.ones_like(g)
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    if act == "gelu":
        p = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def _plain_linear(s):
    x, w = s["x"].float(), s["w"].float()
    g = x @ w.T
    if s["b"] is not None:
        g = g + s["b"]
    a, da = _act(g, s["act"])
    y = a if s["res"] is None else s["res"].float() + a
    y = y.to(s["x"].dtype if s["res"] is None else s["res"].dtype)
    if s["op"] == "linear":
        return y
    dg = s["dy"].float() * da
    return (y, (dg @ w).to(s["x"].dtype), (dg.T @ x).to(s["w"].dtype), dg.sum(0) if s["bias"] else None)


def _heads(t, H):
    """[B, L, heads, D] in 32 bits as [B, H, L, D], shared heads repeated."""
    t = t.float().transpose(1, 2)
    return t if t.shape[1] == H else t.repeat_interleave(H // t.shape[1], dim=1)


def _plain_attention(s):
    H, Hkv, D, Lk, dt = s["H"], s["Hkv"], s["D"], s["Lk"], s["q"].dtype
    q, k, v = _heads(s["q"], H), _heads(s["k"], H), _heads(s["v"], H)
    scale = D ** -0.5
    p = (q @ k.transpose(2, 3)) * scale
    if s["lengths"] is not None:
        hidden = torch.arange(Lk, device=p.device) >= s["lengths"][:, None, None, None]
        p = p.masked_fill(hidden, -math.inf)
        top = p.amax(-1, keepdim=True)
        p = torch.exp(p - torch.where(top == -math.inf, torch.zeros_like(top), top))
        total = p.sum(-1, keepdim=True)
        p = p / torch.where(total == 0, torch.ones_like(total), total)  # no keys: no output
    else:
        p = torch.exp(p - p.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    o = p @ v
    out = o.transpose(1, 2).to(dt)
    if s["op"] == "attn":
        return out
    do = _heads(s["do"], H)
    dv = p.transpose(2, 3) @ do
    dp = do @ v.transpose(2, 3)
    ds = p * (dp - (do * o).sum(-1, keepdim=True)) * scale
    del dp, p
    dq, dk = ds @ k, ds.transpose(2, 3) @ q

    def shared(t):
        return t.unflatten(1, (Hkv, H // Hkv)).sum(2).transpose(1, 2).to(dt)

    return out, dq.transpose(1, 2).to(dt), shared(dk), shared(dv)


def _plain_rotary(s, x, sign):
    dim = s["dim"]
    # far positions' angles need 64 bits
    angle = s["positions"].double()[..., None] * s["inv_freq"] * sign
    amp = _amplitude(s["scaling"])
    cos, sin = (torch.cos(angle) * amp).float()[:, :, None], (torch.sin(angle) * amp).float()[:, :, None]
    v = x.float()
    if s["layout"] == "half":
        a, b = v[..., :dim // 2], v[..., dim // 2:dim]
    else:
        a, b = v[..., 0:dim:2], v[..., 1:dim:2]
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([a, b], -1) if s["layout"] == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, v[..., dim:]], -1).to(x.dtype)


def _bits(n, key, offset, device):
    """n random 32-bit numbers: ten-round Philox 4x32 (Salmon and others, 2011)
    of the counters offset, offset + 1, ..., four numbers to a counter."""
    i = torch.arange((n + 3) // 4, device=device, dtype=torch.int64) + offset
    c = [i & _MASK32, i >> 32, torch.zeros_like(i), torch.zeros_like(i)]
    k0, k1 = key & _MASK32, key >> 32
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((q >> 32) & _MASK32) ^ c[1] ^ k0, q & _MASK32, ((p >> 32) & _MASK32) ^ c[3] ^ k1, p & _MASK32]
        k0, k1 = (k0 + 0x9E3779B9) & _MASK32, (k1 + 0xBB67AE85) & _MASK32
    return torch.stack(c, -1).flatten()[:n]


def _keep(s):
    """What each element is multiplied by: 0, or 1 / (1 - p)."""
    T, d, p = s["T"], s["d"], s["p"]
    kept = _bits(T * d, s["key"], s["offset"], s["x"].device) >= int(round(p * 2 ** 32))
    return kept.view(T, d).float() / (1.0 - p)


# -------------------------------------------------------------------- work
def work(case):
    c = case
    op, e = c["op"], _BYTES[c["dtype"]]
    if op in ("linear", "linear_train"):
        T, k, n = c["T"], c["k"], c["n"]
        out = 4 if c["residual"] == "fp32" else e
        res = 0 if c["residual"] == "none" else out
        b = 4 * n if c["bias"] else 0
        if op == "linear":
            return {"bytes": e * (T * k + n * k) + T * n * (out + res) + b, "flops": 2 * T * k * n}
        return {"bytes": e * 2 * (T * k + n * k) + T * n * (2 * out + res) + 2 * b, "flops": 6 * T * k * n}
    if op in ("attn", "attn_train"):
        B, Lq, Lk, H, Hkv, D = (c[v] for v in ("B", "Lq", "Lk", "H", "Hkv", "D"))
        # ragged lengths are spread evenly: half of the keys
        keys = Lk * (0.5 if c["ragged"] else 1.0)
        pairs = B * H * Lq * keys
        q, kv = e * B * Lq * H * D, e * 2 * B * Hkv * D
        if op == "attn":
            return {"bytes": 2 * q + kv * keys, "flops": 4 * pairs * D}
        return {"bytes": 4 * q + kv * (keys + Lk), "flops": 14 * pairs * D}
    if op in ("rotary", "rotary_train"):
        n = c["B"] * c["L"] * c["H"] * c["D"]
        passes = 1 if op == "rotary" else 2
        return {"bytes": passes * (2 * n * e + 8 * c["B"] * c["L"]), "flops": passes * 3 * n}
    n = c["T"] * c["d"]
    moved = (3 if c["residual"] else 2) + (2 if op == "dropout_train" else 0)
    return {"bytes": moved * n * e, "flops": (2 if op == "dropout" else 4) * n}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """The outputs from the definitions in 64 bits; the gradients by
    differentiating the forward definition, not from the formulas above."""
    s = prepare(case, seed)
    op, f64 = s["op"], torch.float64
    if op in ("linear", "linear_train"):
        if work(case)["flops"] > 2.5e12:
            return None
        grad = op == "linear_train"

        def leaf(t):
            return None if t is None else t.to(f64).requires_grad_(grad)

        x, w, b = leaf(s["x"]), leaf(s["w"]), leaf(s["b"])
        g = torch.nn.functional.linear(x, w, b)
        if s["act"] == "silu":
            g = torch.nn.functional.silu(g)
        elif s["act"] != "none":
            g = torch.nn.functional.gelu(g, approximate="tanh" if s["act"] == "gelu_tanh" else "none")
        y = g if s["res"] is None else g + s["res"].to(f64)
        if not grad:
            return y
        got = torch.autograd.grad(y, [t for t in (x, w, b) if t is not None], s["dy"].to(f64))
        return (y.detach(),) + got[:2] + (got[2] if b is not None else None,)
    if op in ("attn", "attn_train"):
        B, Lq, Lk, H, Hkv, D = (s[v] for v in ("B", "Lq", "Lk", "H", "Hkv", "D"))
        if work(case)["flops"] > 4e12 or B * H * Lq * Lk > 1 << 30:
            return None
        grad = op == "attn_train"
        out = torch.zeros(B, Lq, H, D, dtype=f64, device="cuda")
        grads = [torch.zeros(t.shape, dtype=f64, device="cuda") for t in (s["q"], s["k"], s["v"])]
        lengths = [Lk] * B if s["lengths"] is None else s["lengths"].tolist()
        for b, n in enumerate(lengths):  # one sequence at a time, cut to its keys
            if n == 0:
                continue
            q, k, v = (t.to(f64).requires_grad_(grad) for t in (s["q"][b], s["k"][b, :n], s["v"][b, :n]))
            by_group = q.reshape(Lq, Hkv, H // Hkv, D)
            scores = torch.einsum("qhgd,khd->hgqk", by_group, k) / math.sqrt(D)
            o = torch.einsum("hgqk,khd->qhgd", torch.softmax(scores, -1), v).reshape(Lq, H, D)
            out[b] = o.detach()
            if grad:
                for t, g, cut in zip(grads, torch.autograd.grad(o, (q, k, v), s["do"][b].to(f64)), (Lq, n, n)):
                    t[b, :cut] = g
        return (out,) + tuple(grads) if grad else out
    if op in ("rotary", "rotary_train"):
        # a pair as a complex number, turned by a unit one
        dim = s["dim"]
        f = torch.tensor(_frequencies(dim, s["scaling"]), dtype=f64, device="cuda")
        angle = (s["positions"].to(f64)[..., None] * f)[:, :, None]
        turn = torch.polar(torch.full_like(angle, _amplitude(s["scaling"])), angle)

        def turned(x, turn):
            v = x.to(f64)
            pairs = v[..., :dim].unflatten(-1, (2, dim // 2) if s["layout"] == "half" else (dim // 2, 2))
            at = -2 if s["layout"] == "half" else -1
            z = torch.complex(pairs.select(at, 0), pairs.select(at, 1)) * turn
            return torch.cat([torch.stack([z.real, z.imag], at).flatten(-2), v[..., dim:]], -1)

        y = turned(s["x"], turn)
        return y if op == "rotary" else (y, turned(s["dy"], turn.conj()))
    keep = (_bits(s["T"] * s["d"], s["key"], s["offset"], "cuda") >= round(s["p"] * 2 ** 32)).view(s["T"], s["d"])
    y = torch.where(keep, s["x"].to(f64) / (1 - s["p"]), 0.0)
    y = y if s["res"] is None else y + s["res"].to(f64)
    return y if op == "dropout" else (y, torch.where(keep, s["dy"].to(f64) / (1 - s["p"]), 0.0))
