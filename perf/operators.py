"""The transformer-block operators as cases to time: the gated feed-forward
block, the norms around a block with their gate and residual scale, and the
token embedding, each forward and backward.

Every case has a plain form (elementary torch operations in 32 bits, rounded
once at the end) and the framework's own call; `own` picks which one `run`
takes. `exact` computes the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

_DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
_EPS = 1e-6
_LARGEST_FLOPS = 18 * 4096 * 5120 * 20480
_LARGEST_BYTES = 1_400_000_000


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token through the feed-forward block of the d = 2048 model: a sampling step, bound by the weights
        {"name": "ffn_one_token", "op": "ffn", "T": 1, "d": 2048, "f": 8192, "act": "silu", "dtype": "bf16"},
        # a ragged evaluation batch, forward only
        {"name": "ffn_eval_ragged", "op": "ffn", "T": 777, "d": 2048, "f": 8192, "act": "gelu", "dtype": "bf16"},
        # the smallest training step: the tiny set's matrices, fp16 with a scaled loss; latency counts
        {"name": "ffn_train_tiny", "op": "ffn_train", "T": 201, "d": 64, "f": 256, "act": "silu", "dtype": "fp16"},
        # one training micro-batch of a d = 2048 block, forward and backward
        {"name": "ffn_train_block", "op": "ffn_train", "T": 8192, "d": 2048, "f": 8192, "act": "silu",
         "dtype": "bf16"},
        # the d = 5120 block, forward and backward: the largest
        {"name": "ffn_train_wide", "op": "ffn_train", "T": 4096, "d": 5120, "f": 20480, "act": "gelu_tanh",
         "dtype": "bf16"},
        # a few rows of a small model in fp32: latency counts
        {"name": "norm_small", "op": "norm", "B": 1, "L": 12, "d": 256, "kind": "rms", "post": True, "mod": False,
         "weight": True, "alpha": 0.5, "stream": "fp32", "block": "fp32"},
        # image tokens of a modulated d = 2048 block: layer norm, gate, scale and shift per sample
        {"name": "norm_modulated", "op": "norm", "B": 32, "L": 1024, "d": 2048, "kind": "layer", "post": False,
         "mod": True, "weight": False, "alpha": 1.0, "stream": "fp32", "block": "bf16"},
        {"name": "norm_modulated_grad", "op": "norm_grad", "B": 32, "L": 1024, "d": 2048, "kind": "layer",
         "post": False, "mod": True, "weight": False, "alpha": 1.0, "stream": "fp32", "block": "bf16"},
        # norms on both sides of a d = 5120 block with learned gains and a scaled residual, an odd row count
        {"name": "norm_both_sides_grad", "op": "norm_grad", "B": 1, "L": 8191, "d": 5120, "kind": "rms",
         "post": True, "mod": False, "weight": True, "alpha": 0.7071, "stream": "bf16", "block": "bf16"},
        # the token lookup of one micro-batch from the fp32 master table
        {"name": "embed_lookup", "op": "embed", "T": 8192, "V": 64000, "d": 2048, "scale": 45.25, "pad": 0.0,
         "table": "fp32", "out": "bf16"},
        # its gradient: the whole table is written, a few rows of it from long runs of frequent tokens
        {"name": "embed_grad", "op": "embed_grad", "T": 8192, "V": 64000, "d": 2048, "scale": 45.25, "pad": 0.0,
         "table": "bf16", "out": "bf16"},
        # a long padded batch over a table of odd sizes, fp32 gradient
        {"name": "embed_grad_long", "op": "embed_grad", "T": 65521, "V": 100003, "d": 1001, "scale": 1.0,
         "pad": 0.07, "table": "fp32", "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn_train", "norm", "norm_grad", "embed", "embed_grad"])
    while True:
        if op in ("ffn", "ffn_train"):
            d = 8 * _log(rng, 8, 640)
            c = {"op": op, "T": _log(rng, 1, 8192), "d": d, "f": 8 * max(8, int(d * rng.uniform(1.5, 4.0)) // 8),
                 "act": rng.choice(["silu", "gelu", "gelu_tanh"]), "dtype": rng.choice(["bf16", "bf16", "fp16"])}
        elif op in ("norm", "norm_grad"):
            stream, block = rng.choice([("fp32", "fp32"), ("fp32", "bf16"), ("fp32", "fp16"), ("bf16", "bf16"),
                                        ("fp16", "fp16")])
            d = _log(rng, 16, 8192)
            c = {"op": op, "B": _log(rng, 1, 64), "L": _log(rng, 1, 4096),
                 "d": d if rng.random() < 0.3 else max(16, d // 8 * 8),
                 "kind": rng.choice(["rms", "layer"]), "post": rng.random() < 0.5, "mod": rng.random() < 0.5,
                 "weight": rng.random() < 0.5, "alpha": rng.choice([1.0, 0.7071]), "stream": stream, "block": block}
        else:
            d = _log(rng, 16, 5120)
            c = {"op": op, "T": _log(rng, 1, 65536), "V": _log(rng, 100, 131072),
                 "d": d if rng.random() < 0.3 else max(16, d // 8 * 8),
                 "scale": rng.choice([1.0, round(math.sqrt(d), 3)]), "pad": rng.choice([0.0, 0.1]),
                 "table": rng.choice(["fp32", "bf16"]), "out": rng.choice(["fp32", "bf16", "bf16"])}
        w = work(c)
        if w["flops"] <= _LARGEST_FLOPS and w["bytes"] <= _LARGEST_BYTES and _held(c) <= 1.2e9:
            return c


def _held(c):
    """Elements of the largest tensors a case holds at once (a bound on memory, not on work)."""
    if c["op"] in ("ffn", "ffn_train"):
        return 3 * c["d"] * c["f"] + 8 * c["T"] * (c["d"] + c["f"])
    if c["op"] in ("norm", "norm_grad"):
        return 6 * c["B"] * c["L"] * c["d"]
    return (c["T"] + c["V"]) * c["d"]


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
    if c["op"] in ("ffn", "ffn_train"):
        T, d, f, dt = c["T"], c["d"], c["f"], _DTYPES[c["dtype"]]
        # rows of a normalised residual stream with uneven channels; weights as the optimizer's matrices start
        c["x"] = (_randn(g, T, d) * torch.exp(0.5 * _randn(g, 1, d))).to(dt)
        c["wg"] = (_randn(g, f, d) * 0.02).to(dt)
        c["wu"] = (_randn(g, f, d) * 0.02).to(dt)
        c["wd"] = (_randn(g, d, f) * 0.02).to(dt)
        if c["op"] == "ffn_train":
            # fp16 trains with a scaled loss, so that its gradients stay clear of the type's lowest values
            c["dy"] = (_randn(g, T, d) * (1.0 if c["dtype"] == "fp16" else 1e-3)).to(dt)
    elif c["op"] in ("norm", "norm_grad"):
        B, L, d, rt, bt = c["B"], c["L"], c["d"], _DTYPES[c["stream"]], _DTYPES[c["block"]]
        ch = torch.exp(0.7 * _randn(g, 1, 1, d))
        c["x"] = (_randn(g, B, L, d) * ch + 0.2 * _randn(g, 1, 1, d)).to(rt)
        c["z"] = (_randn(g, B, L, d) * 0.6 + 0.1 * _randn(g, 1, 1, d)).to(bt)
        c["post_weight"] = 1.0 + 0.1 * _randn(g, d) if c["post"] else None
        c["pre_weight"] = 1.0 + 0.1 * _randn(g, d) if c["weight"] else None
        # the modulation layer's output: gate, scale and shift side by side, one row per sample
        m = (_randn(g, B, 3 * d) * 0.3).to(bt) if c["mod"] else None
        c["gate"], c["scale"], c["shift"] = m.chunk(3, dim=1) if c["mod"] else (None, None, None)
        if c["op"] == "norm_grad":
            # what the forward pass left behind: r (in x's place), z and the row statistics
            c["dy"] = (_randn(g, B, L, d) * 1e-2).to(bt)
            c["dr"] = (_randn(g, B, L, d) * 1e-2).to(rt)
            c["r"] = c.pop("x")
            mr, sr = _stats(c["r"].float(), c["kind"])
            mz, sz = _stats(c["z"].float(), c["kind"])
            c["stats"] = torch.cat([mr, sr, mz, sz], dim=-1).reshape(B * L, 4).contiguous()
    else:
        T, V, d = c["T"], c["V"], c["d"]
        # token ranks fall off as in text: a few tokens make up much of a batch
        u = torch.rand(T, generator=g, device="cuda")
        rank = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
        tok = torch.randperm(V, generator=g, device="cuda")[rank]
        if c["pad"] > 0:
            tok[T - int(c["pad"] * T):] = -1
        c["tokens"] = tok
        if c["op"] == "embed":
            c["weight"] = (_randn(g, V, d) * 0.02).to(_DTYPES[c["table"]])
        else:
            c["dout"] = (_randn(g, T, d) * 1e-2).to(_DTYPES[c["out"]])
    return c


def _stats(v, kind):
    """Mean (0 for the rms kind) and reciprocal deviation of every row."""
    m = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[..., :1])
    return m, torch.rsqrt((v - m).square().mean(-1, keepdim=True) + _EPS)


# --------------------------------------------------------------------- run
def run(s):
    return _own_run(s) if own else _plain_run(s)


def _own_run(s):
    import matrix_aware_optimizer_gb300 as prm
    op = s["op"]
    if op == "ffn":
        return prm.gated_ffn(s["x"], s["wg"], s["wu"], s["wd"], act=s["act"])
    if op == "ffn_train":
        y, saved = prm.gated_ffn(s["x"], s["wg"], s["wu"], s["wd"], act=s["act"], save=True)
        return (y,) + tuple(prm.gated_ffn_backward(s["dy"], s["x"], s["wg"], s["wu"], s["wd"], saved, act=s["act"]))
    if op == "norm":
        r, y, _ = prm.block_norm(s["x"], s["z"], kind=s["kind"], alpha=s["alpha"], post_weight=s["post_weight"],
                                 gate=s["gate"], pre_weight=s["pre_weight"], scale=s["scale"], shift=s["shift"],
                                 eps=_EPS)
        return r, y
    if op == "norm_grad":
        return tuple(prm.block_norm_backward(
            s["dy"], s["dr"], s["r"], s["z"], s["stats"], kind=s["kind"], alpha=s["alpha"],
            post_weight=s["post_weight"], gate=s["gate"], pre_weight=s["pre_weight"], scale=s["scale"],
            shift=s["shift"]))
    if op == "embed":
        return prm.embedding(s["tokens"], s["weight"], scale=s["scale"], dtype=_DTYPES[s["out"]])
    return prm.embedding_backward(s["dout"], s["tokens"], s["V"], scale=s["scale"], dtype=_DTYPES[s["table"]])


def _plain_run(s):
    op = s["op"]
    if op == "ffn":
        return _plain_ffn(s)[0].to(s["x"].dtype)
    if op == "ffn_train":
        return _plain_ffn_train(s)
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_grad":
        return _plain_norm_grad(s)
    if op == "embed":
        tok, w = s["tokens"], s["weight"]
        valid = (tok >= 0) & (tok < w.shape[0])
        rows = w[tok.clamp(0, w.shape[0] - 1)].float() * s["scale"]
        return torch.where(valid[:, None], rows, torch.zeros_like(rows)).to(_DTYPES[s["out"]])
    tok, V = s["tokens"], s["V"]
    valid = (tok >= 0) & (tok < V)
    rows = torch.where(valid, tok, torch.full_like(tok, V))  # padding is summed into a row that is cut off
    dw = torch.zeros(V + 1, s["dout"].shape[1], device=tok.device)
    dw.index_add_(0, rows, s["dout"].float())
    return (dw[:V] * s["scale"]).to(_DTYPES[s["table"]])


def _act(g, act):
    """Activation and its derivative."""
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    if act == "gelu":
        p = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def _plain_ffn(s):
    x = s["x"].float()
    g, u = x @ s["wg"].float().T, x @ s["wu"].float().T
    a, da = _act(g, s["act"])
    h = a * u
    return h @ s["wd"].float().T, x, u, a, da, h


def _plain_ffn_train(s):
    dt = s["x"].dtype
    y, x, u, a, da, h = _plain_ffn(s)
    dy = s["dy"].float()
    dh = dy @ s["wd"].float()
    dg, du = dh * u * da, dh * a
    dx = dg @ s["wg"].float() + du @ s["wu"].float()
    return y.to(dt), dx.to(dt), (dg.T @ x).to(dt), (du.T @ x).to(dt), (dy.T @ h).to(dt)


def _per_sample(v):
    return v.float()[:, None, :]


def _plain_norm(s):
    z = s["z"].float()
    if s["post_weight"] is not None:
        m, rs = _stats(z, s["kind"])
        z = (z - m) * rs * s["post_weight"]
    if s["gate"] is not None:
        z = z * _per_sample(s["gate"])
    r = (s["alpha"] * s["x"].float() + z).to(s["x"].dtype)
    # the next norm reads the residual stream as it is stored
    m, rs = _stats(r.float(), s["kind"])
    y = (r.float() - m) * rs
    if s["pre_weight"] is not None:
        y = y * s["pre_weight"]
    if s["scale"] is not None:
        y = y * (1.0 + _per_sample(s["scale"])) + _per_sample(s["shift"])
    return r, y.to(s["z"].dtype)


def _norm_grad(dn, n, rs, kind):
    """Gradient of v -> n = (v - mean) rs from the gradient dn of n."""
    d = dn - n * (dn * n).mean(-1, keepdim=True)
    return rs * (d - dn.mean(-1, keepdim=True) if kind == "layer" else d)


def _plain_norm_grad(s):
    bt, rt, kind = s["z"].dtype, s["r"].dtype, s["kind"]
    dy, r, z = s["dy"].float(), s["r"].float(), s["z"].float()
    st = s["stats"].reshape(*r.shape[:2], 4)
    mr, sr, mz, sz = st[..., 0:1], st[..., 1:2], st[..., 2:3], st[..., 3:4]
    n = (r - mr) * sr
    dn, dpre, dscale, dshift = dy, None, None, None
    if s["scale"] is not None:
        dshift = dy.sum(1).to(bt)
        dscale = (dy * n if s["pre_weight"] is None else dy * n * s["pre_weight"]).sum(1).to(bt)
        dn = dy * (1.0 + _per_sample(s["scale"]))
    if s["pre_weight"] is not None:
        dpre = (dn * n).sum((0, 1))
        dn = dn * s["pre_weight"]
    dr = s["dr"].float() + _norm_grad(dn, n, sr, kind)
    dx = (s["alpha"] * dr).to(rt)
    p, zn = z, None
    if s["post_weight"] is not None:
        zn = (z - mz) * sz
        p = zn * s["post_weight"]
    dgate, dp, dpost = None, dr, None
    if s["gate"] is not None:
        dgate = (dr * p).sum(1).to(bt)
        dp = dr * _per_sample(s["gate"])
    if s["post_weight"] is not None:
        dpost = (dp * zn).sum((0, 1))
        dp = _norm_grad(dp * s["post_weight"], zn, sz, kind)
    return dx, dp.to(bt), dpost, dgate, dpre, dscale, dshift


# -------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] in ("ffn", "ffn_train"):
        T, d, f = c["T"], c["d"], c["f"]
        if c["op"] == "ffn":
            return {"bytes": 2 * (2 * T * d + 3 * d * f), "flops": 6 * T * d * f}
        return {"bytes": 2 * (4 * T * d + 6 * d * f), "flops": 18 * T * d * f}
    if c["op"] in ("norm", "norm_grad"):
        n, d = c["B"] * c["L"], c["d"]
        rs, bs = _BYTES[c["stream"]], _BYTES[c["block"]]
        mod = 3 * c["B"] * d * bs if c["mod"] else 0
        vec = 4 * d * (int(c["post"]) + int(c["weight"]))
        if c["op"] == "norm":
            return {"bytes": n * d * (2 * rs + 2 * bs) + mod + vec, "flops": 12 * n * d}
        return {"bytes": n * d * (3 * rs + 3 * bs) + 16 * n + 2 * mod + 2 * vec, "flops": 25 * n * d}
    T, V, d = c["T"], c["V"], c["d"]
    if c["op"] == "embed":
        # a row that is looked up again need not be read again: the expected number of different tokens
        k = torch.arange(V, dtype=torch.float64)
        p = torch.log((k + 2) / (k + 1)) / math.log(V + 1.0)
        rows = float((1 - (1 - p) ** (T - int(c["pad"] * T))).sum())
        return {"bytes": 8 * T + rows * d * _BYTES[c["table"]] + T * d * _BYTES[c["out"]], "flops": T * d}
    return {"bytes": 8 * T + T * d * _BYTES[c["out"]] + V * d * _BYTES[c["table"]], "flops": 2 * T * d}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """The outputs from the definitions in 64 bits; the gradients by
    differentiating the forward definition, not from the formulas above."""
    s = prepare(case, seed)
    op, f64 = s["op"], torch.float64
    if op in ("ffn", "ffn_train"):
        if work(case)["flops"] > 1e13:
            return None
        grad = op == "ffn_train"
        x, wg, wu, wd = (s[k].to(f64).requires_grad_(grad) for k in ("x", "wg", "wu", "wd"))
        g = torch.nn.functional.linear(x, wg)
        if s["act"] == "silu":
            a = torch.nn.functional.silu(g)
        else:
            a = torch.nn.functional.gelu(g, approximate="tanh" if s["act"] == "gelu_tanh" else "none")
        y = torch.nn.functional.linear(a * torch.nn.functional.linear(x, wu), wd)
        if not grad:
            return y
        return (y.detach(),) + torch.autograd.grad(y, (x, wg, wu, wd), s["dy"].to(f64))
    if op in ("norm", "norm_grad"):
        grad = op == "norm_grad"

        def leaf(k):
            return None if s[k] is None else s[k].to(f64).requires_grad_(grad)

        z, wpost, gate, wpre, scale, shift = (leaf(k) for k in ("z", "post_weight", "gate", "pre_weight", "scale",
                                                               "shift"))

        def norm(v):
            c = v - v.mean(-1, keepdim=True) if s["kind"] == "layer" else v
            return c / torch.sqrt((c * c).mean(-1, keepdim=True) + _EPS)

        b = z if wpost is None else norm(z) * wpost
        b = b if gate is None else gate.unsqueeze(1) * b

        def after(r):
            y = norm(r) if wpre is None else norm(r) * wpre
            return y if scale is None else y * (1 + scale.unsqueeze(1)) + shift.unsqueeze(1)

        if not grad:
            r = (s["alpha"] * s["x"].to(f64) + b).to(s["x"].dtype)
            return r, after(r.to(f64))
        # r as stored is where the graph splits: its gradient goes on to x and to the block's output
        r = s["r"].to(f64).requires_grad_()
        y = after(r)
        want = [v for v in (wpre, scale, shift) if v is not None]
        got = list(torch.autograd.grad(y, [r] + want, s["dy"].to(f64)))
        total = got.pop(0) + s["dr"].to(f64)
        after_grads = [None if v is None else got.pop(0) for v in (wpre, scale, shift)]
        want = [v for v in (z, wpost, gate) if v is not None]
        got = list(torch.autograd.grad(b, want, total))
        before = [None if v is None else got.pop(0) for v in (z, wpost, gate)]
        return tuple([s["alpha"] * total] + before + after_grads)
    tok = s["tokens"]
    if op == "embed":
        w = torch.cat([s["weight"].to(f64), torch.zeros(1, s["d"], dtype=f64, device=tok.device)])
        return w[torch.where(tok < 0, torch.full_like(tok, s["V"]), tok)] * s["scale"]
    kept = tok >= 0
    order = torch.argsort(tok[kept], stable=True)
    ids, counts = torch.unique_consecutive(tok[kept][order], return_counts=True)
    total = torch.zeros(order.numel() + 1, s["d"], dtype=f64, device=tok.device)
    torch.cumsum(s["dout"].to(f64)[kept][order], 0, out=total[1:])
    ends = counts.cumsum(0)
    dw = torch.zeros(s["V"], s["d"], dtype=f64, device=tok.device)
    dw[ids] = (total[ends] - total[ends - counts]) * s["scale"]
    return dw
