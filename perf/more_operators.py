"""Timed cases of the operators between a Transformer's linear layers and of its
loss: the norms around a block with its gate and residual scale, dropout from a
counter-based generator, cross attention to an encoder's states, and log
probabilities with entropy, top alternatives and gradient.

`run` computes an operator in elementary torch operations in binary32, or,
with `own` set, through ring_all_reduce_amd.api.  `exact` gives the same
outputs from the definitions in binary64.

Shapes: T tokens of D features; B sequences of Tq queries and Tk keys, H query
heads on Hkv key heads of dh features; V vocabulary entries.  The sizes come
from the Transformer whose gradient tensors the bucketed workload reduces
(d = 2048, h = 8192, V = 32000).
"""
import functools
import math

import numpy as np
import torch

own = False

EPS = 1e-5
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_M0, _M1 = 0xD2511F53, 0xCD9E8D57    # Philox4x32: multipliers and key increments
_W0, _W1 = 0x9E3779B9, 0xBB67AE85
_LOW = 0xFFFFFFFF


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the residual stream of one decoding step of a few requests, into the next block: latency
        dict(name="norm_step", op="norm", T=8, D=2048, dtype="f32", post="none", pre="layer"),
        # the same of one rank's batch, 32 sequences of 2048, with norms on both sides
        dict(name="norm_batch", op="norm", T=65536, D=2048, dtype="bf16", post="layer", pre="layer"),
        # the backward pass of a short ragged batch on an odd width
        dict(name="norm_grad_ragged", op="norm_grad", T=1027, D=1001, dtype="f32", post="rms", pre="rms"),
        # the backward pass of one rank's batch
        dict(name="norm_grad_batch", op="norm_grad", T=65536, D=2048, dtype="bf16", post="layer", pre="layer"),
        # a short ragged batch
        dict(name="dropout_ragged", op="dropout", T=333, D=1001, dtype="f32", p=0.1, residual=False),
        # a block's output dropped out and added to one rank's residual stream
        dict(name="dropout_batch", op="dropout", T=65536, D=2048, dtype="bf16", p=0.1, residual=True),
        # one decoding step of 16 requests, each against its own source of up to 2048 states
        dict(name="attn_token", op="attn", B=16, Tq=1, Tk=2048, H=16, Hkv=16, dh=128, dtype="bf16"),
        # a training step on a few ragged pairs in binary32, heads of odd width shared by two
        dict(name="attn_grad_ragged", op="attn_grad", B=3, Tq=333, Tk=517, H=6, Hkv=3, dh=60, dtype="f32"),
        # a training step of one rank's micro-batch: forward and backward
        dict(name="attn_grad_batch", op="attn_grad", B=8, Tq=2048, Tk=1024, H=16, Hkv=16, dh=128, dtype="bf16"),
        # the tokens of one decoding step with eight alternatives each: latency
        dict(name="logprob_step", op="logprob", T=8, V=32000, dtype="f32", K=8),
        # log probabilities, entropy and alternatives of a batch that is scored
        dict(name="logprob_batch", op="logprob", T=8192, V=32000, dtype="bf16", K=8),
        # the loss and its gradient for one rank's micro-batch
        dict(name="logprob_grad_batch", op="logprob_grad", T=8192, V=32000, dtype="bf16"),
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]; half of them whole eights."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 16 and rng.random() < 0.5:
        n -= n % 8
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "dropout", "attn", "attn_grad", "attn_grad", "logprob", "logprob_grad"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("norm", "norm_grad"):
        return dict(op=op, T=_size(rng, 1, 16384), D=_size(rng, 64, 8192), dtype=dtype,
                    post=rng.choice(["none", "layer", "rms"]), pre=rng.choice(["layer", "rms"]))
    if op == "dropout":
        return dict(op=op, T=_size(rng, 1, 16384), D=_size(rng, 64, 8192), dtype=dtype, p=rng.choice([0.05, 0.1, 0.5]),
                    residual=rng.random() < 0.5)
    if op in ("attn", "attn_grad"):
        H = rng.choice([1, 2, 4, 6, 8, 12, 16])
        Hkv = rng.choice([h for h in (1, 2, 3, 4, 8, 16) if H % h == 0])
        B, dh = rng.choice([1, 2, 3, 5, 8]), _size(rng, 16, 128)
        # over a single key the gradients of q and k are zero, which says nothing
        Tk = _size(rng, 1 if op == "attn" else 8, 2048)
        # binary32 products run at a sixteenth of the bfloat16 rate
        Tq = 1 if op == "attn" and rng.random() < 0.5 else _size(rng, 2, 1024 if dtype == "bf16" else 256)
        return dict(op=op, B=B, Tq=Tq, Tk=Tk, H=H, Hkv=Hkv, dh=dh, dtype=dtype)
    V = _size(rng, 100, 64000)
    T = max(1, min(_size(rng, 1, 4096), 60_000_000 // V))
    if op == "logprob":
        return dict(op=op, T=T, V=V, dtype=dtype, K=rng.choice([1, 5, 20]))
    return dict(op=op, T=T, V=V, dtype=dtype)


def _lengths(n, most):
    """Lengths of the sequences of a padded batch: from `most` down to half of it."""
    return [most - (i * most) // (2 * n) for i in range(n)]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    """What the program has in hand: activations of unit scale, gradients of
    scale 1e-2, norm weights near one, logits with a few likely tokens, and
    sequences of different lengths in a padded batch."""
    dev = torch.device("cuda") if torch.cuda.is_available() else torch.device("cpu")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = _DT[case["dtype"]]
    op = case["op"]

    def normal(*shape, scale=1.0, shift=0.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale + shift).to(dt)

    s = dict(case)
    if op in ("norm", "norm_grad"):
        T, D = case["T"], case["D"]
        s["o"] = normal(T, D)
        s["gate"] = normal(D, scale=0.2, shift=0.5)
        s["a"], s["s"] = 1.0, 0.5
        for side in ("post", "pre"):
            s[side + "_w"] = normal(D, scale=0.1, shift=1.0) if case[side] != "none" else None
            s[side + "_b"] = normal(D, scale=0.1) if case[side] == "layer" else None
        if op == "norm":
            s["x"] = normal(T, D, scale=2.0)
        else:
            s["h"] = normal(T, D, scale=2.0, shift=0.1)
            s["dh"], s["du"] = normal(T, D, scale=1e-2), normal(T, D, scale=1e-2)
        return s
    if op == "dropout":
        T, D = case["T"], case["D"]
        s["x"] = normal(T, D)
        s["r"] = normal(T, D, scale=2.0) if case["residual"] else None
        s["seed"] = (int(seed) * 0x9E3779B97F4A7C15 + 12345) % (1 << 64)
        s["step"] = torch.randint(0, 1 << 40, (1,), generator=gen, device=dev)
        return s
    if op in ("attn", "attn_grad"):
        B, Tq, Tk, H, Hkv, dh = (case[k] for k in ("B", "Tq", "Tk", "H", "Hkv", "dh"))
        s["q"], s["k"], s["v"] = normal(B * Tq, H * dh), normal(B * Tk, Hkv * dh), normal(B * Tk, Hkv * dh)
        order = torch.randperm(B, generator=gen, device=dev)
        s["klen"] = torch.tensor(_lengths(B, Tk), device=dev)[order]
        s["qlen"] = torch.tensor(_lengths(B, Tq), device=dev) if op == "attn_grad" else None
        if op == "attn_grad":
            s["do"] = normal(B * Tq, H * dh, scale=1e-2)
        return s
    T, V = case["T"], case["V"]
    z = torch.randn(T, V, generator=gen, device=dev)
    s["targets"] = torch.randint(0, V, (T,), generator=gen, device=dev)
    # a trained model gives the token that follows, and some others, most of the weight
    for _ in range(4):
        z.scatter_add_(1, torch.randint(0, V, (T, 1), generator=gen, device=dev),
                       torch.rand(T, 1, generator=gen, device=dev) * 12)
    z.scatter_add_(1, s["targets"].unsqueeze(1), torch.rand(T, 1, generator=gen, device=dev) * 12)
    s["logits"] = z.to(dt)
    s["targets"][torch.rand(T, generator=gen, device=dev) < 0.01] = -1     # padding
    if op == "logprob_grad":
        s["dlogp"] = torch.full((T,), -1.0 / T, device=dev)
        s["dent"] = torch.full((T,), -0.01 / T, device=dev)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _centred(v, kind):
    """(v normalised, 1 / its scale)."""
    if kind == "none":
        return v, None
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * r, r


def _affine(v, w, b):
    v = v if w is None else v * w.float()
    return v if b is None else v + b.float()


def _norm_back(g, v, r, kind):
    """Gradient of the normalised v (its scale r) given g = dy w."""
    if kind == "none":
        return g
    d = g - v * (g * v).mean(1, keepdim=True)
    if kind == "layer":
        d = d - g.mean(1, keepdim=True)
    return d * r


def _plain_norm(s, dt):
    n = _affine(_centred(s["o"].float(), s["post"])[0], s["post_w"], s["post_b"])
    h = s["a"] * s["x"].float() + s["s"] * (s["gate"].float() * n)
    return h.to(dt), _affine(_centred(h, s["pre"])[0], s["pre_w"], s["pre_b"]).to(dt)


def _plain_norm_grad(s, dt):
    ho, ro = _centred(s["o"].float(), s["post"])
    hh, rh = _centred(s["h"].float(), s["pre"])
    du = s["du"].float()
    g = s["dh"].float() + _norm_back(_affine(du, s["pre_w"], None), hh, rh, s["pre"])
    sg = s["s"] * g
    dn = s["gate"].float() * sg
    out = {"dx": s["a"] * g, "do": _norm_back(_affine(dn, s["post_w"], None), ho, ro, s["post"]),
           "dgate": (sg * _affine(ho, s["post_w"], s["post_b"])).sum(0), "dpre_w": (du * hh).sum(0)}
    if s["post_w"] is not None:
        out["dpost_w"] = (dn * ho).sum(0)
    if s["post_b"] is not None:
        out["dpost_b"] = dn.sum(0)
    if s["pre_b"] is not None:
        out["dpre_b"] = du.sum(0)
    return {k: v.to(dt) for k, v in out.items()}


def _mul32(a, b):
    """High and low words of a * b for 32-bit numbers in int64."""
    t = a * (b & 0xFFFF)
    return (a * (b >> 16) + (t >> 16)) >> 16, (a * b) & _LOW


def _threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def _plain_dropout(s, dt):
    T, D, x = s["T"], s["D"], s["x"]
    G = (D + 7) // 8
    c0 = torch.arange(T * G, device=x.device)
    c1, c2 = torch.zeros_like(c0), (s["step"] & _LOW).expand_as(c0)
    c3 = ((s["step"] >> 32) & _LOW).expand_as(c0)
    k0, k1 = s["seed"] & _LOW, s["seed"] >> 32
    for _ in range(10):
        h0, l0 = _mul32(_M0, c0)
        h1, l1 = _mul32(_M1, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + _W0) & _LOW, (k1 + _W1) & _LOW
    words = torch.stack([c0, c1, c2, c3], 1)
    halves = torch.stack([words & 0xFFFF, words >> 16], 2).view(T, G * 8)[:, :D]
    thr = _threshold(s["p"])
    y = torch.where(halves >= thr, x.float() * (65536 / (65536 - thr)), 0.0)
    return (y if s["r"] is None else s["r"].float() + y).to(dt)


def _heads(m, B, heads):
    """[B * n, heads * dh] as [B, heads, n, dh] in binary32."""
    return m.float().view(B, -1, heads, m.shape[1] // heads).transpose(1, 2).contiguous()


def _rows(x, heads):
    """[B, H, n, dh] as [B * n, heads * dh], heads that share summed."""
    B, H, n, dh = x.shape
    return x.view(B, heads, H // heads, n, dh).sum(2).transpose(1, 2).reshape(B * n, heads * dh)


def _product(a, b):
    return torch.matmul(a, b.contiguous())


def _plain_attn(s, dt):
    B, H, Hkv, Tq, Tk = (s[k] for k in ("B", "H", "Hkv", "Tq", "Tk"))
    scale = s["dh"] ** -0.5
    q, k, v = _heads(s["q"], B, H), _heads(s["k"], B, Hkv), _heads(s["v"], B, Hkv)
    k, v = (t.repeat_interleave(H // Hkv, 1) for t in (k, v))
    live = (torch.arange(Tk, device=q.device) < s["klen"].view(B, 1)).view(B, 1, 1, Tk)
    rows = None
    if s["qlen"] is not None:
        rows = (torch.arange(Tq, device=q.device) < s["qlen"].view(B, 1)).view(B, 1, Tq, 1)
    S = torch.where(live, _product(q, k.transpose(2, 3)) * scale, -math.inf)
    m = S.amax(3, keepdim=True)
    P = torch.exp(S - m)
    P = P / P.sum(3, keepdim=True)
    o = _product(P, v)
    if rows is not None:
        o = torch.where(rows, o, 0.0)
    if s["op"] == "attn":
        return _rows(o, H).to(dt)
    do = torch.where(rows, _heads(s["do"], B, H), 0.0)
    dv = _product(P.transpose(2, 3), do)
    dS = P * (_product(do, v.transpose(2, 3)) - (do * o).sum(3, keepdim=True)) * scale
    return tuple(t.to(dt) for t in (_rows(o, H), _rows(_product(dS, k), H), _rows(_product(dS.transpose(2, 3), q), Hkv),
                                    _rows(dv, Hkv)))


def _plain_logprob(s, dt):
    z, t, V = s["logits"].float(), s["targets"], s["V"]
    ok = (t >= 0) & (t < V)
    at = torch.where(ok, t, 0).unsqueeze(1)
    m = z.amax(1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    lt = torch.log(total)
    p = e / total
    ent = lt - (p * d).sum(1, keepdim=True)
    logp = torch.where(ok, (d.gather(1, at) - lt).squeeze(1), 0.0)
    if s["op"] == "logprob":
        top, ids = torch.sort(z, dim=1, descending=True, stable=True)
        K = s["K"]
        return logp, ent.squeeze(1), ids[:, :K].contiguous(), top[:, :K] - m - lt
    dlogp = torch.where(ok, s["dlogp"], 0.0).unsqueeze(1)
    dz = -p * (dlogp + s["dent"].unsqueeze(1) * (d - lt + ent))
    dz.scatter_add_(1, at, dlogp)
    return logp, ent.squeeze(1), dz.to(dt)


def _plain(s):
    dt = _DT[s["dtype"]]
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "dropout": _plain_dropout, "attn": _plain_attn,
            "attn_grad": _plain_attn, "logprob": _plain_logprob, "logprob_grad": _plain_logprob}[s["op"]](s, dt)


# ---------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=None)
def _norm_plan(D, dtype, post, pre):
    """A block's plan, made once as a program that keeps its layers would."""
    from ring_all_reduce_amd import api
    kinds = {"none": api.NORM_NONE, "layer": api.NORM_LAYER, "rms": api.NORM_RMS}
    return api.rar_norm_plan(D, api.F32 if dtype == "f32" else api.BF16, kinds[post], kinds[pre], EPS)


@functools.lru_cache(maxsize=None)
def _attn_plan(H, Hkv, dh, dtype):
    from ring_all_reduce_amd import api
    return api.rar_attn_plan(H, Hkv, dh, api.F32 if dtype == "f32" else api.BF16, dh ** -0.5)


def _framework(s):
    from ring_all_reduce_amd import api
    op, dt = s["op"], _DT[s["dtype"]]
    code = api.F32 if s["dtype"] == "f32" else api.BF16

    def new(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op in ("norm", "norm_grad"):
        T, D = s["T"], s["D"]
        plan = _norm_plan(D, s["dtype"], s["post"], s["pre"])
        if op == "norm":
            h, u = new(T, D), new(T, D)
            api.rar_norm_forward(plan, T, s["x"], s["o"], s["post_w"], s["post_b"], s["gate"], s["pre_w"], s["pre_b"],
                                 h, u, a=s["a"], s=s["s"])
            return h, u
        out = {"dx": new(T, D), "do": new(T, D), "dgate": new(D), "dpre_w": new(D)}
        for name in ("post_w", "post_b", "pre_b"):
            if s[name] is not None:
                out["d" + name] = new(D)
        api.rar_norm_backward(plan, T, s["dh"], s["du"], s["o"], s["h"], s["post_w"], s["post_b"], s["gate"],
                              s["pre_w"], out["dx"], out["do"], dpost_w=out.get("dpost_w"), dpost_b=out.get("dpost_b"),
                              dgate=out["dgate"], dpre_w=out["dpre_w"], dpre_b=out.get("dpre_b"), a=s["a"], s=s["s"])
        return out
    if op == "dropout":
        y = new(s["T"], s["D"])
        api.rar_dropout(s["T"], s["D"], code, s["x"], y, s["p"], s["seed"], step=s["step"], residual=s["r"])
        return y
    if op in ("attn", "attn_grad"):
        B, Tq, Tk = s["B"], s["Tq"], s["Tk"]
        plan = _attn_plan(s["H"], s["Hkv"], s["dh"], s["dtype"])
        o = new(B * Tq, s["H"] * s["dh"])
        if op == "attn":
            api.rar_attn_forward(plan, B, Tq, Tk, s["q"], s["k"], s["v"], o, klen=s["klen"])
            return o
        lse = new(B * Tq, s["H"], dtype=torch.float32)
        lens = dict(qlen=s["qlen"], klen=s["klen"])
        api.rar_attn_forward(plan, B, Tq, Tk, s["q"], s["k"], s["v"], o, lse=lse, **lens)
        dq, dk, dv = new(*s["q"].shape), new(*s["k"].shape), new(*s["v"].shape)
        api.rar_attn_backward(plan, B, Tq, Tk, s["do"], s["q"], s["k"], s["v"], o, lse, dq, dk, dv, **lens)
        return o, dq, dk, dv
    T, V = s["T"], s["V"]
    logp, ent = new(T, dtype=torch.float32), new(T, dtype=torch.float32)
    if op == "logprob":
        ids, top = new(T, s["K"], dtype=torch.int64), new(T, s["K"], dtype=torch.float32)
        api.rar_logprob(T, V, code, s["logits"], s["targets"], logp, ent, top_ids=ids, top_logp=top)
        return logp, ent, ids, top
    dz = new(T, V)
    api.rar_logprob_grad(T, V, code, s["logits"], s["targets"], s["dlogp"], s["dent"], dz, logp=logp, entropy=ent)
    return logp, ent, dz


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


# ---------------------------------------------------------------------------
# Work and exact values
# ---------------------------------------------------------------------------

def work(case):
    op, es = case["op"], 4 if case["dtype"] == "f32" else 2
    if op in ("norm", "norm_grad"):
        n = case["T"] * case["D"]
        return {"bytes": (4 if op == "norm" else 6) * n * es + 10 * case["D"] * es, "flops": (16 if op == "norm" else 40) * n}
    if op == "dropout":
        n = case["T"] * case["D"]
        return {"bytes": (3 if case["residual"] else 2) * n * es, "flops": 12 * n}
    if op in ("attn", "attn_grad"):
        B, H, dh = case["B"], case["H"], case["dh"]
        ks = sum(_lengths(B, case["Tk"]))
        # the lengths meet each other in any order: the mean
        qs = B * case["Tq"] if op == "attn" else sum(_lengths(B, case["Tq"]))
        q, kv, pairs = qs * H * dh * es, ks * case["Hkv"] * dh * es, H * dh * qs * ks / B
        if op == "attn":
            return {"bytes": 2 * q + 2 * kv, "flops": 4 * pairs}
        return {"bytes": 4 * q + 4 * kv, "flops": 14 * pairs}
    n = case["T"] * case["V"]
    if op == "logprob":
        return {"bytes": n * es + case["T"] * (16 + 12 * case["K"]), "flops": 5 * n}
    return {"bytes": 2 * n * es + 24 * case["T"], "flops": 10 * n}


def _exact_scaled(v, kind):
    mu = torch.zeros_like(v[:, :1]) if kind != "layer" else torch.sum(v, 1, keepdim=True) / v.shape[1]
    if kind == "none":
        return mu, torch.ones_like(mu)
    var = torch.sum(torch.square(v - mu), 1, keepdim=True) / v.shape[1]
    return mu, 1 / torch.sqrt(var + EPS)


def _exact_norm(s):
    def wide(name, other):
        return torch.full((s["D"],), other, dtype=torch.float64, device=s["o"].device) if s[name] is None else s[name].double()

    o, gate, a, c = s["o"].double(), s["gate"].double(), s["a"], s["s"]
    w1, b1, w2, b2 = wide("post_w", 1.0), wide("post_b", 0.0), wide("pre_w", 1.0), wide("pre_b", 0.0)
    mo, ro = _exact_scaled(o, s["post"])
    n = (o - mo) * ro * w1 + b1
    if s["op"] == "norm":
        h = torch.addcmul(a * s["x"].double(), n, gate, value=c)
        mh, rh = _exact_scaled(h, s["pre"])
        return h, (h - mh) * rh * w2 + b2
    D = s["D"]
    h, du, dh = s["h"].double(), s["du"].double(), s["dh"].double()

    def back(dy, v, w, mu, r, kind):
        # dv = r (g - mean(g) - vh mean(g vh)), g = dy w; without the mean's term for rms
        g = dy * w
        if kind == "none":
            return g
        vh = (v - mu) * r
        first = torch.sum(g, 1, keepdim=True) / D if kind == "layer" else 0.0
        return (g - first - vh * (torch.sum(g * vh, 1, keepdim=True) / D)) * r

    mh, rh = _exact_scaled(h, s["pre"])
    g = dh + back(du, h, w2, mh, rh, s["pre"])
    dn = g * gate * c
    out = {"dx": a * g, "do": back(dn, o, w1, mo, ro, s["post"]), "dgate": c * torch.sum(g * n, 0),
           "dpre_w": torch.sum(du * (h - mh) * rh, 0)}
    if s["post_w"] is not None:
        out["dpost_w"] = torch.sum(dn * (o - mo) * ro, 0)
    if s["post_b"] is not None:
        out["dpost_b"] = torch.sum(dn, 0)
    if s["pre_b"] is not None:
        out["dpre_b"] = torch.sum(du, 0)
    return out


def _exact_dropout(s):
    T, D = s["T"], s["D"]
    G = (D + 7) // 8
    low = np.uint64(_LOW)
    step = int(s["step"].item())
    c = [np.arange(T * G, dtype=np.uint64), np.zeros(T * G, np.uint64), np.full(T * G, step & _LOW, np.uint64),
         np.full(T * G, step >> 32, np.uint64)]
    key = [s["seed"] & _LOW, s["seed"] >> 32]
    for r in range(10):
        a, b = c[0] * np.uint64(_M0), c[2] * np.uint64(_M1)      # whole products fit 64 bits
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64((key[0] + r * _W0) & _LOW), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64((key[1] + r * _W1) & _LOW), a & low]
    draws = np.stack(c, 1).astype("<u4").view("<u2").reshape(T, G * 8)[:, :D]
    thr = _threshold(s["p"])
    keep = torch.from_numpy((draws >= thr).astype(np.float64)).to(s["x"].device)
    y = s["x"].double() * keep * (65536 / (65536 - thr))
    return y if s["r"] is None else y + s["r"].double()


def _exact_attn(s):
    B, H, Hkv, Tq, Tk, dh = (s[k] for k in ("B", "H", "Hkv", "Tq", "Tk", "dh"))
    share = H // Hkv
    outs = {"o": torch.zeros(B, Tq, H, dh, dtype=torch.float64, device=s["q"].device)}
    q, k, v = (s[n].double().view(B, -1, h, dh) for n, h in (("q", H), ("k", Hkv), ("v", Hkv)))
    grad = s["op"] == "attn_grad"
    if grad:
        do = s["do"].double().view(B, Tq, H, dh)
        outs.update(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    klen = s["klen"].tolist()
    qlen = [Tq] * B if s["qlen"] is None else s["qlen"].tolist()
    for b in range(B):
        nq, nk = qlen[b], klen[b]
        for h in range(H):
            g = h // share
            Q, K, W = q[b, :nq, h], k[b, :nk, g], v[b, :nk, g]
            P = torch.softmax(Q @ K.t() / math.sqrt(dh), 1)
            outs["o"][b, :nq, h] = P @ W
            if not grad:
                continue
            G = do[b, :nq, h]
            X = G @ W.t()
            dS = P * (X - torch.sum(P * X, 1, keepdim=True)) / math.sqrt(dh)
            outs["dq"][b, :nq, h] = dS @ K
            outs["dk"][b, :nk, g] += dS.t() @ Q
            outs["dv"][b, :nk, g] += P.t() @ G
    flat = [t.reshape(-1, t.shape[2] * dh) for t in outs.values()]
    return tuple(flat) if grad else flat[0]


def _exact_logprob(s):
    z, t, V = s["logits"], s["targets"], s["V"]
    T = z.shape[0]
    lp = torch.empty(T, V, dtype=torch.float64, device=z.device)
    torch.log_softmax(z.double(), 1, out=lp)
    p = torch.exp(lp)
    ent = -torch.sum(p * lp, 1)
    live = torch.nonzero((t >= 0) & (t < V)).squeeze(1)
    logp = torch.zeros(T, dtype=torch.float64, device=z.device)
    logp[live] = lp[live, t[live]]
    if s["op"] == "logprob":
        # one whole number a logit that orders by value, then by the lower index
        bits = z.float().view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
        ids = torch.topk(key * V + (V - 1 - torch.arange(V, device=z.device)), s["K"], dim=1).values
        ids = V - 1 - torch.remainder(ids, V)
        return logp, ent, ids, torch.gather(lp, 1, ids)
    w = s["dlogp"].double() * ((t >= 0) & (t < V))
    dz = -w.unsqueeze(1) * p - s["dent"].double().unsqueeze(1) * p * (lp + ent.unsqueeze(1))
    dz[live, t[live]] += w[live]
    return logp, ent, dz


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("norm", "norm_grad"):
        return _exact_norm(s)
    if op == "dropout":
        return _exact_dropout(s)
    if op in ("attn", "attn_grad"):
        return _exact_attn(s)
    return _exact_logprob(s)
