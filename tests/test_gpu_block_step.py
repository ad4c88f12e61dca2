"""A training step of a decoder's layer with cross attention: embedding, norms,
projections, attention to an encoder's states, dropout, feed-forward layer and
loss, forward and backward through the library, against automatic
differentiation in 64 bits; then the gradients' all-reduce over two ranks, and the
step captured into a graph."""
import math

import pytest
import torch

import block_ref as R
from ring_all_reduce_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS, P_DROP, SEED = 1e-5, 0.2, 1234
B, TQ, TK, D, H, HKV, DH, F, V = 3, 17, 29, 64, 4, 2, 16, 96, 131
T, TE = B * TQ, B * TK
NARROW = HKV * DH

# the parameters, in the order in which the backward pass makes their gradients
SHAPES = dict(w_out=(D, V), ln3_b=(D,), ln3_w=(D,), b2=(D,), w2=(F, D), b1=(F,), w1=(D, F), ln2_b=(D,), ln2_w=(D,),
              gate=(D,), post_b=(D,), post_w=(D,), bo=(D,), wo=(H * DH, D), bkv=(2 * NARROW,), wkv=(D, 2 * NARROW),
              bq=(H * DH,), wq=(D, H * DH), ln1_b=(D,), ln1_w=(D,), table=(V, D))


def parameters(seed):
    g = torch.Generator().manual_seed(seed)
    out = {}
    for n, s in SHAPES.items():
        t = torch.randn(*s, generator=g)
        if len(s) == 2:
            t = t * s[0] ** -0.5 if n != "table" else t * D ** -0.5
        elif n.startswith(("ln", "post")) and n.endswith("w") or n == "gate":
            t = 1 + 0.2 * t
        else:
            t = 0.1 * t
        out[n] = t
    return out


def batch(seed):
    g = torch.Generator().manual_seed(100 + seed)
    ids = torch.randint(0, V, (T,), generator=g)
    targets = torch.randint(0, V, (T,), generator=g)
    targets[::7] = -1                                     # padding
    states = torch.randn(TE, D, generator=g)
    klen = torch.tensor([TK, 11, 20])
    return ids, targets, states, klen


def plain_step(w, ids, targets, states, klen, mask, mscale):
    """Loss and gradients by automatic differentiation in 64 bits."""
    w = {n: t.double().requires_grad_() for n, t in w.items()}
    ln = torch.nn.functional.layer_norm

    x0 = math.sqrt(D) * w["table"][ids]
    u = ln(x0, (D,), w["ln1_w"], w["ln1_b"], EPS)
    q = (u @ w["wq"] + w["bq"]).view(B, TQ, H, DH)
    kv = (states.double() @ w["wkv"] + w["bkv"]).view(B, TK, 2, HKV, DH)
    o = []
    for b in range(B):
        k, v = (kv[b, :klen[b], i].repeat_interleave(H // HKV, 1).transpose(0, 1) for i in (0, 1))
        p = torch.softmax(q[b].transpose(0, 1) @ k.transpose(1, 2) * DH ** -0.5, 2)
        o.append((p @ v).transpose(0, 1).reshape(TQ, H * DH))
    z = torch.cat(o) @ w["wo"] + w["bo"]
    z = torch.where(mask, z * mscale, 0.0)
    n = z / torch.sqrt((z * z).mean(1, keepdim=True) + EPS) * w["post_w"] + w["post_b"]
    h1 = x0 + 0.5 * w["gate"] * n
    u1 = ln(h1, (D,), w["ln2_w"], w["ln2_b"], EPS)
    a = u1 @ w["w1"] + w["b1"]
    f = 0.5 * a * torch.special.erfc(-a / 2 ** 0.5) @ w["w2"] + w["b2"]
    u2 = ln(h1 + f, (D,), w["ln3_w"], w["ln3_b"], EPS)
    lp = torch.log_softmax(u2 @ w["w_out"], 1)
    ok = targets >= 0
    loss = -(lp.gather(1, targets.clamp(min=0).unsqueeze(1)).squeeze(1) * ok).sum() / T
    grads = torch.autograd.grad(loss, list(w.values()))
    return loss.item(), dict(zip(w, grads))


class Step:
    """The same through the library; gradients land in one arena, in the order of SHAPES."""

    def __init__(self):
        self.linears = {n: api.rar_linear_plan(*SHAPES["w" + n], api.F32, act) for n, act in (
            ("q", 0), ("kv", 0), ("o", 0), ("1", api.ACT_GELU), ("2", 0), ("_out", 0))}
        self.first = api.rar_norm_plan(D, api.F32, api.NORM_NONE, api.NORM_LAYER, EPS)
        self.mid = api.rar_norm_plan(D, api.F32, api.NORM_RMS, api.NORM_LAYER, EPS)
        self.attn = api.rar_attn_plan(H, HKV, DH, api.F32)
        self.arena = torch.empty(sum(math.prod(s) for s in SHAPES.values()), device=DEV)
        self.grad, at = {}, 0
        for n, s in SHAPES.items():
            self.grad[n] = self.arena[at:at + math.prod(s)].view(s)
            at += math.prod(s)
        new = lambda *s: torch.full(s, math.nan, device=DEV)  # noqa: E731
        self.m = {n: new(T, D) for n in ("x0", "u0", "z", "zd", "h1", "u1", "f2", "h2", "u2", "du2", "dh2", "df2",
                                         "du1", "dh1", "dzd", "dz", "dx0", "du0", "o", "do", "q", "dq")}
        self.kv, self.dkv = new(TE, 2 * NARROW), new(TE, 2 * NARROW)
        self.f, self.pre, self.df = new(T, F), new(T, F), new(T, F)
        self.logits, self.lse, self.logp = new(T, V), new(T, H), new(T)
        self.dlogp = torch.full((T,), -1.0 / T, device=DEV)
        self.step = torch.tensor([7], device=DEV)

    def linear(self, n, x, w, y, bias=None, pre=None):
        api.rar_linear_forward(self.linears[n], x.shape[0], x, w["w" + n], bias, None, y, pre=pre)

    def back(self, n, dy, x, w, dx, bias=None, pre=None):
        api.rar_linear_backward(self.linears[n], x.shape[0], dy, x, w["w" + n], pre, dx, self.grad["w" + n],
                                self.grad[bias] if bias else None)

    def __call__(self, w, ids, targets, states, klen):
        m, g = self.m, self.grad
        k, v = self.kv[:, :NARROW], self.kv[:, NARROW:]
        api.rar_embed_lookup(V, D, api.F32, w["table"], T, ids, m["x0"], math.sqrt(D))
        api.rar_norm_forward(self.first, T, m["x0"], None, None, None, None, w["ln1_w"], w["ln1_b"], None, m["u0"])
        self.linear("q", m["u0"], w, m["q"], w["bq"])
        self.linear("kv", states, w, self.kv, w["bkv"])
        api.rar_attn_forward(self.attn, B, TQ, TK, m["q"], k, v, m["o"], lse=self.lse, klen=klen)
        self.linear("o", m["o"], w, m["z"], w["bo"])
        api.rar_dropout(T, D, api.F32, m["z"], m["zd"], P_DROP, SEED, step=self.step)
        api.rar_norm_forward(self.mid, T, m["x0"], m["zd"], w["post_w"], w["post_b"], w["gate"], w["ln2_w"],
                             w["ln2_b"], m["h1"], m["u1"], s=0.5)
        self.linear("1", m["u1"], w, self.f, w["b1"], pre=self.pre)
        self.linear("2", self.f, w, m["f2"], w["b2"])
        api.rar_norm_forward(self.first, T, m["h1"], m["f2"], None, None, None, w["ln3_w"], w["ln3_b"], m["h2"],
                             m["u2"])
        self.linear("_out", m["u2"], w, self.logits)
        # the loss and its gradient, over the logits
        api.rar_logprob_grad(T, V, api.F32, self.logits, targets, self.dlogp, None, self.logits, logp=self.logp)
        self.back("_out", self.logits, m["u2"], w, m["du2"])
        api.rar_norm_backward(self.first, T, None, m["du2"], m["f2"], m["h2"], None, None, None, w["ln3_w"], m["dh2"],
                              m["df2"], dpre_w=g["ln3_w"], dpre_b=g["ln3_b"])
        self.back("2", m["df2"], self.f, w, self.df, "b2")
        self.back("1", self.df, m["u1"], w, m["du1"], "b1", pre=self.pre)
        api.rar_norm_backward(self.mid, T, m["dh2"], m["du1"], m["zd"], m["h1"], w["post_w"], w["post_b"], w["gate"],
                              w["ln2_w"], m["dh1"], m["dzd"], g["post_w"], g["post_b"], g["gate"], g["ln2_w"],
                              g["ln2_b"], s=0.5)
        api.rar_dropout(T, D, api.F32, m["dzd"], m["dz"], P_DROP, SEED, step=self.step)
        self.back("o", m["dz"], m["o"], w, m["do"], "bo")
        dk, dv = self.dkv[:, :NARROW], self.dkv[:, NARROW:]
        api.rar_attn_backward(self.attn, B, TQ, TK, m["do"], m["q"], k, v, m["o"], self.lse, m["dq"], dk, dv, klen=klen)
        self.back("kv", self.dkv, states, w, None, "bkv")
        self.back("q", m["dq"], m["u0"], w, m["du0"], "bq")
        api.rar_norm_backward(self.first, T, m["dh1"], m["du0"], None, m["x0"], None, None, None, w["ln1_w"], m["dx0"],
                              None, dpre_w=g["ln1_w"], dpre_b=g["ln1_b"])
        api.rar_embed_grad(V, D, api.F32, T, ids, m["dx0"], g["table"], math.sqrt(D))


def compare(got, want):
    # about twenty operators behind one another, each off by at most n 2^-24 of its result's norm, n <= 200 terms of a
    # sum: 2^-12 of the norm
    for n in SHAPES:
        d = (got[n].double().cpu() - want[n]).norm().item()
        assert d <= 2 ** -12 * want[n].norm().item(), (n, d, want[n].norm().item())


def test_step_of_two_ranks():
    w = parameters(0)
    wd = {n: t.to(DEV) for n, t in w.items()}
    keep, scale = R.keep_mask(T, D, P_DROP, SEED, 7)
    want, steps = [], []
    for rank in range(2):
        ids, targets, states, klen = batch(rank)
        loss, grads = plain_step(w, ids, targets, states, klen, keep, scale)
        step = Step()
        step(wd, *(t.to(DEV) for t in (ids, targets, states, klen)))
        got = -step.logp.double().sum().item() / T
        assert abs(got - loss) <= 2 ** -14 * abs(loss)
        compare(step.grad, grads)
        want.append(grads)
        steps.append(step)
    buckets = api.rar_bucket_plan([math.prod(s) for s in SHAPES.values()], api.F32, 16384)
    api.rar_bucket_allreduce_arena(buckets, [s.arena for s in steps])
    mean = {n: (want[0][n] + want[1][n]) / 2 for n in SHAPES}
    for s in steps:
        compare(s.grad, mean)


def test_step_in_a_graph():
    wd = {n: t.to(DEV) for n, t in parameters(1).items()}
    args = [t.to(DEV) for t in batch(5)]
    step = Step()
    step(wd, *args)
    torch.cuda.synchronize()
    first = step.arena.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(wd, *args)
    for n in range(3):
        step.arena.fill_(math.nan)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(step.arena, first), f"replay {n}"
        step(wd, *args)                                   # eagerly between the replays
        assert torch.equal(step.arena, first)
    # other inputs in the same buffers
    other = [t.to(DEV) for t in batch(6)]
    for a, b in zip(args, other):
        a.copy_(b)
    graph.replay()
    got = step.arena.clone()
    step(wd, *other)
    assert torch.equal(step.arena, got)
