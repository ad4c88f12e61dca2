"""Attention, norms and log probabilities where a workgroup goes on for long: rings
of LDS tiles that are filled again and again, workgroups that take row after row,
rows that are collected behind one another.  References and bounds are those of
block_ref.py."""
import math

import pytest
import torch

import block_ref as R
from ring_all_reduce_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CODE = {"f32": api.F32, "bf16": api.BF16}
BOTH = ["f32", "bf16"]
INF, NAN = math.inf, math.nan


def rand(gen, *shape, dtype="f32", scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=gen) * scale + shift).to(R.DT[dtype])


def nan(*shape, dtype="f32"):
    return torch.full(shape, NAN, dtype=R.DT[dtype], device=DEV)


def dev(t):
    return None if t is None else t.to(DEV)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

def test_attention_in_bf16_rounds_weights_once():
    # The weights' rounding errors are independent and relative to each term, so a sum of terms of random sign is off
    # by what its own rounding adds: both together sqrt 2 of that.  A tenth more for the sums in binary32 and delta,
    # which comes of the rounded o (of values of a few hundredths of v's).
    B, Tq, Tk, H, dh = 3, 700, 900, 8, 128
    g = torch.Generator().manual_seed(1)
    q, do = (rand(g, B * Tq, H * dh, dtype="bf16").to(DEV) for _ in range(2))
    k, v = (rand(g, B * Tk, H * dh, dtype="bf16").to(DEV) for _ in range(2))
    plan = api.rar_attn_plan(H, H, dh, api.BF16)
    o, dq, dk, dv = (torch.empty_like(t) for t in (q, q, k, v))
    lse = nan(B * Tq, H)
    api.rar_attn_forward(plan, B, Tq, Tk, q, k, v, o, lse=lse)
    api.rar_attn_backward(plan, B, Tq, Tk, do, q, k, v, o, lse, dq, dk, dv)
    Q, K, V, G = (R.heads(t, B, H).contiguous() for t in (q, k, v, do))
    T = lambda t: t.transpose(2, 3).contiguous()  # noqa: E731
    P = torch.softmax(dh ** -0.5 * (Q @ T(K)), 3)
    X = G @ T(V)
    dS = dh ** -0.5 * P * (X - (P * X).sum(3, keepdim=True))
    want = dict(o=P @ V, dq=dS @ K, dk=T(dS) @ Q, dv=T(P) @ G)
    for got, (n, t) in zip((o, dq, dk, dv), want.items()):
        t = R.rows(t)
        once = (t.bfloat16().double() - t).norm()
        assert (got.double() - t).norm() <= 1.1 * math.sqrt(2) * once, n


# (B, Tq, Tk, H, Hkv, dh): so many workgroups that nothing is cut and each passes 5 to 16 stages, or is cut into long
# parts; runs of queries that go from one shared head to the next; every width class
LONG = [(3, 500, 430, 16, 16, 128), (5, 200, 400, 24, 8, 60), (1, 1000, 1000, 12, 12, 96), (4, 1024, 350, 16, 16, 32),
        (2, 470, 900, 16, 8, 77)]
# one token, some rows on the vector units, up to a tile on rings of a wave's own: 256 key heads, so nothing is cut
FEW = [(16, 1, 1000, 16, 16, 128), (16, 1, 700, 32, 16, 72), (32, 2, 900, 16, 8, 64), (16, 5, 1000, 32, 16, 128),
       (16, 32, 700, 16, 16, 64), (16, 9, 1000, 16, 16, 30), (32, 3, 1000, 32, 8, 90)]


def lengths(B, most):
    """Whole, and then ever shorter: down to half, one and nothing."""
    n = [most - i * most // (2 * B) for i in range(B)]
    if B > 2:
        n[-1], n[-2] = 0, 1
    return torch.tensor(n)


@pytest.mark.parametrize("shape", LONG + FEW, ids=str)
@pytest.mark.parametrize("dtype", BOTH)
def test_attention_of_many_stages(shape, dtype):
    B, Tq, Tk, H, Hkv, dh = shape
    g = torch.Generator().manual_seed(sum(shape))
    q, do = (rand(g, B * Tq, H * dh, dtype=dtype) for _ in range(2))
    k, v = (rand(g, B * Tk, Hkv * dh, dtype=dtype) for _ in range(2))
    ql, kl = lengths(B, Tq).flip(0), lengths(B, Tk)
    ql[B // 2] = Tq
    plan = api.rar_attn_plan(H, Hkv, dh, CODE[dtype])
    d = [dev(t) for t in (q, k, v)]
    lens = dict(qlen=dev(ql), klen=dev(kl))
    ws = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in api.rar_attn_workspace(plan, B, Tq, Tk)]
    out = []
    for _ in range(2):
        o, lse = nan(B * Tq, H * dh, dtype=dtype), nan(B * Tq, H)
        api.rar_attn_forward(plan, B, Tq, Tk, *d, o, lse=lse, ws=ws[0], **lens)
        grads = [torch.full_like(t, NAN) for t in d]
        api.rar_attn_backward(plan, B, Tq, Tk, dev(do), *d, o, lse, *grads, ws=ws[1], **lens)
        out.append([o, lse, *grads])
    assert all(torch.equal(a, b) for a, b in zip(*out))
    (ro, eo), (rl, el) = R.attn_forward(q, k, v, B, H, Hkv, dh ** -0.5, ql, kl, dtype)
    R.check(o, ro, eo, "o")
    gone = rl == -INF
    assert (lse.cpu()[gone] == -INF).all()
    R.check(torch.where(gone, 0.0, lse.cpu()), torch.where(gone, 0.0, rl), el, "lse")
    want = R.attn_backward(do, q, k, v, o.cpu(), lse.cpu(), B, H, Hkv, dh ** -0.5, ql, kl, dtype)
    for t, (r, e), n in zip(grads, want, ("dq", "dk", "dv")):
        R.check(t, r, e, n)


@pytest.mark.parametrize("dtype", BOTH)
def test_attention_copies_of_many_groups(dtype):
    # more 16-byte groups to copy than lanes of a launch copy at once (2^22)
    B, Tq, Tk, H, dh = 2, 5, 17000, 16, 63 if dtype == "bf16" else 31
    g = torch.Generator().manual_seed(5)
    q, do = (rand(g, B * Tq, H * dh, dtype=dtype) for _ in range(2))
    k, v = (rand(g, B * Tk, H * dh, dtype=dtype) for _ in range(2))
    plan = api.rar_attn_plan(H, H, dh, CODE[dtype])
    o, lse = nan(B * Tq, H * dh, dtype=dtype), nan(B * Tq, H)
    api.rar_attn_forward(plan, B, Tq, Tk, dev(q), dev(k), dev(v), o, lse=lse)
    (ro, eo), _ = R.attn_forward(q, k, v, B, H, H, dh ** -0.5, None, None, dtype)
    R.check(o, ro, eo, "o")
    grads = [torch.full_like(dev(t), NAN) for t in (q, k, v)]
    api.rar_attn_backward(plan, B, Tq, Tk, dev(do), dev(q), dev(k), dev(v), o, lse, *grads)
    want = R.attn_backward(do, q, k, v, o.cpu(), lse.cpu(), B, H, H, dh ** -0.5, None, None, dtype)
    for t, (r, e), n in zip(grads, want, ("dq", "dk", "dv")):
        R.check(t, r, e, n)


@pytest.mark.parametrize("Tq,Tk", [(2, 70), (40, 200), (300, 700)])
@pytest.mark.parametrize("dtype", BOTH)
def test_attention_gradient_of_queries_without_keys(Tq, Tk, dtype):
    B, H, dh = 2, 2, 40
    g = torch.Generator().manual_seed(Tq)
    q, do = (rand(g, B * Tq, H * dh, dtype=dtype) for _ in range(2))
    k, v = (rand(g, B * Tk, H * dh, dtype=dtype) for _ in range(2))
    plan = api.rar_attn_plan(H, H, dh, CODE[dtype])

    def run(q, k):
        o, lse = nan(B * Tq, H * dh, dtype=dtype), nan(B * Tq, H)
        api.rar_attn_forward(plan, B, Tq, Tk, dev(q), dev(k), dev(v), o, lse=lse)
        grads = [torch.full_like(dev(t), NAN) for t in (q, k, v)]
        api.rar_attn_backward(plan, B, Tq, Tk, dev(do), dev(q), dev(k), dev(v), o, lse, *grads)
        return o.cpu(), lse.cpu(), *(t.cpu() for t in grads)

    # every score of the first sequence is -infinity, none of the second's
    q1, k1 = q.clone(), k.clone()
    q1[:Tq], k1[:Tk] = q[:Tq].abs() + 1, -INF
    o, lse, dq, dk, dv = run(q1, k1)
    assert (o[:Tq] == 0).all() and (lse[:Tq] == -INF).all()
    assert (dq[:Tq] == 0).all() and (dk[:Tk] == 0).all() and (dv[:Tk] == 0).all()
    q1[:Tq] = k1[:Tk] = 0
    want = R.attn_backward(do, q1, k1, v, o, lse, B, H, H, dh ** -0.5, None, None, dtype)
    for t, (r, e), n in zip((dq, dk, dv), want, ("dq", "dk", "dv")):
        R.check(t, r, e, n)
    # one query's scores are: its dq is zero, the others' stay, and dk has what it multiplies in one column
    k2 = k.clone()
    k2[:, 0] = k[:, 0].abs() + 1
    q2 = q.clone()
    q2[1, 0] = -INF
    o, lse, dq, dk, dv = run(q2, k2)
    assert (o[1, :dh] == 0).all() and (lse[1, 0] == -INF).all() and (dq[1, :dh] == 0).all()
    assert torch.isnan(dk[:Tk, 0]).all()
    q2[1, 0] = dk[:Tk, 0] = 0
    want = R.attn_backward(do, q2, k2, v, o, lse, B, H, H, dh ** -0.5, None, None, dtype)
    want[1][0][:Tk, 0] = 0
    for t, (r, e), n in zip((dq, dk, dv), want, ("dq", "dk", "dv")):
        R.check(t, r, e, n)
