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
