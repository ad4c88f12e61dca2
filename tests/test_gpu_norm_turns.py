"""The norms around a block where every workgroup takes row after row, in place and
not.  A column sum's bound counts the additions that a term passes through, so that
a row too many or too few shows."""
import math

import pytest
import torch

import block_ref as R
from ring_all_reduce_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CODE = {"f32": api.F32, "bf16": api.BF16}

# (T, D): each number of lanes a row (64 to 1024) and rows beyond the registers; three turns of the forward kernel's
# grid, the last one broken, and five or six of the backward kernel's
TURNS = [(16421, 100), (8253, 700), (4129, 1500), (2069, 3000), (1043, 5000), (1033, 8200)]


def column_sums(v, m, post, pre, eps, s, dtype, turns):
    """{name: (value, bound)} of the vectors' gradients.  A term is added in its workgroup (`turns` rows, of up to
    four beside each other), then over at most three chunks, four exchanges and 16 waves."""
    E, u = R.E, R.U[dtype]
    n = turns + 3 + 3 + 4 + 16
    g, eg = R.norm_backward(m["dh"], m["du"], m["o"], m["h"], v["post_w"], v["post_b"], v["gate"], v["pre_w"], post,
                            pre, eps, 1.0, s, "f32")["dx"]
    zero = torch.zeros_like(g)
    oh, eoh, _ = R._stats(m["o"].double(), zero, post, eps)
    hh, ehh, _ = R._stats(m["h"].double(), zero, pre, eps)
    du = m["du"].double()

    def total(a, ea, b, eb):
        t = (a * b).abs()
        return (a * b).sum(0), (ea * b.abs() + a.abs() * eb + (n + 1) * E * t).sum(0)

    one = torch.ones_like(g)
    A, eA = total(g, eg, oh, eoh)
    B, eB = total(g, eg, one, zero)
    w, b, sg = v["post_w"].double(), v["post_b"].double(), s * v["gate"].double()
    out = dict(dpre_w=total(du, zero, hh, ehh), dpre_b=total(du, zero, one, zero),
               dpost_w=(sg * A, sg.abs() * (eA + 3 * E * A.abs())), dpost_b=(sg * B, sg.abs() * (eB + 3 * E * B.abs())),
               dgate=(s * (w * A + b * B),
                      abs(s) * (w.abs() * eA + b.abs() * eB + 4 * E * ((w * A).abs() + (b * B).abs()))))
    return {k: (t, 1.1 * e * (1 + u) + u * t.abs()) for k, (t, e) in out.items()}



@pytest.mark.parametrize("kinds", [("layer", "layer"), ("rms", "layer"), ("layer", "rms")], ids=str)
@pytest.mark.parametrize("shape", TURNS, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_of_many_turns(shape, kinds, dtype):
    T, D = shape
    post, pre = kinds
    g = torch.Generator().manual_seed(T + D)

    def rand(*size, scale=1.0, shift=0.0):
        return (torch.randn(*size, generator=g) * scale + shift).to(R.DT[dtype])

    v = {n: rand(D, scale=0.3, shift=sh) for n, sh in (("post_w", 1.0), ("post_b", 0.0), ("gate", 0.5), ("pre_w", 1.0),
                                                       ("pre_b", 0.0))}
    m = {n: rand(T, D, shift=sh) for n, sh in (("x", 3.0), ("o", -0.5), ("h", 3.0), ("dh", 0.0), ("du", 0.1))}
    eps, s = 1e-5, 1.5
    plan = api.rar_norm_plan(D, CODE[dtype], R.KINDS[post], R.KINDS[pre], eps)
    d, w = {n: t.to(DEV) for n, t in v.items()}, {n: t.to(DEV) for n, t in m.items()}
    h, u = (torch.full_like(w["x"], math.nan) for _ in range(2))
    vectors = [d[n] for n in ("post_w", "post_b", "gate", "pre_w", "pre_b")]
    api.rar_norm_forward(plan, T, w["x"], w["o"], *vectors, h, u, s=s)
    want = R.norm_forward(m["x"], m["o"], *(v[n] for n in ("post_w", "post_b", "gate", "pre_w", "pre_b")), post, pre,
                          eps, 1.0, s, dtype)
    R.check(h, *want[0], "h")
    R.check(u, *want[1], "u")
    x, u2 = w["x"].clone(), torch.full_like(u, math.nan)
    api.rar_norm_forward(plan, T, x, w["o"], *vectors, x, u2, s=s)           # h over x
    assert torch.equal(x, h) and torch.equal(u2, u)

    names = ("dpost_w", "dpost_b", "dgate", "dpre_w", "dpre_b")
    vectors = [d[n] for n in ("post_w", "post_b", "gate", "pre_w")]
    ws = torch.full((api.rar_norm_workspace(plan, T),), 255, dtype=torch.uint8, device=DEV)
    out = {n: torch.full((D,), math.nan, dtype=R.DT[dtype], device=DEV) for n in names}
    dx, do = (torch.full_like(w["x"], math.nan) for _ in range(2))
    api.rar_norm_backward(plan, T, w["dh"], w["du"], w["o"], w["h"], *vectors, dx, do, **out, s=s, ws=ws)
    want = R.norm_backward(m["dh"], m["du"], m["o"], m["h"], *(v[n] for n in ("post_w", "post_b", "gate", "pre_w")),
                           post, pre, eps, 1.0, s, dtype)
    R.check(dx, *want["dx"], "dx")
    R.check(do, *want["do"], "do")
    lanes = next(n for n in (64, 128, 256, 512, 1024, 1 << 30) if n * 8 >= D)
    most = 768 if lanes <= 256 else (512 if lanes == 512 else 256)
    turns = -(-T // (most * max(1, 256 // lanes)))
    assert turns >= 3
    want = column_sums(v, m, post, pre, eps, s, dtype, turns)
    # (the bounds tell a row too few: without the last one they would not hold; in bf16 a long sum's rounding hides it)
    short = column_sums(v, {n: t[:-1] for n, t in m.items()}, post, pre, eps, s, dtype, turns)
    for n, (t, e) in want.items():
        R.check(out[n], t, e, n)
        assert dtype == "bf16" or ((t - short[n][0]).abs() > e + short[n][1]).any()
    again = {n: torch.full_like(t, math.nan) for n, t in out.items()}
    dh, o = w["dh"].clone(), w["o"].clone()
    # dx over dh, do over o
    api.rar_norm_backward(plan, T, dh, w["du"], o, w["h"], *vectors, dh, o, **again, s=s, ws=ws)
    assert torch.equal(dh, dx) and torch.equal(o, do)
    assert all(torch.equal(again[n], out[n]) for n in names)
