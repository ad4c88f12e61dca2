"""Argument checks of the norms around a block, dropout, cross attention and log
probabilities, and their references, without a GPU: every call here is refused
before it would reach a kernel, or has no rows to work on."""
import numpy as np
import pytest
import torch

import block_ref as R
from ring_all_reduce_amd import api
from ring_all_reduce_amd._lib import lib

A = [(i + 1) << 40 for i in range(24)]   # addresses far apart; never dereferenced
WS = A[23]
NAN, INF = float("nan"), float("inf")


def status(fn, *a, **k):
    with pytest.raises(api.RarError) as e:
        fn(*a, **k)
    return e.value.status


def pick(given, default):
    return default if given is None else given


# ---------------------------------------------------------------------------
# Norms
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("args", [(0, 0, 1, 1, 1e-5), ((1 << 20) + 1, 0, 1, 1, 1e-5), (8, 2, 1, 1, 1e-5),
                                  (8, 0, 3, 1, 1e-5), (8, 0, 1, -1, 1e-5), (8, 0, 1, 1, 0.0), (8, 0, 1, 1, -1.0),
                                  (8, 0, 1, 1, NAN), (8, 0, 1, 1, INF)])
def test_norm_plan_refuses(args):
    assert status(api.rar_norm_plan, *args) == api.EINVAL


def test_norm_plan_and_workspace():
    assert lib().rar_norm_plan(8, 0, 1, 1, 1e-5, None) == api.EINVAL
    assert lib().rar_norm_destroy(None) == api.OK
    assert lib().rar_norm_workspace(None, 1, None) == api.EINVAL
    for D in (1, 64, 513, 2048, 8192, 8193, 1 << 20):
        p = api.rar_norm_plan(D)
        assert api.rar_norm_workspace(p, 0) == 0
        for T in (1, 3, 1000, 1 << 24):
            n = api.rar_norm_workspace(p, T)
            assert n % 16 == 0 and n >= 16 * D and n <= 1 << 30
        assert status(api.rar_norm_workspace, p, -1) == api.EINVAL
        assert status(api.rar_norm_workspace, p, (1 << 24) + 1) == api.EINVAL
        api.rar_norm_destroy(p)


def norm_forward(p, T=10, x=A[0], ldx=None, o=A[1], ldo=None, w1=A[2], b1=A[3], gate=A[4], a=1.0, s=1.0, w2=A[5],
                 b2=A[6], h=A[7], ldh=None, u=A[8], ldu=None):
    D = p.D
    return lib().rar_norm_forward(p.handle, T, x, pick(ldx, D), o, pick(ldo, D), w1, b1, gate, a, s, w2, b2, h,
                                  pick(ldh, D), u, pick(ldu, D), None)


def test_norm_forward_refuses():
    for dt in (api.F32, api.BF16):
        p = api.rar_norm_plan(96, dt, api.NORM_LAYER, api.NORM_RMS)
        es = 4 if dt == api.F32 else 2
        for kw in (dict(x=0), dict(h=0, u=0), dict(T=-1), dict(T=(1 << 24) + 1), dict(ldx=95), dict(ldo=95),
                   dict(ldh=95), dict(ldu=95), dict(ldu=(1 << 22) + 1), dict(u=A[0]), dict(h=A[1]), dict(u=A[1]),
                   dict(u=A[7]), dict(h=A[0] + es), dict(h=A[0], ldh=200), dict(h=A[2]), dict(u=A[6]),
                   dict(u=A[4] - 96 * 9 * es)):
            assert norm_forward(p, **kw) == api.EINVAL, kw
        for kw in (dict(x=A[0] + 1), dict(o=A[1] + 1), dict(w1=A[2] + 1), dict(b1=A[3] + 1), dict(gate=A[4] + 1),
                   dict(w2=A[5] + 1), dict(b2=A[6] + 1), dict(h=A[7] + 1), dict(u=A[8] + 1)):
            assert norm_forward(p, **kw) == api.EALIGN, kw
        assert norm_forward(p, T=0, x=0, o=0, h=0, u=0) == api.OK
    assert lib().rar_norm_forward(None, 1, A[0], 8, 0, 8, 0, 0, 0, 1.0, 1.0, 0, 0, A[1], 8, 0, 8, None) == api.EINVAL


def norm_backward(p, T=10, dh=A[0], lddh=None, du=A[1], lddu=None, o=A[2], ldo=None, h=A[3], ldh=None, w1=A[4],
                  b1=A[5], gate=A[6], w2=A[7], dx=A[8], lddx=None, do=A[9], lddo=None, dw1=A[10], db1=A[11],
                  dgate=A[12], dw2=A[13], db2=A[14], ws=WS, nb=1 << 34):
    D = p.D
    return lib().rar_norm_backward(p.handle, T, dh, pick(lddh, D), du, pick(lddu, D), o, pick(ldo, D), h, pick(ldh, D),
                                   w1, b1, gate, 1.0, 1.0, w2, dx, pick(lddx, D), do, pick(lddo, D), dw1, db1, dgate,
                                   dw2, db2, 0, ws, nb, None)


def test_norm_backward_refuses():
    for dt in (api.F32, api.BF16):
        p = api.rar_norm_plan(96, dt, api.NORM_LAYER, api.NORM_RMS)
        need = api.rar_norm_workspace(p, 10)
        for kw in (dict(o=0), dict(h=0), dict(ws=0), dict(T=-1), dict(lddh=95), dict(lddu=95), dict(ldo=95),
                   dict(ldh=95), dict(lddx=95), dict(lddo=95), dict(lddo=1 << 23), dict(nb=need - 1), dict(nb=-1),
                   dict(dx=A[1]), dict(dx=A[2]), dict(dx=A[3]), dict(do=A[0]), dict(do=A[3]), dict(do=A[8]),
                   dict(dx=A[0], lddx=200), dict(do=A[2], lddo=200), dict(dw1=A[0]), dict(db1=A[2]), dict(dgate=A[6]),
                   dict(dw2=A[7]), dict(db2=A[13] + 8), dict(ws=A[8]), dict(dgate=WS + 96)):
            assert norm_backward(p, **kw) == api.EINVAL, kw
        for kw in (dict(dh=A[0] + 1), dict(du=A[1] + 1), dict(o=A[2] + 1), dict(h=A[3] + 1), dict(w1=A[4] + 1),
                   dict(gate=A[6] + 1), dict(w2=A[7] + 1), dict(dx=A[8] + 1), dict(do=A[9] + 1), dict(dw1=A[10] + 1),
                   dict(db2=A[14] + 1), dict(ws=WS + 8)):
            assert norm_backward(p, **kw) == api.EALIGN, kw
        nothing = dict(dx=0, do=0, dw1=0, db1=0, dgate=0, dw2=0, db2=0)
        assert norm_backward(p, **nothing) == api.OK
        assert norm_backward(p, T=0, dh=0, du=0, o=0, h=0, ws=0, nb=0, **nothing) == api.OK
        # gradients of what the plan does not have
        p = api.rar_norm_plan(96, dt, api.NORM_NONE, api.NORM_NONE)
        for kw in (dict(dw1=0, db1=0), dict(dw2=0, db2=0), dict(db1=0, dw2=0, db2=0), dict(dw1=0, db1=0, db2=0)):
            assert norm_backward(p, **kw) == api.EINVAL, kw


# ---------------------------------------------------------------------------
# Dropout
# ---------------------------------------------------------------------------

def test_dropout_refuses():
    def call(T=5, D=96, dt=0, p=0.1, step=A[3], x=A[0], ldx=96, r=A[1], ldr=96, y=A[2], ldy=96):
        return lib().rar_dropout(T, D, dt, p, 7, step, x, ldx, r, ldr, y, ldy, None)

    for kw in (dict(T=-1), dict(T=(1 << 24) + 1), dict(D=0), dict(D=(1 << 20) + 1), dict(dt=2), dict(p=-0.01),
               dict(p=1.01), dict(p=NAN), dict(x=0), dict(y=0), dict(ldx=95), dict(ldr=95), dict(ldy=95),
               dict(y=A[0] + 4), dict(y=A[1] + 96 * 4), dict(y=A[0], ldy=100), dict(y=A[3]),
               dict(T=1 << 24, D=1 << 20, ldx=1 << 20, ldr=1 << 20, ldy=1 << 20)):
        assert call(**kw) == api.EINVAL, kw
    for kw in (dict(x=A[0] + 2), dict(r=A[1] + 2), dict(y=A[2] + 2), dict(step=A[3] + 4)):
        assert call(**kw) == api.EALIGN, kw
    assert call(T=0, x=0, y=0) == api.OK
    with pytest.raises(ValueError):
        api.rar_dropout(1, 8, api.F32, A[0], A[1], 0.1, 1 << 64)
    with pytest.raises(ValueError):
        api.rar_dropout(1, 8, api.F32, A[0], A[1], 0.1, -1)


def test_philox_reference_is_the_published_generator():
    # Random123's known-answer test of philox4x32 with ten rounds: counter and key of zeros, of ones, and of pi's digits
    kat = [((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
           ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
           ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
            (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))]
    for counter, key, want in kat:
        got = R.philox(np.array([counter], dtype=np.uint64), key)[0]
        assert tuple(int(v) for v in got) == want


# ---------------------------------------------------------------------------
# Cross attention
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("args", [(0, 1, 8, 0, 1.0), (4, 0, 8, 0, 1.0), (4, 3, 8, 0, 1.0), (4, 8, 8, 0, 1.0),
                                  (4, 4, 0, 0, 1.0), (4, 4, 129, 0, 1.0), (4, 4, 8, 2, 1.0), (4, 4, 8, 0, 0.0),
                                  (4, 4, 8, 0, -1.0), (4, 4, 8, 0, NAN), (4, 4, 8, 0, INF), (1 << 14, 1, 65, 0, 1.0)])
def test_attn_plan_refuses(args):
    assert status(api.rar_attn_plan, *args) == api.EINVAL


def test_attn_workspace():
    assert lib().rar_attn_plan(4, 2, 8, 0, 1.0, None) == api.EINVAL
    assert lib().rar_attn_destroy(None) == api.OK
    assert lib().rar_attn_workspace(None, 1, 1, 1, None, None) == api.EINVAL
    p = api.rar_attn_plan(4, 2, 60, api.BF16)
    assert lib().rar_attn_workspace(p.handle, 1, 1, 1, None, None) == api.OK
    for B, Tq, Tk in ((0, 0, 0), (1, 1, 0), (1, 0, 1), (2, 1, 1000), (3, 500, 700), (1, 1, 1 << 24), (1, 1 << 24, 1)):
        f, b = api.rar_attn_workspace(p, B, Tq, Tk)
        assert f % 16 == 0 and b % 16 == 0 and b >= 0 and f >= 0
    for B, Tq, Tk in ((-1, 1, 1), (1, -1, 1), (1, 1, -1), (65536, 1, 1), (1, (1 << 24) + 1, 1), (2, 1, 1 << 24),
                      (1 << 15, 1 << 10, 1)):
        assert status(api.rar_attn_workspace, p, B, Tq, Tk) == api.EINVAL
    # more rows of heads than a launch takes
    p = api.rar_attn_plan(1 << 14, 1 << 14, 64, api.BF16)
    assert status(api.rar_attn_workspace, p, 1, 1 << 24, 1) == api.EINVAL


def attn_forward(p, B=3, Tq=5, Tk=70, q=A[0], ldq=None, k=A[1], ldk=None, v=A[2], ldv=None, qlen=A[3], klen=A[4],
                 o=A[5], ldo=None, lse=A[6], ws=WS, nb=1 << 34):
    w, n = p.H * p.dh, p.Hkv * p.dh
    return lib().rar_attn_forward(p.handle, B, Tq, Tk, q, pick(ldq, w), k, pick(ldk, n), v, pick(ldv, n), qlen, klen,
                                  o, pick(ldo, w), lse, ws, nb, None)


def attn_backward(p, B=3, Tq=5, Tk=70, do=A[0], lddo=None, q=A[1], ldq=None, k=A[2], ldk=None, v=A[3], ldv=None,
                  qlen=A[4], klen=A[5], o=A[6], ldo=None, lse=A[7], dq=A[8], lddq=None, dk=A[9], lddk=None, dv=A[10],
                  lddv=None, ws=WS, nb=1 << 34):
    w, n = p.H * p.dh, p.Hkv * p.dh
    return lib().rar_attn_backward(p.handle, B, Tq, Tk, do, pick(lddo, w), q, pick(ldq, w), k, pick(ldk, n), v,
                                   pick(ldv, n), qlen, klen, o, pick(ldo, w), lse, dq, pick(lddq, w), dk, pick(lddk, n),
                                   dv, pick(lddv, n), ws, nb, None)


def test_attn_forward_refuses():
    for dt in (api.F32, api.BF16):
        es = 4 if dt == api.F32 else 2
        p = api.rar_attn_plan(4, 2, 24, dt)
        need = api.rar_attn_workspace(p, 3, 5, 70)[0]
        for kw in (dict(q=0), dict(k=0), dict(v=0), dict(o=0), dict(ws=0), dict(B=-1), dict(B=65536), dict(Tq=-1),
                   dict(Tk=-1), dict(ldq=95), dict(ldo=95), dict(ldk=47), dict(ldv=47), dict(ldk=(1 << 22) + 1),
                   dict(nb=need - 1), dict(o=A[0]), dict(o=A[1]), dict(o=A[2] + 16), dict(o=A[3]), dict(o=A[4]),
                   dict(lse=A[0]), dict(lse=A[5]), dict(ws=A[5]), dict(ws=A[1]), dict(o=WS + 64),
                   dict(o=A[0] + 15 * 96 * es - es)):
            assert attn_forward(p, **kw) == api.EINVAL, kw
        for kw in (dict(q=A[0] + 1), dict(k=A[1] + 1), dict(v=A[2] + 1), dict(o=A[5] + 1), dict(qlen=A[3] + 4),
                   dict(klen=A[4] + 4), dict(lse=A[6] + 2), dict(ws=WS + 8)):
            assert attn_forward(p, **kw) == api.EALIGN, kw
        assert attn_forward(p, Tq=0, q=0, o=0) == api.OK
        assert attn_forward(p, B=0, q=0, o=0, k=0, v=0) == api.OK


def test_attn_backward_refuses():
    for dt in (api.F32, api.BF16):
        p = api.rar_attn_plan(4, 2, 24, dt)
        need = api.rar_attn_workspace(p, 3, 5, 70)[1]
        for kw in (dict(do=0), dict(q=0), dict(k=0), dict(v=0), dict(o=0), dict(lse=0), dict(ws=0), dict(B=-1),
                   dict(Tq=-1), dict(lddo=95), dict(ldq=95), dict(ldk=47), dict(ldv=47), dict(ldo=95), dict(lddq=95),
                   dict(lddk=47), dict(lddv=47), dict(nb=need - 1), dict(dq=A[0]), dict(dq=A[1]), dict(dk=A[2]),
                   dict(dv=A[3]), dict(dv=A[9]), dict(dq=A[6]), dict(dk=A[7]), dict(dk=A[5]), dict(ws=A[8]),
                   dict(ws=A[0])):
            assert attn_backward(p, **kw) == api.EINVAL, kw
        for kw in (dict(do=A[0] + 1), dict(q=A[1] + 1), dict(k=A[2] + 1), dict(v=A[3] + 1), dict(qlen=A[4] + 4),
                   dict(klen=A[5] + 4), dict(o=A[6] + 1), dict(lse=A[7] + 2), dict(dq=A[8] + 1), dict(dk=A[9] + 1),
                   dict(dv=A[10] + 1), dict(ws=WS + 8)):
            assert attn_backward(p, **kw) == api.EALIGN, kw
        assert attn_backward(p, dq=0, dk=0, dv=0) == api.OK
        assert attn_backward(p, B=0) == api.OK
        assert attn_backward(p, Tq=0, Tk=0) == api.OK


# ---------------------------------------------------------------------------
# Log probabilities
# ---------------------------------------------------------------------------

def test_logprob_refuses():
    def value(T=5, V=100, dt=0, z=A[0], ld=100, scale=1.0, t=A[1], lp=A[2], ent=A[3], K=4, ids=A[4], tl=A[5]):
        return lib().rar_logprob(T, V, dt, z, ld, scale, t, lp, ent, K, ids, tl, None)

    for kw in (dict(T=-1), dict(T=(1 << 24) + 1), dict(V=0), dict(V=(1 << 20) + 1, ld=1 << 21), dict(dt=2),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(z=0), dict(ld=99), dict(t=0),
               dict(K=-1), dict(K=33), dict(ids=0), dict(tl=0), dict(lp=A[0]), dict(ent=A[2]), dict(ids=A[5]),
               dict(tl=A[0] + 400), dict(lp=A[1] + 4)):
        assert value(**kw) == api.EINVAL, kw
    for kw in (dict(z=A[0] + 2), dict(t=A[1] + 4), dict(lp=A[2] + 2), dict(ent=A[3] + 2), dict(ids=A[4] + 4),
               dict(tl=A[5] + 2)):
        assert value(**kw) == api.EALIGN, kw
    assert value(T=0, z=0) == api.OK

    def grad(T=5, V=100, dt=0, z=A[0], ld=100, scale=1.0, t=A[1], dlp=A[2], de=A[3], lp=A[4], ent=A[5], dz=A[6],
             lddz=100):
        return lib().rar_logprob_grad(T, V, dt, z, ld, scale, t, dlp, de, lp, ent, dz, lddz, None)

    for kw in (dict(T=-1), dict(V=0), dict(dt=-1), dict(scale=0.0), dict(z=0), dict(dz=0), dict(ld=99), dict(lddz=99),
               dict(t=0), dict(t=0, lp=0), dict(t=0, dlp=0), dict(dz=A[0] + 4), dict(dz=A[0], lddz=104), dict(dz=A[1]),
               dict(dz=A[2]), dict(lp=A[2]), dict(ent=A[0] + 4), dict(lp=A[6]), dict(lp=A[5])):
        assert grad(**kw) == api.EINVAL, kw
    for kw in (dict(z=A[0] + 2), dict(dz=A[6] + 2), dict(t=A[1] + 4), dict(dlp=A[2] + 2), dict(de=A[3] + 2),
               dict(lp=A[4] + 2), dict(ent=A[5] + 2)):
        assert grad(**kw) == api.EALIGN, kw
    assert grad(T=0, z=0, dz=0) == api.OK


def test_binding_refuses_wrong_tensors():
    p = api.rar_norm_plan(8)
    x = torch.zeros(4, 8)
    for bad in (x.double(), x[:3], torch.zeros(4, 16)[:, ::2], x):   # the last: not on the GPU
        with pytest.raises(ValueError):
            api.rar_norm_forward(p, 4, bad, None, None, None, None, None, None, A[0], A[1])
    a = api.rar_attn_plan(2, 1, 8)
    with pytest.raises(ValueError):
        api.rar_attn_forward(a, 1, 4, 4, torch.zeros(4, 8), A[0], A[1], A[2])
    with pytest.raises(ValueError):
        api.rar_attn_forward(a, 1, 4, 4, A[0], A[1], A[2], A[3], klen=torch.zeros(1, dtype=torch.int32), ws=None)
    with pytest.raises(TypeError):
        api.rar_logprob(4, 8, api.F32, A[0], A[1], A[2], top_ids=A[3], top_logp=A[4])
    with pytest.raises(ValueError):
        api.rar_logprob(4, 8, api.F32, A[0], A[1], A[2], top_ids=torch.zeros(4, 2, dtype=torch.int64),
                        top_logp=torch.zeros(4, 3))


# ---------------------------------------------------------------------------
# The references against automatic differentiation
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("post", R.KINDS)
@pytest.mark.parametrize("pre", R.KINDS)
def test_norm_reference(post, pre):
    g = torch.Generator().manual_seed(1)
    T, D, eps, a, s = 5, 13, 1e-3, 0.7, 1.3
    x, o, dh, du = (torch.randn(T, D, generator=g, dtype=torch.float64) for _ in range(4))
    w1, b1, gate, w2, b2 = (torch.randn(D, generator=g, dtype=torch.float64) for _ in range(5))
    leaves = [t.requires_grad_() for t in (x, o, w1, b1, gate, w2, b2)]

    def norm(v, w, b, kind):
        if kind == "none":
            return v
        d = v - v.mean(1, keepdim=True) if kind == "layer" else v
        return d / torch.sqrt((d * d).mean(1, keepdim=True) + eps) * w + b

    h = a * x + s * gate * norm(o, w1, b1, post)
    u = norm(h, w2, b2, pre)
    (rh, _), (ru, _) = R.norm_forward(x, o, w1, b1, gate, w2, b2, post, pre, eps, a, s, "f32")
    assert torch.allclose(rh, h) and torch.allclose(ru, u)
    want = torch.autograd.grad((h * dh).sum() + (u * du).sum(), leaves, allow_unused=True)
    got = R.norm_backward(dh, du, o, h, w1, b1, gate, w2, post, pre, eps, a, s, "f32")
    for name, v in zip(("dx", "do", "dpost_w", "dpost_b", "dgate", "dpre_w", "dpre_b"), want):
        if v is not None:
            assert torch.allclose(got[name][0], v), name


@pytest.mark.parametrize("H,Hkv", [(2, 2), (6, 2)])
def test_attn_reference(H, Hkv):
    g = torch.Generator().manual_seed(2)
    B, Tq, Tk, dh, scale = 3, 4, 7, 5, 0.6
    q, k, v, do = (torch.randn(B * n, h * dh, generator=g, dtype=torch.float64, requires_grad=True)
                   for n, h in ((Tq, H), (Tk, Hkv), (Tk, Hkv), (Tq, H)))
    qlen, klen = torch.tensor([4, 2, 0]), torch.tensor([7, 1, 3])
    out = []
    for b in range(B):
        for t in range(Tq):
            for h in range(H):
                kk = k.view(B, Tk, Hkv, dh)[b, :klen[b], h // (H // Hkv)]
                vv = v.view(B, Tk, Hkv, dh)[b, :klen[b], h // (H // Hkv)]
                p = torch.softmax(scale * kk @ q.view(B, Tq, H, dh)[b, t, h], 0)
                out.append(p @ vv if t < qlen[b] else 0 * vv[0])
    o = torch.stack(out).view(B * Tq, H * dh)
    (ro, _), (lse, _) = R.attn_forward(q.detach(), k.detach(), v.detach(), B, H, Hkv, scale, qlen, klen, "f32")
    assert torch.allclose(ro, o)
    want = torch.autograd.grad((o * do.detach()).sum(), [q, k, v])
    got = R.attn_backward(*(t.detach() for t in (do, q, k, v)), ro.detach(), lse, B, H, Hkv, scale, qlen, klen, "f32")
    for (x, _), y in zip(got, want):
        assert torch.allclose(x, y)


def test_logprob_reference():
    g = torch.Generator().manual_seed(3)
    T, V, scale = 6, 11, 0.8
    z = torch.randn(T, V, generator=g, dtype=torch.float64, requires_grad=True)
    t = torch.randint(0, V, (T,), generator=g)
    t[1] = -1
    dl, de = torch.randn(T, generator=g, dtype=torch.float64), torch.randn(T, generator=g, dtype=torch.float64)
    lp = torch.log_softmax(z * scale, 1)
    logp = torch.where(t >= 0, lp.gather(1, t.clamp(min=0).unsqueeze(1)).squeeze(1), 0.0)
    ent = -(lp.exp() * lp).sum(1)
    (a, _), (b, _) = R.logprob(z.detach(), t, scale)
    assert torch.allclose(a, logp) and torch.allclose(b, ent)
    want, = torch.autograd.grad((logp * dl + ent * de).sum(), [z])
    assert torch.allclose(R.logprob_grad(z.detach(), t, dl, de, scale, "f32")[0], want)
    ids, top, _ = R.top(z.detach(), scale, 4)
    v, i = torch.topk(lp, 4)
    assert (ids == i).all() and torch.allclose(top, v)
