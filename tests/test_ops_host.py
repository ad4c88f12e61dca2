"""Argument checks and host tables of the gradient-producing operators, without
a GPU: every call here is refused before it would reach a kernel, or has no
rows to work on."""
import ctypes
import pathlib
import re

import numpy as np
import pytest
import torch

import ops_ref as R
import ops_sizes as S
from ring_all_reduce_amd import api
from ring_all_reduce_amd._lib import lib

A = [(i + 1) << 40 for i in range(16)]   # addresses far apart; never dereferenced
WS = A[15]


def status(fn, *a, **k):
    with pytest.raises(api.RarError) as e:
        fn(*a, **k)
    return e.value.status


def linear(K=64, N=96, dtype=api.F32, act=api.ACT_GELU):
    return api.rar_linear_plan(K, N, dtype, act)


@pytest.mark.parametrize("K,N,dt,act", [(0, 4, 0, 0), (4, 0, 0, 0), (-1, 4, 0, 0), ((1 << 20) + 1, 4, 0, 0),
                                        (4, (1 << 20) + 1, 1, 0), (4, 4, 2, 0), (4, 4, -1, 0), (4, 4, 0, 3),
                                        (4, 4, 0, -1)])
def test_linear_plan_refuses(K, N, dt, act):
    with pytest.raises(api.RarError) as e:
        api.rar_linear_plan(K, N, dt, act)
    assert e.value.status == api.EINVAL
    assert lib().rar_linear_plan(4, 4, 0, 0, None) == api.EINVAL


def test_linear_workspace():
    p = linear()
    assert api.rar_linear_workspace(p, 0) == (0, 0)
    assert api.rar_linear_workspace(p, 1)[0] == 0     # few rows: nothing is split or copied
    f, b = api.rar_linear_workspace(p, 100)
    assert f > 0 and b > f
    last = (0, 0)
    for T in (5, 10, 100, 1000, 100_000, 1 << 24):
        f, b = api.rar_linear_workspace(p, T)
        assert f % 16 == 0 and b % 16 == 0 and f > 0 and b > last[1] // 64
        last = (f, b)
    assert status(api.rar_linear_workspace, p, -1) == api.EINVAL
    assert status(api.rar_linear_workspace, p, (1 << 24) + 1) == api.EINVAL
    assert lib().rar_linear_workspace(None, 1, None, None) == api.EINVAL
    assert lib().rar_linear_workspace(p.handle, 1, None, None) == api.OK
    api.rar_linear_destroy(p)
    assert lib().rar_linear_destroy(None) == api.OK


def forward(p, T=10, x=A[0], ldx=None, w=A[1], b=A[2], r=A[3], ldr=None, y=A[4], ldy=None, pre=A[5], ldp=None, sc=None,
            ws=WS, nb=1 << 34):
    n = lambda v, d: d if v is None else v
    return lib().rar_linear_forward(p.handle, T, x, n(ldx, p.K), w, b, r, n(ldr, p.N), y, n(ldy, p.N), pre, n(ldp, p.N),
                                    sc, ws, nb, None)


def backward(p, T=10, dy=A[0], lddy=None, x=A[1], ldx=None, xs=None, w=A[2], pre=A[3], ldp=None, ps=None, dx=A[4],
             lddx=None, dw=A[5], db=A[6], acc=0, ws=WS, nb=1 << 34):
    n = lambda v, d: d if v is None else v
    return lib().rar_linear_backward(p.handle, T, dy, n(lddy, p.N), x, n(ldx, p.K), xs, w, pre, n(ldp, p.N), ps, dx,
                                     n(lddx, p.K), dw, db, acc, ws, nb, None)


def test_linear_forward_refuses():
    for dt in (api.F32, api.BF16):
        p = linear(dtype=dt)
        es = 4 if dt == api.F32 else 2
        need = api.rar_linear_workspace(p, 10)[0]
        row = p.N * es
        for kw in (dict(x=None), dict(w=None), dict(y=None), dict(ws=None), dict(pre=None, sc=A[7]), dict(T=-1),
                   dict(T=(1 << 24) + 1), dict(ldx=63), dict(ldy=95), dict(ldr=95), dict(ldp=95),
                   dict(ldx=(1 << 22) + 1), dict(ldy=1 << 23), dict(nb=need - 1), dict(nb=-1),
                   dict(y=A[0]), dict(y=A[1]), dict(y=A[2]), dict(y=A[3] + row), dict(r=A[4], ldr=200), dict(pre=A[4]),
                   dict(pre=A[3]), dict(pre=A[0]), dict(ws=A[0]), dict(y=A[15] + 64), dict(pre=A[5], sc=A[5] + 96),
                   dict(y=A[0] + 10 * 64 * es - es), dict(sc=A[4])):
            assert forward(p, **kw) == api.EINVAL, kw
        for kw in (dict(x=A[0] + 1), dict(w=A[1] + 1), dict(b=A[2] + 1), dict(r=A[3] + 1), dict(y=A[4] + 1),
                   dict(pre=A[5] + 1), dict(pre=A[5] + 8, sc=A[7]), dict(ws=WS + 8)):
            assert forward(p, **kw) == api.EALIGN, kw
        assert forward(p, T=0, x=None, y=None) == api.OK
        assert lib().rar_linear_forward(None, 1, A[0], 64, A[1], None, None, 96, A[4], 96, None, 96, None, WS, 1 << 30,
                                        None) == api.EINVAL


def test_linear_backward_refuses():
    for dt in (api.F32, api.BF16):
        p = linear(dtype=dt)
        need = api.rar_linear_workspace(p, 10)[1]
        for kw in (dict(dy=None), dict(ws=None), dict(w=None), dict(x=None), dict(pre=None), dict(T=-1), dict(lddy=95),
                   dict(ldx=63), dict(lddx=63), dict(ldp=95), dict(lddx=1 << 23), dict(nb=need - 1), dict(dx=A[0]),
                   dict(dx=A[1]), dict(dw=A[2]), dict(db=A[3]), dict(dx=A[5]), dict(db=A[5] + 8), dict(ws=A[1]),
                   dict(xs=A[4]), dict(ps=A[5]), dict(dw=A[15])):
            assert backward(p, **kw) == api.EINVAL, kw
        for kw in (dict(dy=A[0] + 1), dict(x=A[1] + 1), dict(x=A[1] + 8, xs=A[7]), dict(w=A[2] + 1), dict(pre=A[3] + 1),
                   dict(pre=A[3] + 8, ps=A[8]), dict(dx=A[4] + 1), dict(dw=A[5] + 1), dict(db=A[6] + 1),
                   dict(ws=WS + 4)):
            assert backward(p, **kw) == api.EALIGN, kw
        assert backward(p, T=0, dy=None, x=None, pre=None, dx=None, dw=None, db=None, ws=None, nb=0) == api.OK


def test_embed_refuses():
    L = lib()

    def look(V=50, D=8, dt=0, table=A[0], T=5, ids=A[1], out=A[2], ldo=8):
        return L.rar_embed_lookup(V, D, dt, table, T, ids, 1.0, out, ldo, None)

    for kw in (dict(V=0), dict(V=(1 << 30) + 1), dict(D=0), dict(D=(1 << 20) + 1), dict(dt=2), dict(T=-1), dict(ldo=7),
               dict(table=None), dict(ids=None), dict(out=None), dict(out=A[0]), dict(out=A[0] + 50 * 32 - 4),
               dict(out=A[1]), dict(T=(1 << 24) + 1)):
        assert look(**kw) == api.EINVAL, kw
    for kw in (dict(table=A[0] + 2), dict(ids=A[1] + 4), dict(out=A[2] + 2)):
        assert look(**kw) == api.EALIGN, kw
    assert look(T=0, table=None, ids=None, out=None) == api.OK

    need = api.rar_embed_grad_workspace(50, 8, 5)
    assert need > 0
    for a in ((0, 8, 5), (50, 0, 5), (50, 8, -1)):
        assert status(api.rar_embed_grad_workspace, *a) == api.EINVAL
    assert L.rar_embed_grad_workspace(50, 8, 5, None) == api.EINVAL

    def grad(V=50, D=8, dt=0, T=5, ids=A[1], dy=A[0], lddy=8, g=A[2], ws=WS, nb=need):
        return L.rar_embed_grad(V, D, dt, T, ids, dy, lddy, 1.0, 0, g, ws, nb, None)

    for kw in (dict(V=0), dict(D=0), dict(dt=3), dict(T=-1), dict(lddy=7), dict(ids=None), dict(dy=None), dict(g=None),
               dict(ws=None), dict(nb=need - 1), dict(g=A[0]), dict(g=A[1]), dict(g=WS), dict(ws=A[0]),
               dict(V=1 << 30, D=1 << 20, nb=1 << 62),
               dict(T=1 << 24, D=1 << 20, lddy=1 << 20, nb=1 << 62)):
        assert grad(**kw) == api.EINVAL, kw
    for kw in (dict(ids=A[1] + 4), dict(dy=A[0] + 2), dict(g=A[2] + 2), dict(ws=WS + 8)):
        assert grad(**kw) == api.EALIGN, kw


def test_ckpt_size_and_refusals():
    assert api.rar_ckpt_size(1) == (32, 1)
    assert api.rar_ckpt_size(32) == (32, 1)
    assert api.rar_ckpt_size(33) == (64, 2)
    assert api.CKPT_GROUP == 32
    for D in (0, -3, (1 << 20) + 1):
        assert status(api.rar_ckpt_size, D) == api.EINVAL
    L = lib()
    st = lambda T=4, D=40, dt=0, x=A[0], ld=40, c=A[1], s=A[2]: L.rar_ckpt_store(T, D, dt, x, ld, c, s, None)
    ld = lambda T=4, D=40, dt=0, c=A[1], s=A[2], act=0, y=A[0], ldy=40: L.rar_ckpt_load(T, D, dt, c, s, act, y, ldy,
                                                                                        None)
    for kw in (dict(T=-1), dict(D=0), dict(dt=2), dict(x=None), dict(c=None), dict(s=None), dict(ld=39), dict(c=A[0]),
               dict(s=A[0]), dict(s=A[1] + 255)):
        assert st(**kw) == api.EINVAL, kw
    for kw in (dict(x=A[0] + 2), dict(c=A[1] + 8)):
        assert st(**kw) == api.EALIGN, kw
    for kw in (dict(act=3), dict(y=None), dict(c=None), dict(s=None), dict(ldy=39), dict(y=A[1]), dict(y=A[2])):
        assert ld(**kw) == api.EINVAL, kw
    assert ld(c=A[1] + 4) == api.EALIGN
    assert st(T=0, x=None, c=None, s=None) == api.OK and ld(T=0, y=None, c=None, s=None) == api.OK


def test_binding_checks_tensors_before_the_call():
    # CPU tensors: type, shape and layout are refused first, then the device
    p = linear(8, 16, api.BF16, api.ACT_RELU)
    h = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    f = lambda *s: torch.zeros(*s)
    good = dict(x=A[0], w=A[1], bias=A[2], residual=A[3], y=A[4])

    def fwd(**kw):
        a = {**good, **kw}
        api.rar_linear_forward(p, 4, a["x"], a["w"], a["bias"], a["residual"], a["y"], pre=a.get("pre"),
                               pre_scales=a.get("sc"), ws=a.get("ws"))

    for kw, say in ((dict(x=f(4, 8)), "dtype"), (dict(x=h(5, 8)), "shape"), (dict(x=h(32)), "shape"),
                    (dict(x=h(4, 16)[:, ::2]), "contiguous"), (dict(w=h(8, 15)), "elements"),
                    (dict(w=h(16, 8).T), "contiguous"), (dict(bias=f(16)), "dtype"), (dict(y=h(4, 17)), "shape"),
                    (dict(y=h(1, 16).expand(4, 16)), "overlap"), (dict(pre=h(4, 16), sc=h(4, 1)), "dtype"),
                    (dict(x=h(4, 8)), "GPU"), (dict(w=h(8, 16)), "GPU")):
        with pytest.raises(ValueError, match=say):
            fwd(**kw)
    with pytest.raises(TypeError):
        fwd(x="no")
    with pytest.raises(ValueError, match="dtype"):
        api.rar_embed_lookup(5, 8, api.F32, A[0], 3, torch.zeros(3, dtype=torch.int32), A[1])
    with pytest.raises(ValueError, match="elements"):
        api.rar_embed_grad(5, 8, api.F32, 3, A[0], A[1], f(5, 7))
    with pytest.raises(ValueError, match="elements"):
        api.rar_ckpt_store(3, 40, api.F32, A[0], torch.zeros(3, 40, dtype=torch.uint8), A[1])
    with pytest.raises(TypeError):
        api.rar_embed_grad(5, 8, api.F32, 3, A[0], A[1], A[2], ws=A[3])


def test_plain_checkpoint_definition():
    # the 64-bit reference the GPU tests use: nearest of all e4m3 values, ties to even, smallest fitting exponent
    g = torch.Generator().manual_seed(4)
    x = torch.randn(20, 70, generator=g) * torch.exp2(torch.randint(-30, 30, (20, 70), generator=g).float())
    x[0, :32] = -1.0
    x[0, :2] = torch.tensor([float("inf"), float("nan")])
    codes, scales, vals = R.quantise(x)
    back = R.values(codes, scales, 70).numpy()
    assert ((back == vals) | ((back != back) & (vals != vals))).all()
    s = torch.from_numpy(scales.astype("float64") - 127).exp2().repeat_interleave(32, 1)[:, :70].numpy()
    v = x.double().numpy()
    fine = (v == v) & (abs(v) != float("inf"))
    # half a step: 2^-4 of the value, or half the smallest step
    assert (abs(vals - v)[fine] <= (abs(v) * 2.0 ** -4 + s * 2.0 ** -10)[fine]).all()
    assert vals[0, 2] == -1 and vals[0, 0] != vals[0, 0] and vals[0, 1] != vals[0, 1]


def test_sizes_of_embedding_chunks():
    # The workspace holds two rows of partial sums a chunk and one a group of 32 chunks, beside the sort's lists (16
    # bytes a token and 1024 a workgroup of 4096): chunks of 32 sorted positions need a quarter of what chunks of 8 do.
    def chunk(T, V, D):
        part = api.rar_embed_grad_workspace(V, D, T) - 16 * T - (T + 4095) // 4096 * 1024
        return T * 2.03 * 4 * ((D + 511) // 512 * 512) / part

    for T, V, D in S.EMBED_32:
        assert (D + 511) // 512 > 1 and 30 < chunk(T, V, D) < 34
    assert 7 < chunk(9000, 70000, 9) < 9


@pytest.mark.parametrize("private", [True, False])
def test_current_device_and_stream_by_public_calls_alone(monkeypatch, private):
    # the binding asks torch's internal calls for the current device and stream, and the public ones where a torch
    # lacks those
    class Stream:
        cuda_stream = 0x1230

    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    for name, value in (("_cuda_getDevice", lambda: 3), ("_cuda_getCurrentRawStream", lambda dev: 0x1230 + dev - 3)):
        if private:
            monkeypatch.setattr(torch._C, name, value, raising=False)
        else:
            monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(api, "_get_device", None)
    assert api._here() == 3 and api._on(None) == 0x1230 and api._on(Stream) == 0x1230 and api._on(7) == 7


@pytest.mark.parametrize("dtype,degree,fit", [("f32", 8, 1.02e-7), ("bf16", 6, 5.2e-6)])
def test_normal_tail_is_as_good_as_its_comment_says(dtype, degree, fit):
    # the polynomial of act.h, its constants rounded as there, against exp(x^2) erfc(x) in 64 bits
    src = (pathlib.Path(R.__file__).parents[1] / "ring_all_reduce_amd" / "csrc" / "act.h").read_text()
    assert f"{fit:.3g}".replace("e-0", "e-") in src
    body = src[src.index("void normal_tail"):]
    c = np.float32(np.float32(re.search(r"kWide \? 0\.33f : 0\.44f\) \* (0\.70710678118654752)f", body)[1]) *
                   np.float32(0.33 if dtype == "f32" else 0.44))
    half = body[:body.index("} else {")] if dtype == "f32" else body[body.index("} else {"):body.index("q *= t")]
    coeff = [np.float32(0.5) * np.float32(v) for v in re.findall(r"0\.5f \* (-?[0-9.]+)f", half)]
    assert len(coeff) == degree

    def tail(z):
        t = 1 / (1 + float(c) * z)
        q = torch.zeros_like(t)
        for a in coeff:
            q = q * t + float(a)
        return q * t

    x = torch.linspace(0, 10, 400001, dtype=torch.float64)
    rel = (tail(x * 2 ** 0.5) / (torch.special.erfcx(x) / 2) - 1).abs().max().item()
    assert rel < fit * 1.005
    # with the exponential's argument as binary32 rounds it: z^2 * 2^-24 more
    z = (x * 2 ** 0.5).float()[(x > 0) & (x < 9.3)]
    e = torch.exp2((z * (z * torch.tensor(-0.72134752044448170, dtype=torch.float32))).double())
    z = z.double()
    want = torch.special.erfc(z / 2 ** 0.5) / 2
    assert ((tail(z) * e - want).abs() <= (fit * 1.05 + z * z * 2.0 ** -24) * want).all()
    # what the header promises of gelu (|z| times the tail) and its derivative (the tail and |z| times the density)
    off = (tail(z) * e - want).abs()
    dens = (e - torch.exp(-z * z / 2)).abs() * (2 * np.pi) ** -0.5
    assert (torch.maximum(z * off, off + z * dens) <= 2.0 ** (-20 if dtype == "f32" else -18) * (1 + z)).all()
    if dtype == "bf16":
        assert fit * 700 < R.U["bf16"]
