"""The norms around a block, dropout, cross attention and log probabilities on the
GPU, against plain 64-bit forms at the sizes, layouts and values where they can
go wrong.  Bounds count roundings (see block_ref.py); nothing is fitted to
results."""
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


def nan(*shape, dtype):
    return torch.full(shape, NAN, dtype=R.DT[dtype], device=DEV)


def dev(t):
    return None if t is None else t.to(DEV)


def strided(t, extra, offset=0):
    """t on the GPU as a view of a wider matrix (rows t.shape[1] + extra apart), NaN around it."""
    big = torch.full((t.shape[0] + 1, t.shape[1] + extra), NAN, dtype=t.dtype, device=DEV)
    v = big[:t.shape[0], offset:offset + t.shape[1]]
    v.copy_(t.to(DEV))
    return v


def around_is_untouched(view):
    base = view._base
    outside = torch.ones(base.shape, dtype=torch.bool, device=DEV)
    c = view.storage_offset() % base.shape[1]
    outside[:view.shape[0], c:c + view.shape[1]] = False
    assert torch.isnan(base[outside].float()).all()


def same_bits(a, b):
    i = {2: torch.int16, 4: torch.int32, 8: torch.int64}[a.element_size()]
    return bool((a.contiguous().view(i) == b.contiguous().view(i)).all())


# ---------------------------------------------------------------------------
# Norms
# ---------------------------------------------------------------------------

# (T, D): one element, one row, widths at and around what a wave, a workgroup and registers take, and beyond them
NORM = [(1, 1), (3, 7), (1, 64), (17, 511), (9, 512), (5, 513), (130, 1000), (33, 1024), (40, 1025), (70, 2048),
        (6, 2049), (31, 4096), (3, 4100), (5, 8192), (4, 8193), (3, 20011), (2, 70001), (5001, 40), (2100, 96)]
NORM_KINDS = [("none", "layer"), ("layer", "layer"), ("rms", "rms"), ("layer", "none"), ("rms", "layer"),
              ("none", "none")]


def norm_inputs(g, T, D, dtype):
    v = {n: rand(g, D, dtype=dtype, scale=0.3, shift=sh) for n, sh in (("post_w", 1.0), ("post_b", 0.0), ("gate", 0.5),
                                                                       ("pre_w", 1.0), ("pre_b", 0.0))}
    # a mean far from zero, as a residual stream has
    m = {n: rand(g, T, D, dtype=dtype, shift=sh) for n, sh in (("x", 3.0), ("o", -0.5), ("h", 3.0), ("dh", 0.0),
                                                               ("du", 0.1))}
    return v, m


@pytest.mark.parametrize("kinds", NORM_KINDS, ids=str)
@pytest.mark.parametrize("shape", NORM, ids=str)
@pytest.mark.parametrize("dtype", BOTH)
def test_norm(shape, kinds, dtype):
    T, D = shape
    post, pre = kinds
    g = torch.Generator().manual_seed(T * 31 + D)
    v, m = norm_inputs(g, T, D, dtype)
    eps, a, s = 1e-5, 0.75, 1.5
    plan = api.rar_norm_plan(D, CODE[dtype], R.KINDS[post], R.KINDS[pre], eps)
    for vec in (v, dict.fromkeys(v)):
        d = {n: dev(t) for n, t in vec.items()}
        h, u = nan(T, D, dtype=dtype), nan(T, D, dtype=dtype)
        api.rar_norm_forward(plan, T, dev(m["x"]), dev(m["o"]), d["post_w"], d["post_b"], d["gate"], d["pre_w"],
                             d["pre_b"], h, u, a=a, s=s)
        want = R.norm_forward(m["x"], m["o"], vec["post_w"], vec["post_b"], vec["gate"], vec["pre_w"], vec["pre_b"],
                              post, pre, eps, a, s, dtype)
        R.check(h, *want[0], "h")
        R.check(u, *want[1], "u")
        out = {n: nan(T, D, dtype=dtype) for n in ("dx", "do")}
        names = ["dgate"] + (["dpost_w", "dpost_b"] if post != "none" else []) + (
            ["dpre_w", "dpre_b"] if pre != "none" else [])
        out.update({n: nan(D, dtype=dtype) for n in names})
        api.rar_norm_backward(plan, T, dev(m["dh"]), dev(m["du"]), dev(m["o"]), dev(m["h"]), d["post_w"], d["post_b"],
                              d["gate"], d["pre_w"], out["dx"], out["do"], **{n: out[n] for n in names}, a=a, s=s)
        want = R.norm_backward(m["dh"], m["du"], m["o"], m["h"], vec["post_w"], vec["post_b"], vec["gate"],
                               vec["pre_w"], post, pre, eps, a, s, dtype)
        for n, t in out.items():
            R.check(t, *want[n], n)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("D", [72, 2048, 9001])
def test_norm_parts(D, dtype):
    # without a block's output, without one of the gradients, without one of the outputs
    T, eps = 23, 1e-5
    g = torch.Generator().manual_seed(D)
    v, m = norm_inputs(g, T, D, dtype)
    plan = api.rar_norm_plan(D, CODE[dtype], api.NORM_RMS, api.NORM_LAYER, eps)
    d, w = {n: dev(t) for n, t in v.items()}, {n: dev(t) for n, t in m.items()}
    u = nan(T, D, dtype=dtype)
    api.rar_norm_forward(plan, T, w["x"], None, None, None, None, d["pre_w"], d["pre_b"], None, u)
    R.check(u, *R.norm_forward(m["x"], None, None, None, None, v["pre_w"], v["pre_b"], "rms", "layer", eps, 1, 1,
                               dtype)[1], "u without o")
    h = nan(T, D, dtype=dtype)
    api.rar_norm_forward(plan, T, w["x"], w["o"], d["post_w"], d["post_b"], d["gate"], None, None, h, None, s=0.5)
    R.check(h, *R.norm_forward(m["x"], m["o"], v["post_w"], v["post_b"], v["gate"], None, None, "rms", "layer", eps, 1,
                               0.5, dtype)[0], "h without u")
    for dh, du in (("dh", None), (None, "du")):
        dx, do, dg = nan(T, D, dtype=dtype), nan(T, D, dtype=dtype), nan(D, dtype=dtype)
        dw, db = nan(D, dtype=dtype), nan(D, dtype=dtype)
        api.rar_norm_backward(plan, T, w.get(dh), w.get(du), w["o"], w["h"], d["post_w"], d["post_b"], d["gate"],
                              d["pre_w"], dx, do, dgate=dg, dpre_w=dw, dpre_b=db)
        want = R.norm_backward(m.get(dh), m.get(du), m["o"], m["h"], v["post_w"], v["post_b"], v["gate"], v["pre_w"],
                               "rms", "layer", eps, 1, 1, dtype)
        for n, t in (("dx", dx), ("do", do), ("dgate", dg), ("dpre_w", dw), ("dpre_b", db)):
            R.check(t, *want[n], f"{n} of {dh or du}")
    dx, dw = nan(T, D, dtype=dtype), nan(D, dtype=dtype)
    api.rar_norm_backward(plan, T, w["dh"], w["du"], None, w["h"], None, None, None, d["pre_w"], dx, None, dpre_w=dw)
    want = R.norm_backward(m["dh"], m["du"], None, m["h"], None, None, None, v["pre_w"], "rms", "layer", eps, 1, 1,
                           dtype)
    R.check(dx, *want["dx"], "dx without o")
    R.check(dw, *want["dpre_w"], "dpre_w without o")


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("extra,offset", [(8, 0), (8, 8), (3, 1)])
@pytest.mark.parametrize("D", [200, 1001, 5003, 8200])
def test_norm_strides_and_in_place(D, extra, offset, dtype):
    T, eps = 37, 1e-5
    g = torch.Generator().manual_seed(4)
    v, m = norm_inputs(g, T, D, dtype)
    plan = api.rar_norm_plan(D, CODE[dtype], api.NORM_LAYER, api.NORM_LAYER, eps)
    d, w = {n: dev(t) for n, t in v.items()}, {n: strided(t, extra, offset) for n, t in m.items()}
    u = strided(torch.zeros(T, D, dtype=R.DT[dtype]), extra, offset)
    api.rar_norm_forward(plan, T, w["x"], w["o"], d["post_w"], d["post_b"], d["gate"], d["pre_w"], d["pre_b"], w["x"],
                         u)                                             # h over x
    want = R.norm_forward(m["x"], m["o"], v["post_w"], v["post_b"], v["gate"], v["pre_w"], v["pre_b"], "layer",
                          "layer", eps, 1, 1, dtype)
    R.check(w["x"], *want[0], "h")
    R.check(u, *want[1], "u")
    sums = {n: rand(g, D, dtype=dtype) for n in ("dpost_w", "dpost_b", "dgate", "dpre_w", "dpre_b")}
    got = {n: dev(t) for n, t in sums.items()}
    api.rar_norm_backward(plan, T, w["dh"], w["du"], w["o"], w["h"], d["post_w"], d["post_b"], d["gate"], d["pre_w"],
                          w["dh"], w["o"], **got, accumulate=True)      # dx over dh, do over o
    want = R.norm_backward(m["dh"], m["du"], m["o"], m["h"], v["post_w"], v["post_b"], v["gate"], v["pre_w"], "layer",
                           "layer", eps, 1, 1, dtype, before=sums)
    got.update(dx=w["dh"], do=w["o"])
    for n, t in got.items():
        R.check(t, *want[n], n)
    for n in ("x", "dh", "o"):
        around_is_untouched(w[n])
    around_is_untouched(u)


def test_norm_without_rows_and_bad_values():
    plan = api.rar_norm_plan(40, api.F32, api.NORM_NONE, api.NORM_LAYER)
    e = torch.empty(0, 40, device=DEV)
    api.rar_norm_forward(plan, 0, e, None, None, None, None, None, None, None, e.clone())
    dw, db = torch.full((40,), 2.0, device=DEV), nan(40, dtype="f32")
    api.rar_norm_backward(plan, 0, e, e, None, e, None, None, None, None, None, None, dpre_w=dw, accumulate=True)
    assert (dw == 2).all()
    api.rar_norm_backward(plan, 0, e, e, None, e, None, None, None, None, None, None, dpre_b=db)
    assert (db == 0).all()
    x = torch.randn(6, 40, device=DEV)
    want = torch.empty_like(x)
    api.rar_norm_forward(plan, 6, x, None, None, None, None, None, None, None, want)
    x[2, 3], x[4, 39] = NAN, INF
    u = torch.empty_like(x)
    api.rar_norm_forward(plan, 6, x, None, None, None, None, None, None, None, u)
    bad = torch.tensor([2, 4], device=DEV)
    assert torch.isnan(u[bad]).all()
    keep = torch.tensor([0, 1, 3, 5], device=DEV)
    assert same_bits(u[keep], want[keep])


def test_norm_gradient_against_differences():
    T, D, eps = 7, 45, 1e-2
    g = torch.Generator().manual_seed(8)
    v, m = norm_inputs(g, T, D, "f32")
    plan = api.rar_norm_plan(D, api.F32, api.NORM_RMS, api.NORM_LAYER, eps)
    d, w = {n: dev(t) for n, t in v.items()}, {n: dev(t) for n, t in m.items()}

    def loss(x, o):
        h, u = torch.empty_like(x), torch.empty_like(x)
        api.rar_norm_forward(plan, T, x, o, d["post_w"], d["post_b"], d["gate"], d["pre_w"], d["pre_b"], h, u)
        return h, ((h.double() * w["dh"].double()).sum() + (u.double() * w["du"].double()).sum()).item()

    h, _ = loss(w["x"], w["o"])
    dx, do = torch.empty_like(h), torch.empty_like(h)
    api.rar_norm_backward(plan, T, w["dh"], w["du"], w["o"], h, d["post_w"], d["post_b"], d["gate"], d["pre_w"], dx, do)
    # a step of 2^-6 along a direction: the loss, a sum of 2 T D binary32 values of unit size, is known to about
    # 2^-22 * sqrt(2 T D) and its third derivative contributes 2^-12 of the gradient's size
    for name, grad in (("x", dx), ("o", do)):
        r = torch.randn(T, D, generator=g).to(DEV)
        r /= r.norm()
        step = 2.0 ** -6
        args = [{"x": w["x"], "o": w["o"]} for _ in range(2)]
        args[0][name] = w[name] + step * r
        args[1][name] = w[name] - step * r
        diff = (loss(**args[0])[1] - loss(**args[1])[1]) / (2 * step)
        want = (grad.double() * r.double()).sum().item()
        assert abs(diff - want) < 2 ** -8 * grad.double().norm().item() + 2 ** -22 * (2 * T * D) ** 0.5 / step


# ---------------------------------------------------------------------------
# Dropout
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,D", [(1, 1), (3, 7), (5, 8), (17, 501), (64, 2048), (1000, 9), (2, 100003)])
@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_dropout(T, D, dtype, p):
    g = torch.Generator().manual_seed(T + D)
    x, r = rand(g, T, D, dtype=dtype), rand(g, T, D, dtype=dtype)
    seed, step = 0xFEDCBA9876543210, (1 << 62) + 12345
    for res in (r, None):
        y = nan(T, D, dtype=dtype)
        api.rar_dropout(T, D, CODE[dtype], dev(x), y, p, seed, step=torch.tensor([step], device=DEV), residual=dev(res))
        R.check(y, *R.dropout(x, res, p, seed, step, dtype), "y")
    y = nan(T, D, dtype=dtype)
    api.rar_dropout(T, D, CODE[dtype], dev(x), y, p, 5)
    R.check(y, *R.dropout(x, None, p, 5, 0, dtype), "y at step 0")


@pytest.mark.parametrize("dtype", BOTH)
def test_dropout_edges(dtype):
    T, D = 70, 203
    g = torch.Generator().manual_seed(1)
    x = rand(g, T, D, dtype=dtype)
    y = nan(T, D, dtype=dtype)
    api.rar_dropout(T, D, CODE[dtype], dev(x), y, 0.0, 9)
    assert same_bits(y, dev(x))
    api.rar_dropout(T, D, CODE[dtype], dev(x), y, 1.0, 9)
    assert (y == 0).all()
    # a dropped element counts as zero whatever it holds; kept ones propagate
    keep, scale = R.keep_mask(T, D, 0.25, 9, -1)
    bad = torch.full((T, D), NAN, dtype=R.DT[dtype])
    step = torch.tensor([-1], device=DEV)
    api.rar_dropout(T, D, CODE[dtype], dev(bad), y, 0.25, 9, step=step)
    assert (torch.isnan(y.cpu()) == keep).all() and (y.cpu()[~keep] == 0).all()
    # views, in place over x and over the residual; the mask follows from the place in the matrix, not the memory
    want, bound = R.dropout(x, None, 0.25, 9, -1, dtype)
    v = strided(x, 5, 3)
    api.rar_dropout(T, D, CODE[dtype], v, v, 0.25, 9, step=step)
    R.check(v, want, bound, "over x")
    around_is_untouched(v)
    r = rand(g, T, D, dtype=dtype)
    rv = strided(r, 5, 3)
    api.rar_dropout(T, D, CODE[dtype], dev(x), rv, 0.25, 9, step=step, residual=rv)
    R.check(rv, *R.dropout(x, r, 0.25, 9, -1, dtype), "over the residual")
    around_is_untouched(rv)
    e = torch.empty(0, D, dtype=R.DT[dtype], device=DEV)
    api.rar_dropout(0, D, CODE[dtype], e, e, 0.5, 1)


def test_dropout_numbers_pass_32_bits():
    # groups of eight are numbered past 2^32: the first and the last rows against the definition, in place
    T, D, p, seed, last = 1 << 24, 2056, 0.25, 99, 3
    x = torch.empty(T, D, dtype=torch.bfloat16, device=DEV)
    x.fill_(1.0)
    api.rar_dropout(T, D, api.BF16, x, x, p, seed)
    first = (T - last) * (D // 8)
    assert first > 1 << 32
    assert torch.equal(x[T - last:].cpu() != 0, R.keep_mask(last, D, p, seed, 0, first)[0])
    assert torch.equal(x[:last].cpu() != 0, R.keep_mask(last, D, p, seed, 0)[0])
    del x
    torch.cuda.empty_cache()


def test_dropout_step_is_read_in_every_replay():
    T, D, p, seed = 33, 100, 0.3, 77
    x = torch.randn(T, D, device=DEV)
    y, step = torch.empty_like(x), torch.zeros(1, dtype=torch.int64, device=DEV)
    api.rar_dropout(T, D, api.F32, x, y, p, seed, step=step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        api.rar_dropout(T, D, api.F32, x, y, p, seed, step=step)
    step.zero_()
    for n in range(1, 4):
        graph.replay()
        R.check(y, *R.dropout(x.cpu(), None, p, seed, n, "f32"), f"replay {n}")
        x.normal_()
        torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# Cross attention
# ---------------------------------------------------------------------------

# (B, Tq, Tk, H, Hkv, dh): one of everything, few rows, whole and broken tiles of queries and keys, shared heads,
# widths in each class and between, split keys
ATTN = [(1, 1, 1, 1, 1, 1), (1, 1, 5, 1, 1, 16), (2, 1, 300, 4, 2, 64), (3, 7, 129, 3, 1, 40), (2, 5, 1000, 8, 1, 128),
        (1, 32, 33, 1, 1, 96), (1, 33, 64, 2, 2, 32), (2, 130, 70, 2, 1, 60), (1, 257, 300, 4, 2, 128),
        (2, 64, 128, 6, 3, 77), (1, 1, 4100, 2, 1, 128), (5, 3, 65, 1, 1, 100), (2, 200, 31, 2, 2, 127),
        (1, 700, 20, 2, 1, 8), (3, 96, 257, 4, 4, 33)]


def attn_inputs(g, B, Tq, Tk, H, Hkv, dh, dtype, scale=1.0):
    return (rand(g, B * Tq, H * dh, dtype=dtype, scale=scale), rand(g, B * Tk, Hkv * dh, dtype=dtype, scale=scale),
            rand(g, B * Tk, Hkv * dh, dtype=dtype), rand(g, B * Tq, H * dh, dtype=dtype))


def lengths(g, B, most, ragged):
    if not ragged:
        return None
    n = torch.randint(0, most + 1, (B,), generator=g)
    n[0] = most
    return n


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("shape", ATTN, ids=str)
@pytest.mark.parametrize("dtype", BOTH)
def test_attention(shape, dtype, ragged):
    B, Tq, Tk, H, Hkv, dh = shape
    g = torch.Generator().manual_seed(sum(shape))
    q, k, v, do = attn_inputs(g, *shape, dtype)
    ql, kl = lengths(g, B, Tq, ragged), lengths(g, B, Tk, ragged)
    scale = dh ** -0.5
    plan = api.rar_attn_plan(H, Hkv, dh, CODE[dtype])
    o, lse = nan(B * Tq, H * dh, dtype=dtype), nan(B * Tq, H, dtype="f32")
    api.rar_attn_forward(plan, B, Tq, Tk, dev(q), dev(k), dev(v), o, lse=lse, qlen=dev(ql), klen=dev(kl))
    (ro, eo), (rl, el) = R.attn_forward(q, k, v, B, H, Hkv, scale, ql, kl, dtype)
    R.check(o, ro, eo, "o")
    gone = rl == -INF
    assert (lse.cpu()[gone] == -INF).all()
    R.check(torch.where(gone, 0.0, lse.cpu()), torch.where(gone, 0.0, rl), el, "lse")
    o2 = nan(B * Tq, H * dh, dtype=dtype)
    api.rar_attn_forward(plan, B, Tq, Tk, dev(q), dev(k), dev(v), o2, qlen=dev(ql), klen=dev(kl))
    assert same_bits(o, o2)
    dq, dk, dv = (torch.full_like(dev(t), NAN) for t in (q, k, v))
    api.rar_attn_backward(plan, B, Tq, Tk, dev(do), dev(q), dev(k), dev(v), o, lse, dq, dk, dv, qlen=dev(ql),
                          klen=dev(kl))
    want = R.attn_backward(do, q, k, v, o.cpu(), lse.cpu(), B, H, Hkv, scale, ql, kl, dtype)
    for t, (r, e), n in zip((dq, dk, dv), want, ("dq", "dk", "dv")):
        R.check(t, r, e, n)
    for keep in range(3):    # one gradient alone
        out = [torch.full_like(t, NAN) if i == keep else None for i, t in enumerate((dq, dk, dv))]
        api.rar_attn_backward(plan, B, Tq, Tk, dev(do), dev(q), dev(k), dev(v), o, lse, *out, qlen=dev(ql),
                              klen=dev(kl))
        assert same_bits(out[keep], (dq, dk, dv)[keep])


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("extra,offset", [(8, 0), (8, 8), (3, 1), (16, 4)])
@pytest.mark.parametrize("Tq", [3, 150])
def test_attention_strides_and_padding(Tq, extra, offset, dtype):
    # every matrix a view with NaN around it, NaN in the rows that do not count, lengths outside their range
    B, Tk, H, Hkv, dh = 3, 140, 4, 2, 24
    g = torch.Generator().manual_seed(6)
    q, k, v, do = attn_inputs(g, B, Tq, Tk, H, Hkv, dh, dtype)
    ql, kl = torch.tensor([Tq + 5, 2, 1]), torch.tensor([77, 1 << 40, -3])
    for m, n, lens in ((q, Tq, ql), (do, Tq, ql), (k, Tk, kl), (v, Tk, kl)):
        for b in range(B):
            m.view(B, n, -1)[b, max(0, min(n, int(lens[b]))):] = NAN
    sq, sk, sv, sdo = (strided(t, extra, offset) for t in (q, k, v, do))
    zero = lambda t: strided(torch.zeros_like(t), extra, offset)  # noqa: E731
    o, lse = zero(q), nan(B * Tq, H, dtype="f32")
    plan = api.rar_attn_plan(H, Hkv, dh, CODE[dtype], 0.3)
    api.rar_attn_forward(plan, B, Tq, Tk, sq, sk, sv, o, lse=lse, qlen=dev(ql), klen=dev(kl))
    (ro, eo), (rl, _) = R.attn_forward(q, k, v, B, H, Hkv, 0.3, ql, kl, dtype)
    R.check(o, ro, eo, "o")
    assert ((lse.cpu() == -INF) == (rl == -INF)).all()
    dq, dk, dv = zero(q), zero(k), zero(v)
    api.rar_attn_backward(plan, B, Tq, Tk, sdo, sq, sk, sv, o, lse, dq, dk, dv, qlen=dev(ql), klen=dev(kl))
    want = R.attn_backward(do, q, k, v, o.cpu(), lse.cpu(), B, H, Hkv, 0.3, ql, kl, dtype)
    for t, (r, e), n in zip((dq, dk, dv), want, ("dq", "dk", "dv")):
        R.check(t, r, e, n)
    for t in (o, dq, dk, dv):
        around_is_untouched(t)


@pytest.mark.parametrize("dtype", BOTH)
def test_attention_keys_and_values_side_by_side(dtype):
    # one projection's output holds keys and values; their gradients go into one matrix too
    B, Tq, Tk, H, dh = 2, 40, 90, 2, 64
    g = torch.Generator().manual_seed(7)
    q, k, v, do = attn_inputs(g, B, Tq, Tk, H, H, dh, dtype)
    both = torch.cat([k, v], 1).to(DEV)
    ks, vs = both[:, :H * dh], both[:, H * dh:]
    plan = api.rar_attn_plan(H, H, dh, CODE[dtype])
    o, lse = nan(B * Tq, H * dh, dtype=dtype), nan(B * Tq, H, dtype="f32")
    api.rar_attn_forward(plan, B, Tq, Tk, dev(q), ks, vs, o, lse=lse)
    grads = torch.full_like(both, NAN)
    dq = nan(B * Tq, H * dh, dtype=dtype)
    api.rar_attn_backward(plan, B, Tq, Tk, dev(do), dev(q), ks, vs, o, lse, dq, grads[:, :H * dh], grads[:, H * dh:])
    want = R.attn_backward(do, q, k, v, o.cpu(), lse.cpu(), B, H, H, dh ** -0.5, None, None, dtype)
    for t, (r, e), n in zip((dq, grads[:, :H * dh], grads[:, H * dh:]), want, ("dq", "dk", "dv")):
        R.check(t, r, e, n)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("Tq", [2, 70])
def test_attention_without_queries_or_keys(Tq, dtype):
    H, dh = 2, 16
    plan = api.rar_attn_plan(H, H, dh, CODE[dtype])
    q, do = (torch.randn(Tq, H * dh, device=DEV).to(R.DT[dtype]) for _ in range(2))
    e = torch.empty(0, H * dh, dtype=R.DT[dtype], device=DEV)
    o, lse = nan(Tq, H * dh, dtype=dtype), nan(Tq, H, dtype="f32")
    api.rar_attn_forward(plan, 1, Tq, 0, q, e, e, o, lse=lse)
    assert (o == 0).all() and (lse == -INF).all()
    dq = nan(Tq, H * dh, dtype=dtype)
    api.rar_attn_backward(plan, 1, Tq, 0, do, q, e, e, o, lse, dq, e.clone(), e.clone())
    assert (dq == 0).all()
    api.rar_attn_forward(plan, 1, 0, Tq, e, q, q, e.clone())
    dk, dv = nan(Tq, H * dh, dtype=dtype), nan(Tq, H * dh, dtype=dtype)
    api.rar_attn_backward(plan, 1, 0, Tq, e, e, q, q, e, lse[:0], e.clone(), dk, dv)
    assert (dk == 0).all() and (dv == 0).all()


@pytest.mark.parametrize("Tq", [2, 40])
def test_attention_large_and_infinite_scores(Tq):
    B, Tk, H, dh = 1, 200, 1, 32
    g = torch.Generator().manual_seed(9)
    for dtype in BOTH:
        # scores up to some hundreds: the softmax is nearly one key's, and nothing overflows
        q, k, v, do = attn_inputs(g, B, Tq, Tk, H, H, dh, dtype, scale=6.0)
        plan = api.rar_attn_plan(H, H, dh, CODE[dtype], 1.0)
        o, lse = nan(Tq, dh, dtype=dtype), nan(Tq, 1, dtype="f32")
        api.rar_attn_forward(plan, B, Tq, Tk, dev(q), dev(k), dev(v), o, lse=lse)
        (ro, eo), (rl, el) = R.attn_forward(q, k, v, B, H, H, 1.0, None, None, dtype)
        R.check(o, ro, eo, "o")
        R.check(lse, rl, el, "lse")
        # a key whose score is -infinity has no weight; every score -infinity leaves nothing; NaN stays in its row
        q = torch.ones(Tq, dh, dtype=R.DT[dtype])
        k2 = k.abs()
        k2[5] = -INF
        api.rar_attn_forward(plan, B, Tq, Tk, dev(q), dev(k2), dev(v), o, lse=lse)
        rest = torch.arange(Tk) != 5
        (ro, eo), _ = R.attn_forward(q, k2[rest], v[rest], B, H, H, 1.0, None, None, dtype)
        R.check(o, ro, eo, "o with a masked key")
        api.rar_attn_forward(plan, B, Tq, Tk, dev(q), torch.full_like(dev(k), -INF), dev(v), o, lse=lse)
        assert (o == 0).all() and (lse == -INF).all()
        dq, dk, dv = nan(Tq, dh, dtype=dtype), torch.full_like(dev(k), NAN), torch.full_like(dev(k), NAN)
        q = rand(g, Tq, dh, dtype=dtype)
        q[1] = NAN
        api.rar_attn_forward(plan, B, Tq, Tk, dev(q), dev(k), dev(v), o, lse=lse)
        bad = torch.isnan(o).all(1)
        assert bad[1] and bad.sum() == 1 and not torch.isnan(o[~bad]).any()


@pytest.mark.parametrize("dtype", BOTH)
def test_attention_long_cache(dtype):
    # keys whose offsets pass 2^31 elements; the last sequence is the one that is looked at
    B, Tk, ld = 3, 1 << 18, 1 << 12
    big = torch.zeros(B * Tk, ld, dtype=R.DT[dtype], device=DEV)
    H, dh, n = 2, 64, 300
    g = torch.Generator().manual_seed(10)
    q, k, v, do = attn_inputs(g, 1, 2, n, H, H, dh, dtype)
    ks, vs = big[:, :H * dh], big[:, ld - H * dh:]
    ks[2 * Tk:2 * Tk + n], vs[2 * Tk:2 * Tk + n] = dev(k), dev(v)
    q3, do3 = dev(q).repeat(B, 1), dev(do).repeat(B, 1)
    kl = torch.tensor([0, 1, n])
    plan = api.rar_attn_plan(H, H, dh, CODE[dtype])
    o, lse = nan(2 * B, H * dh, dtype=dtype), nan(2 * B, H, dtype="f32")
    api.rar_attn_forward(plan, B, 2, Tk, q3, ks, vs, o, lse=lse, klen=dev(kl))
    (ro, eo), _ = R.attn_forward(q, k, v, 1, H, H, dh ** -0.5, None, None, dtype)
    R.check(o[4:], ro, eo, "o")
    assert (o[:2] == 0).all()
    dq = nan(2 * B, H * dh, dtype=dtype)
    api.rar_attn_backward(plan, B, 2, Tk, do3, q3, ks, vs, o, lse, dq, None, None, klen=dev(kl))
    want = R.attn_backward(do, q, k, v, o[4:].cpu(), lse[4:].cpu(), 1, H, H, dh ** -0.5, None, None, dtype)
    R.check(dq[4:], *want[0], "dq")


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("Tq", [2, 10, 130])
def test_attention_rows_as_far_apart_as_allowed(Tq, dtype):
    # leading dimension 2^22: a tile's last row lies almost 2^31 bytes behind its first; all matrices in one
    Tk, H, Hkv, dh, ld = 140, 2, 1, 128, 1 << 22
    g = torch.Generator().manual_seed(12)
    q, k, v, do = attn_inputs(g, 1, Tq, Tk, H, Hkv, dh, dtype)
    big = torch.full((Tk, ld), NAN, dtype=R.DT[dtype], device=DEV)
    at = iter(range(ld - 8 * 256, ld, 256))

    def inside(rows, cols, t=None):
        c = next(at)
        m = big[:rows, c:c + cols]
        return m if t is None else m.copy_(dev(t))

    sq, sdo, sk, sv = inside(Tq, H * dh, q), inside(Tq, H * dh, do), inside(Tk, dh, k), inside(Tk, dh, v)
    o, dq, dk, dv = inside(Tq, H * dh), inside(Tq, H * dh), inside(Tk, dh), inside(Tk, dh)
    lse = nan(Tq, H, dtype="f32")
    plan = api.rar_attn_plan(H, Hkv, dh, CODE[dtype])
    api.rar_attn_forward(plan, 1, Tq, Tk, sq, sk, sv, o, lse=lse)
    (ro, eo), _ = R.attn_forward(q, k, v, 1, H, Hkv, dh ** -0.5, None, None, dtype)
    R.check(o, ro, eo, "o")
    api.rar_attn_backward(plan, 1, Tq, Tk, sdo, sq, sk, sv, o, lse, dq, dk, dv)
    want = R.attn_backward(do, q, k, v, o.cpu(), lse.cpu(), 1, H, Hkv, dh ** -0.5, None, None, dtype)
    for t, (r, e), n in zip((dq, dk, dv), want, ("dq", "dk", "dv")):
        R.check(t, r, e, n)


def test_attention_gradient_against_differences():
    B, Tq, Tk, H, Hkv, dh = 2, 5, 9, 2, 1, 12
    g = torch.Generator().manual_seed(11)
    m = dict(zip("qkvg", (dev(t) for t in attn_inputs(g, B, Tq, Tk, H, Hkv, dh, "f32"))))
    kl = torch.tensor([9, 4], device=DEV)
    plan = api.rar_attn_plan(H, Hkv, dh, api.F32)

    def run(q, k, v, g):
        o, lse = torch.empty_like(q), torch.empty(B * Tq, H, device=DEV)
        api.rar_attn_forward(plan, B, Tq, Tk, q, k, v, o, lse=lse, klen=kl)
        return o, lse, (o.double() * g.double()).sum().item()

    o, lse, _ = run(**m)
    grads = [torch.empty_like(m[n]) for n in "qkv"]
    api.rar_attn_backward(plan, B, Tq, Tk, m["g"], m["q"], m["k"], m["v"], o, lse, *grads, klen=kl)
    # as for the norms: the loss is known to 2^-22 sqrt(n) of its terms, the third derivative gives 2^-12
    for n, grad in zip("qkv", grads):
        r = torch.randn(m[n].shape, generator=g).to(DEV)
        r /= r.norm()
        step = 2.0 ** -6
        diff = (run(**{**m, n: m[n] + step * r})[2] - run(**{**m, n: m[n] - step * r})[2]) / (2 * step)
        want = (grad.double() * r.double()).sum().item()
        assert abs(diff - want) < 2 ** -8 * grad.double().norm().item() + 2 ** -22 * (B * Tq * H * dh) ** 0.5 / step


# ---------------------------------------------------------------------------
# Log probabilities
# ---------------------------------------------------------------------------

# (T, V): one element, widths at and around what a wave, a workgroup and registers take, and beyond
LOGPROB = [(1, 1), (3, 2), (5, 33), (7, 500), (9, 2048), (6, 2049), (4, 8192), (3, 8195), (5, 32000), (2, 32769),
           (3, 65536), (2, 65537), (2, 131_072), (1, 200_003), (300, 40), (2100, 64), (515, 16001), (600, 32001),
           (520, 20_011), (3, 40_009)]


def logits(g, T, V, dtype):
    z = torch.randn(T, V, generator=g) * 3
    z[:, 0] += 5
    return z.to(R.DT[dtype])


@pytest.mark.parametrize("shape", LOGPROB, ids=str)
@pytest.mark.parametrize("dtype", BOTH)
def test_logprob(shape, dtype):
    T, V = shape
    g = torch.Generator().manual_seed(T + V)
    z = logits(g, T, V, dtype)
    t = torch.randint(-1, V + 1, (T,), generator=g)
    t[0] = V - 1
    for K, scale in ((8, 1.0), (32, 0.7), (1, 1.0)):
        logp, ent = nan(T, dtype="f32"), nan(T, dtype="f32")
        ids, top = torch.full((T, K), -7, device=DEV), nan(T, K, dtype="f32")
        api.rar_logprob(T, V, CODE[dtype], dev(z), dev(t), logp, ent, top_ids=ids, top_logp=top, scale=scale)
        s = float(torch.tensor(scale))
        (rl, el), (re, ee) = R.logprob(z, t, s)
        R.check(logp, rl, el, "logp")
        R.check(ent, re, ee, "entropy")
        if T <= 300:
            ri, rt, et = R.top(z, s, K)
            assert (ids.cpu() == ri).all()
            on = ri >= 0
            assert (top.cpu()[~on] == -INF).all()
            R.check(torch.where(on, top.cpu(), 0.0), torch.where(on, rt, 0.0), et, "alternatives")
    logp2 = nan(T, dtype="f32")
    api.rar_logprob(T, V, CODE[dtype], dev(z), dev(t), logp2)
    assert same_bits(logp, logp2)


@pytest.mark.parametrize("shape", LOGPROB, ids=str)
@pytest.mark.parametrize("dtype", BOTH)
def test_logprob_gradient(shape, dtype):
    T, V = shape
    g = torch.Generator().manual_seed(T * 3 + V)
    z = logits(g, T, V, dtype)
    t = torch.randint(-1, V + 1, (T,), generator=g)
    t[0] = V - 1
    dl, de = torch.randn(T, generator=g), torch.randn(T, generator=g)
    dl[t < 0] = NAN                                   # padding: not looked at
    for a, b, scale in ((dl, de, 1.0), (dl, None, 0.7), (None, de, 1.0)):
        s = float(torch.tensor(scale))
        dz, logp, ent = nan(T, V, dtype=dtype), nan(T, dtype="f32"), nan(T, dtype="f32")
        api.rar_logprob_grad(T, V, CODE[dtype], dev(z), dev(t) if a is not None else None, dev(a), dev(b), dz,
                             logp=logp if a is not None else None, entropy=ent, scale=scale)
        R.check(dz, *R.logprob_grad(z, t if a is not None else None, a, b, s, dtype), "dz")
        (rl, el), (re, ee) = R.logprob(z, t, s)
        if a is not None:
            R.check(logp, rl, el, "logp")
        R.check(ent, re, ee, "entropy")
        over = dev(z)                                 # dz over the logits
        api.rar_logprob_grad(T, V, CODE[dtype], over, dev(t), dev(a), dev(b), over, scale=scale)
        assert torch.equal(over, dz)                  # (without targets a zero may have the other sign)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("V", [300, 5000, 30001, 70000, 140_000])
def test_logprob_ties_masks_and_bad_values(V, dtype):
    T, K = 10, 20
    g = torch.Generator().manual_seed(V)
    z = torch.randn(T, V, generator=g).to(R.DT[dtype])
    z[0] = 1.5                                        # all alike
    z[1] = torch.arange(V).float().to(z.dtype)        # rising (in bf16 with long runs of ties)
    z[2] = -torch.arange(V).float().to(z.dtype)
    z[3] = -INF
    z[3, 7], z[3, V - 1] = 0.0, -0.0                  # two are left, and they tie
    z[4] = -INF                                       # nothing is left
    z[5, ::2] = torch.finfo(z.dtype).min
    z[6, 1::3] = -INF
    z[7] = (z[7] * 4).round().clamp(-1, 1)            # three values
    z[8, 3] = NAN
    z[9, 4] = INF
    t = torch.tensor([0, V - 1, 5, 7, 2, 0, 1, 9, 3, 4])
    t6 = int(t[6])
    logp, ent = nan(T, dtype="f32"), nan(T, dtype="f32")
    ids, top = torch.full((T, K), -7, device=DEV), nan(T, K, dtype="f32")
    api.rar_logprob(T, V, CODE[dtype], dev(z), dev(t), logp, ent, top_ids=ids, top_logp=top)
    ri, rt, et = R.top(z[:8], 1.0, K)
    assert (ids.cpu()[:8] == ri).all()
    on = ri >= 0
    assert (top.cpu()[:8][~on] == -INF).all()
    R.check(torch.where(on, top.cpu()[:8], 0.0), torch.where(on, rt, 0.0), et, "alternatives")
    assert (ids[8:] == -1).all() and torch.isnan(top[8:]).all()
    assert torch.isnan(logp[8:]).all() and torch.isnan(ent[8:]).all()
    assert logp[4] == -INF and ent[4] == 0
    assert z[6, t6] == -INF and logp[6] == -INF
    rows = torch.tensor([0, 1, 2, 3, 5, 7])
    (rl, el), (re, ee) = R.logprob(z[rows], t[rows], 1.0)
    R.check(logp.cpu()[rows], rl, el, "logp")
    R.check(ent.cpu()[rows], re, ee, "entropy")
    dl, de = torch.randn(T, generator=g), torch.randn(T, generator=g)
    dz = nan(T, V, dtype=dtype)
    api.rar_logprob_grad(T, V, CODE[dtype], dev(z), dev(t), dev(dl), dev(de), dz)
    assert (dz[4] == 0).all() and torch.isnan(dz[8:]).all()
    rows = torch.tensor([0, 1, 2, 3, 5, 6, 7])
    want, bound = R.logprob_grad(z[rows], t[rows], dl[rows], de[rows], 1.0, dtype)
    R.check(dz.cpu()[rows], want, bound, "dz")


@pytest.mark.parametrize("dtype", BOTH)
def test_logprob_views_and_far_rows(dtype):
    # rows whose offsets pass 2^31 elements, NaN between them
    T, V, ld = 70000, 250, 32003
    big = torch.full((T, ld), NAN, dtype=R.DT[dtype], device=DEV)
    g = torch.Generator().manual_seed(12)
    n = 40
    z = logits(g, n, V, dtype)
    view = big[:, 5:5 + V]
    view.zero_()
    view[T - n:] = dev(z)
    t = torch.zeros(T, dtype=torch.int64)
    t[T - n:] = torch.randint(0, V, (n,), generator=g)
    dl = torch.randn(T, generator=g)
    logp, ent = nan(T, dtype="f32"), nan(T, dtype="f32")
    api.rar_logprob_grad(T, V, CODE[dtype], view, dev(t), dev(dl), None, view, logp=logp, entropy=ent)
    want, bound = R.logprob_grad(z, t[T - n:], dl[T - n:], None, 1.0, dtype)
    R.check(view[T - n:], want, bound, "dz")
    assert torch.isnan(big[:, :5].float()).all() and torch.isnan(big[:, 5 + V:].float()).all()
    (rl, el), _ = R.logprob(z, t[T - n:], 1.0)
    R.check(logp[T - n:], rl, el, "logp")


# ---------------------------------------------------------------------------
# Streams, graphs, repeatability
# ---------------------------------------------------------------------------

def everything(dtype):
    """Every operator once on fixed inputs; returns a function that runs them and its outputs."""
    g = torch.Generator().manual_seed(20)
    T, D, V = 300, 520, 1003
    dt = R.DT[dtype]
    new = lambda *s, t=dt: torch.full(s, NAN if t.is_floating_point else -7, dtype=t, device=DEV)  # noqa: E731
    x, o, dh, du = (rand(g, T, D, dtype=dtype).to(DEV) for _ in range(4))
    w = rand(g, D, dtype=dtype).to(DEV)
    norm = api.rar_norm_plan(D, CODE[dtype], api.NORM_LAYER, api.NORM_RMS)
    B, Tq, Tk, H, dh_ = 3, 100, 260, 4, 130 // 2
    attn = api.rar_attn_plan(H, 2, dh_, CODE[dtype])
    q, k, v, do = (t.to(DEV) for t in attn_inputs(g, B, Tq, Tk, H, 2, dh_, dtype))
    kl = torch.tensor([260, 3, 100], device=DEV)
    z, t = logits(g, T, V, dtype).to(DEV), torch.randint(0, V, (T,), generator=g).to(DEV)
    dl = torch.randn(T, generator=g).to(DEV)
    out = dict(h=new(T, D), u=new(T, D), dx=new(T, D), do=new(T, D), dw=new(D), y=new(T, D), o=new(B * Tq, H * dh_),
               lse=new(B * Tq, H, t=torch.float32), dq=new(B * Tq, H * dh_), dk=new(*k.shape), dv=new(*v.shape),
               o1=new(B, H * dh_), logp=new(T, t=torch.float32), ids=new(T, 5, t=torch.int64),
               top=new(T, 5, t=torch.float32), dz=new(T, V))
    sizes = [api.rar_norm_workspace(norm, T), *api.rar_attn_workspace(attn, B, Tq, Tk),
             api.rar_attn_workspace(attn, B, 1, Tk)[0]]
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]

    def run(stream=None, own=True):
        a = ws if own else [None] * 4
        api.rar_norm_forward(norm, T, x, o, w, w, w, w, None, out["h"], out["u"], stream=stream)
        api.rar_norm_backward(norm, T, dh, du, o, out["h"], w, w, w, w, out["dx"], out["do"], dpre_w=out["dw"], ws=a[0],
                              stream=stream)
        api.rar_dropout(T, D, CODE[dtype], out["u"], out["y"], 0.2, 3, residual=out["h"], stream=stream)
        api.rar_attn_forward(attn, B, Tq, Tk, q, k, v, out["o"], lse=out["lse"], klen=kl, ws=a[1], stream=stream)
        api.rar_attn_backward(attn, B, Tq, Tk, do, q, k, v, out["o"], out["lse"], out["dq"], out["dk"], out["dv"],
                              klen=kl, ws=a[2], stream=stream)
        api.rar_attn_forward(attn, B, 1, Tk, q[:B], k, v, out["o1"], klen=kl, ws=a[3], stream=stream)
        api.rar_logprob(T, V, CODE[dtype], z, t, out["logp"], top_ids=out["ids"], top_logp=out["top"], stream=stream)
        api.rar_logprob_grad(T, V, CODE[dtype], z, t, dl, None, out["dz"], stream=stream)

    return run, out


@pytest.mark.parametrize("dtype", BOTH)
def test_runs_repeat_on_streams_and_in_graphs(dtype):
    run, out = everything(dtype)
    run()
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in out.items()}

    def clear():
        for t in out.values():
            t.fill_(5)

    def compare(what):
        torch.cuda.synchronize()
        for n, t in out.items():
            assert same_bits(t, want[n]), f"{n} {what}"

    clear()
    run(own=False)
    compare("again, workspaces of the binding's")
    clear()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run(stream=s, own=False)
    compare("on a stream given")
    clear()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        run()
    compare("on torch's current stream")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for n in range(3):
        clear()
        torch.cuda.synchronize()
        graph.replay()
        compare(f"in replay {n}")
        run()
        compare(f"eagerly behind replay {n}")


@pytest.mark.parametrize("dtype", BOTH)
def test_two_streams_at_once(dtype):
    # plans are shared, workspaces are not
    run_a, a = everything(dtype)
    run_b, b = everything(dtype)
    run_a()
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in a.items()}
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        run_a(stream=s1)
        run_b(stream=s2)
    torch.cuda.synchronize()
    for n in want:
        assert same_bits(a[n], want[n]) and same_bits(b[n], want[n]), n
