"""The embedding, the linear layer and 8-bit checkpoints on the GPU, against
plain 64-bit forms at the sizes, layouts and values where they can go wrong.
Bounds count roundings (see ops_ref.py); nothing is fitted to results."""
import ctypes

import numpy as np
import pytest
import torch

import ops_ref as R
from ring_all_reduce_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CODE = {"f32": api.F32, "bf16": api.BF16}
BOTH = ["f32", "bf16"]


def rand(gen, *shape, dtype="f32", scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(R.DT[dtype])


def nan_like(*shape, dtype):
    return torch.full(shape, float("nan"), dtype=R.DT[dtype], device=DEV)


def strided(t, extra, offset=0):
    """t on the GPU as a view of a wider matrix (rows t.shape[1] + extra apart), NaN around it."""
    big = torch.full((t.shape[0] + 1, t.shape[1] + extra), float("nan"), dtype=t.dtype, device=DEV)
    v = big[:t.shape[0], offset:offset + t.shape[1]]
    v.copy_(t.to(DEV))
    return v


# ---------------------------------------------------------------------------
# Linear layer
# ---------------------------------------------------------------------------

# (T, K, N): one element, one token, odd sizes, whole and broken tiles, split reductions, more than 192 tiles of 256
SHAPES = [(1, 1, 1), (1, 8, 8), (3, 5, 7), (17, 64, 32), (1, 2048, 520), (7, 300, 1000), (129, 257, 131),
          (300, 512, 264), (64, 1000, 72), (515, 96, 640), (5001, 40, 24), (130, 8, 4096),
          (2, 2056, 72), (4, 1000, 136), (3, 4104, 200)]
BIG = [(3000, 72, 4200), (2900, 136, 4104)]


LINEAR = [(s, dt, a) for s in SHAPES for dt in BOTH for a in R.ACTS]
LINEAR += [(s, "bf16", a) for s in BIG for a in ("none", "gelu")]


@pytest.mark.parametrize("shape,dtype,act", LINEAR, ids=str)
def test_linear_forward(shape, dtype, act):
    T, K, N = shape
    g = torch.Generator().manual_seed(T * 31 + K + N)
    x, w = rand(g, T, K, dtype=dtype), rand(g, K, N, dtype=dtype, scale=K ** -0.5)
    b, r = rand(g, N, dtype=dtype), rand(g, T, N, dtype=dtype)
    plan = api.rar_linear_plan(K, N, CODE[dtype], R.ACTS[act])
    for bias, res in ((b, r), (None, None)) if shape not in BIG else ((b, r),):
        y, z = nan_like(T, N, dtype=dtype), nan_like(T, N, dtype=dtype)
        api.rar_linear_forward(plan, T, x.to(DEV), w.to(DEV), None if bias is None else bias.to(DEV),
                               None if res is None else res.to(DEV), y, pre=z)
        (ry, ey), (rz, ez) = R.forward(x, w, bias, res, act, dtype)
        R.check(z, rz, ez, "z")
        R.check(y, ry, ey, "y")


@pytest.mark.parametrize("shape,dtype,act", LINEAR, ids=str)
def test_linear_backward(shape, dtype, act):
    T, K, N = shape
    g = torch.Generator().manual_seed(T * 37 + K + N)
    dy, x, z = (rand(g, T, n, dtype=dtype) for n in (N, K, N))
    w = rand(g, K, N, dtype=dtype, scale=K ** -0.5)
    dw0, db0 = rand(g, K, N, dtype=dtype), rand(g, N, dtype=dtype)
    plan = api.rar_linear_plan(K, N, CODE[dtype], R.ACTS[act])
    for acc in (False, True):
        dx = nan_like(T, K, dtype=dtype)
        dw = dw0.to(DEV) if acc else nan_like(K, N, dtype=dtype)
        db = db0.to(DEV) if acc else nan_like(N, dtype=dtype)
        api.rar_linear_backward(plan, T, dy.to(DEV), x.to(DEV), w.to(DEV), z.to(DEV), dx, dw, db, accumulate=acc)
        ref = R.backward(dy, x, w, z, act, dtype, *((dw0, db0) if acc else ()))
        for got, (want, bound), what in zip((dx, dw, db), ref, ("dx", "dw", "db")):
            R.check(got, want, bound, f"{what} accumulate={acc}")


@pytest.mark.parametrize("dtype", BOTH)
def test_big_dw_tiles(dtype):
    # more than 192 tiles of 256 in K x N, and a reduction over few and odd rows
    T, K, N = 67, 3400, 4104
    g = torch.Generator().manual_seed(5)
    dy, x = rand(g, T, N, dtype=dtype), rand(g, T, K, dtype=dtype)
    plan = api.rar_linear_plan(K, N, CODE[dtype], api.ACT_NONE)
    dw = nan_like(K, N, dtype=dtype)
    api.rar_linear_backward(plan, T, dy.to(DEV), x.to(DEV), None, None, None, dw, None)
    want, bound = R.backward(dy, x, torch.zeros(K, N), torch.zeros(T, N), "none", dtype)[1]
    R.check(dw, want, bound, "dw")


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("extra,offset", [(8, 0), (8, 8), (3, 1), (1, 0)])
def test_linear_strides_and_surroundings(dtype, extra, offset):
    # every matrix a view of a wider one with NaN around it: nothing outside is read into a result or written
    T, K, N = 150, 136, 200
    g = torch.Generator().manual_seed(11)
    x, r, dy, z0 = (rand(g, T, n, dtype=dtype) for n in (K, N, N, N))
    w, b = rand(g, K, N, dtype=dtype, scale=0.1), rand(g, N, dtype=dtype)
    plan = api.rar_linear_plan(K, N, CODE[dtype], api.ACT_GELU)
    xs, rs, dys, zs = (strided(t, extra, offset) for t in (x, r, dy, z0))
    y, z, dx = (strided(torch.zeros(T, n, dtype=R.DT[dtype]), extra, offset) for n in (N, N, K))
    api.rar_linear_forward(plan, T, xs, w.to(DEV), b.to(DEV), rs, y, pre=z)
    (ry, ey), (rz, ez) = R.forward(x, w, b, r, "gelu", dtype)
    R.check(y, ry, ey, "y")
    R.check(z, rz, ez, "z")
    dw, db = nan_like(K, N, dtype=dtype), nan_like(N, dtype=dtype)
    api.rar_linear_backward(plan, T, dys, xs, w.to(DEV), zs, dx, dw, db)
    for got, (want, bound), what in zip((dx, dw, db), R.backward(dy, x, w, z0, "gelu", dtype), ("dx", "dw", "db")):
        R.check(got, want, bound, what)
    for view in (y, z, dx):
        cols = view.shape[1]
        base = view._base
        outside = torch.ones_like(base, dtype=torch.bool)
        outside[:T, offset:offset + cols] = False
        assert torch.isnan(base[outside].float()).all()


@pytest.mark.parametrize("dtype", BOTH)
def test_residual_in_place_and_side_by_side_outputs(dtype):
    T, K, N = 70, 64, 96
    g = torch.Generator().manual_seed(3)
    x, w, r = rand(g, T, K, dtype=dtype), rand(g, K, N, dtype=dtype), rand(g, T, N, dtype=dtype)
    plan = api.rar_linear_plan(K, N, CODE[dtype], api.ACT_RELU)
    both = torch.zeros(T, 2 * N, dtype=R.DT[dtype], device=DEV)
    y, z = both[:, :N], both[:, N:]
    y.copy_(r)
    api.rar_linear_forward(plan, T, x.to(DEV), w.to(DEV), None, y, y, pre=z)
    (ry, ey), (rz, ez) = R.forward(x, w, None, r, "relu", dtype)
    R.check(y, ry, ey, "y")
    R.check(z, rz, ez, "z")


@pytest.mark.parametrize("dtype", BOTH)
def test_backward_parts_alone_equal_the_whole(dtype):
    T, K, N = 90, 72, 56
    g = torch.Generator().manual_seed(9)
    dy, x, z, w = (rand(g, *s, dtype=dtype).to(DEV) for s in ((T, N), (T, K), (T, N), (K, N)))
    plan = api.rar_linear_plan(K, N, CODE[dtype], api.ACT_GELU)
    whole = [nan_like(T, K, dtype=dtype), nan_like(K, N, dtype=dtype), nan_like(N, dtype=dtype)]
    api.rar_linear_backward(plan, T, dy, x, w, z, *whole)
    for k, (xx, ww) in enumerate(((None, w), (x, None), (None, None))):
        part = [None] * 3
        part[k] = torch.full_like(whole[k], float("nan"))
        api.rar_linear_backward(plan, T, dy, xx, ww, z, *part)
        assert torch.equal(part[k], whole[k])


@pytest.mark.parametrize("dtype", BOTH)
def test_no_rows(dtype):
    K, N = 24, 40
    plan = api.rar_linear_plan(K, N, CODE[dtype], api.ACT_GELU)
    td = R.DT[dtype]
    e = lambda n: torch.empty(0, n, dtype=td, device=DEV)
    w = torch.ones(K, N, dtype=td, device=DEV)
    api.rar_linear_forward(plan, 0, e(K), w, None, None, e(N), pre=e(N))
    dw, db = nan_like(K, N, dtype=dtype), nan_like(N, dtype=dtype)
    api.rar_linear_backward(plan, 0, e(N), e(K), w, e(N), e(K), dw, db)
    assert not dw.any() and not db.any()
    dw.fill_(3)
    api.rar_linear_backward(plan, 0, e(N), e(K), w, e(N), e(K), dw, None, accumulate=True)
    assert (dw == 3).all()
    grad = nan_like(7, 5, dtype=dtype)
    ids = torch.empty(0, dtype=torch.int64, device=DEV)
    api.rar_embed_grad(7, 5, CODE[dtype], 0, ids, e(5), grad)
    assert not grad.any()
    api.rar_embed_lookup(7, 5, CODE[dtype], grad, 0, ids, e(5))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
def test_activation_values(dtype, act):
    # the activation and its derivative over every bf16 value: z = x * 1, dx = act'(z)
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    x = v.to(R.DT[dtype]).reshape(-1, 1)
    T = x.shape[0]
    one = torch.ones(1, 1, dtype=R.DT[dtype])
    plan = api.rar_linear_plan(1, 1, CODE[dtype], R.ACTS[act])
    y, dx = nan_like(T, 1, dtype=dtype), nan_like(T, 1, dtype=dtype)
    api.rar_linear_forward(plan, T, x.to(DEV), one.to(DEV), None, None, y)
    api.rar_linear_backward(plan, T, torch.ones(T, 1, dtype=R.DT[dtype], device=DEV), None, one.to(DEV), x.to(DEV), dx,
                            None, None)
    z = x.double()
    u = R.U[dtype]
    want = R.act(z, act)
    # relative to the value itself, far tail included: the exponential's argument carries z^2 / 2 * 2^-22, and
    # results under 2^-126 may be flushed to zero
    rel = (2.0 ** -20 + z * z * 2.0 ** -22 if act == "gelu" else 0 * z)
    R.check(y, want, (rel + 1.01 * u) * want.abs() + 2.0 ** -120, "act")
    want = R.act_grad(z, act)
    slack = rel * (R.phi(z) + (z.abs() * torch.exp(-z * z / 2) * 0.4)) if act == "gelu" else 0 * z
    R.check(dx, want, slack + 2.02 * u * want.abs() + 2.0 ** -120, "act'")


@pytest.mark.parametrize("dtype", BOTH)
def test_infinities_and_nan(dtype):
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[inf], [-inf], [nan], [2.0]], dtype=R.DT[dtype], device=DEV)
    one = torch.ones(1, 1, dtype=R.DT[dtype], device=DEV)
    for act, y_want, d_want in (("relu", [inf, 0, nan, 2], [1, 0, nan, 1]),
                                ("gelu", [inf, 0, nan, None], [1, 0, nan, None]),
                                ("none", [inf, -inf, nan, 2], [1, 1, 1, 1])):
        plan = api.rar_linear_plan(1, 1, CODE[dtype], R.ACTS[act])
        y, dx = nan_like(4, 1, dtype=dtype), nan_like(4, 1, dtype=dtype)
        api.rar_linear_forward(plan, 4, x, one, None, None, y)
        api.rar_linear_backward(plan, 4, torch.ones_like(y), None, one, x, dx, None, None)
        for got, want in ((y, y_want), (dx, d_want)):
            for a, b in zip(got.flatten().tolist(), want):
                assert b is None or a == b or (a != a and b != b), (act, got, want)
    # a NaN row stays in its row, a NaN column of W in its column, whatever tile they share
    T, K, N = 40, 72, 48
    g = torch.Generator().manual_seed(2)
    xs, w = rand(g, T, K, dtype=dtype), rand(g, K, N, dtype=dtype)
    xs[7, 3] = nan
    w[5, 11] = inf
    plan = api.rar_linear_plan(K, N, CODE[dtype])
    y = torch.zeros(T, N, dtype=R.DT[dtype], device=DEV)
    api.rar_linear_forward(plan, T, xs.to(DEV), w.to(DEV), None, None, y)
    bad = ~torch.isfinite(y).cpu()
    want = torch.zeros(T, N, dtype=torch.bool)
    want[7], want[:, 11] = True, True
    assert torch.equal(bad, want)


# ---------------------------------------------------------------------------
# 8-bit checkpoints
# ---------------------------------------------------------------------------

def make_ckpt(x, dtype):
    T, D = x.shape
    pitch, groups = api.rar_ckpt_size(D)
    codes = torch.full((T, pitch), 0x55, dtype=torch.uint8, device=DEV)
    scales = torch.full((T, groups), 0x55, dtype=torch.uint8, device=DEV)
    api.rar_ckpt_store(T, D, CODE[dtype], x, codes, scales)
    return codes, scales


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,D", [(1, 1), (1, 31), (1, 32), (2, 33), (5, 77), (64, 8), (67, 1001), (300, 512),
                                 (3, 8200)])
def test_ckpt_store_and_load(T, D, dtype):
    g = torch.Generator().manual_seed(T + D)
    x = rand(g, T, D, dtype=dtype) * torch.exp2(torch.randint(-20, 20, (T, D), generator=g)).to(R.DT[dtype])
    x[torch.rand(T, D, generator=g) < 0.1] = 0
    codes, scales, vals = R.quantise(x)
    for view in (x.to(DEV), strided(x, 8, 8), strided(x, 3, 1)):
        c, s = make_ckpt(view, dtype)
        assert np.array_equal(s.cpu().numpy(), scales)
        got = c.cpu().numpy()
        zero = (codes & 127) == 0
        assert np.array_equal(np.where(zero, 0, got), np.where(zero, 0, codes)) and not (got[zero] & 127).any()
    for act in ("none", "relu", "gelu"):
        want = R.act(torch.from_numpy(vals), act)
        for y in (nan_like(T, D, dtype=dtype), strided(torch.zeros(T, D, dtype=R.DT[dtype]), 3, 1)):
            api.rar_ckpt_load(T, D, CODE[dtype], c, s, y, act=R.ACTS[act])
            if act == "gelu":
                v = torch.from_numpy(vals)
                rel = 2.0 ** -20 + v * v * 2.0 ** -22
                R.check(y, want, (rel + 1.01 * R.U[dtype]) * want.abs() + 2.0 ** -120, "gelu")
            else:
                # four significant bits: exact in either type
                assert torch.equal(y.double().cpu(), want)


def test_ckpt_every_bf16_value_and_scale():
    # every finite bf16 magnitude against group maxima across the exponent range
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = bits[torch.randperm(65536, generator=torch.Generator().manual_seed(1))].reshape(-1, 32).clone()
    y = bits.reshape(-1, 32).clone()
    for t in (x, y):
        codes, scales, vals = R.quantise(t)
        c, s = make_ckpt(t.to(DEV), "bf16")
        assert np.array_equal(s.cpu().numpy(), scales)
        got = R.values(c.cpu().numpy(), s.cpu().numpy(), 32).numpy()
        assert np.array_equal(got, vals, equal_nan=True)
        z = torch.empty(t.shape, dtype=torch.float32, device=DEV)
        api.rar_ckpt_load(t.shape[0], 32, api.F32, c, s, z)
        # four significant bits of a value next to 2^128 may round to 2^128, which binary32 holds as infinity
        with np.errstate(over="ignore"):
            assert np.array_equal(z.cpu().numpy(), vals.astype(np.float32), equal_nan=True)


def test_ckpt_load_reads_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.uint8).reshape(8, 32).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8).repeat_interleave(8).reshape(-1, 1)
    want = R.values(codes.numpy(), scales.numpy(), 32)
    want[scales.flatten() == 255] = float("nan")
    y = torch.empty(2048, 32, dtype=torch.float32, device=DEV)
    api.rar_ckpt_load(2048, 32, api.F32, codes.to(DEV), scales.to(DEV), y)
    f32 = want.float()
    got = y.cpu()
    fine = ~torch.isnan(f32)
    assert torch.equal(~torch.isnan(got), fine) and torch.equal(got[fine], f32[fine])


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("shape", [(1, 1, 1), (5, 33, 70), (200, 264, 136), (67, 1000, 31), (3000, 72, 4200)], ids=str)
def test_forward_writes_the_checkpoint_of_z(shape, dtype):
    T, K, N = shape
    g = torch.Generator().manual_seed(K)
    x, w, b = rand(g, T, K, dtype=dtype), rand(g, K, N, dtype=dtype, scale=K ** -0.5), rand(g, N, dtype=dtype)
    plan = api.rar_linear_plan(K, N, CODE[dtype], api.ACT_GELU)
    y, z, y2 = (nan_like(T, N, dtype=dtype) for _ in range(3))
    args = plan, T, x.to(DEV), w.to(DEV), b.to(DEV), None
    api.rar_linear_forward(*args, y, pre=z)
    want_c, want_s = make_ckpt(z, dtype)
    c, s = torch.full_like(want_c, 0x55), torch.full_like(want_s, 0x55)
    api.rar_linear_forward(*args, y2, pre=c, pre_scales=s)
    assert torch.equal(y, y2) and torch.equal(c, want_c) and torch.equal(s, want_s)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 5, 7), (130, 257, 131), (515, 96, 640), (67, 3400, 4104)], ids=str)
def test_backward_from_checkpoints(shape, act, dtype):
    T, K, N = shape
    g = torch.Generator().manual_seed(T + K + N)
    dy, x, z = (rand(g, T, n, dtype=dtype) for n in (N, K, N))
    w = rand(g, K, N, dtype=dtype, scale=K ** -0.5)
    plan = api.rar_linear_plan(K, N, CODE[dtype], R.ACTS[act])
    (xc, xs), (zc, zs) = make_ckpt(x.to(DEV), dtype), make_ckpt(z.to(DEV), dtype)
    xv = torch.from_numpy(R.quantise(x)[2])
    zv = torch.from_numpy(R.quantise(z)[2])
    for use_x, use_z in ((True, True), (True, False), (False, True)):
        out = [nan_like(T, K, dtype=dtype), nan_like(K, N, dtype=dtype), nan_like(N, dtype=dtype)]
        api.rar_linear_backward(plan, T, dy.to(DEV), xc if use_x else x.to(DEV), w.to(DEV), zc if use_z else z.to(DEV),
                                *out, x_scales=xs if use_x else None, pre_scales=zs if use_z else None)
        ref = R.backward(dy, xv if use_x else x, w, zv if use_z else z, act, dtype)
        for got, (want, bound), what in zip(out, ref, ("dx", "dw", "db")):
            R.check(got, want, bound, f"{what} x8={use_x} z8={use_z}")


# ---------------------------------------------------------------------------
# Embedding
# ---------------------------------------------------------------------------

EMBED = [(1, 1, 1), (1, 5, 8), (63, 7, 3), (33, 300, 520), (4096, 50, 24), (4097, 300, 40), (9000, 70000, 9),
         (20000, 11, 130), (5000, 256, 513), (4500, 66000, 16), (8192, 40, 1536), (8193, 30, 2056), (700, 9, 1024)]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,V,D", EMBED)
def test_embedding(T, V, D, dtype):
    g = torch.Generator().manual_seed(T + V + D)
    ids = torch.randint(0, V, (T,), generator=g)
    if T > 8:
        ids[torch.rand(T, generator=g) < 0.5] = V // 2          # one frequent token
        ids[torch.rand(T, generator=g) < 0.05] = -1             # padding
        ids[3], ids[5], ids[6] = V, 2 ** 40, -2 ** 40           # outside
    scale = 1.7
    table, dy = rand(g, V, D, dtype=dtype), rand(g, T, D, dtype=dtype)
    ok = (ids >= 0) & (ids < V)
    s32 = torch.tensor(scale, dtype=torch.float32)
    want = torch.where(ok[:, None], (table[torch.where(ok, ids, 0)].float() * s32), torch.zeros(())).to(R.DT[dtype])
    for out in (nan_like(T, D, dtype=dtype), strided(torch.zeros(T, D, dtype=R.DT[dtype]), 3, 1)):
        api.rar_embed_lookup(V, D, CODE[dtype], table.to(DEV), T, ids.to(DEV), out, scale)
        assert torch.equal(out.cpu(), want)                     # one product, one rounding
    g0 = rand(g, V, D, dtype=dtype)
    for acc in (False, True):
        for d in (dy.to(DEV), strided(dy, 8, 8), strided(dy, 3, 1)):
            grad = g0.to(DEV) if acc else nan_like(V, D, dtype=dtype)
            api.rar_embed_grad(V, D, CODE[dtype], T, ids.to(DEV), d, grad, scale, accumulate=acc)
            want_g, bound = R.embed_grad(V, ids, dy, scale, dtype, g0 if acc else None)
            R.check(grad, want_g, bound, f"grad accumulate={acc}")
            if acc:
                idle = torch.bincount(ids[ok], minlength=V) == 0
                assert torch.equal(grad.cpu()[idle], g0[idle])


@pytest.mark.parametrize("T", [7, 8, 9, 31, 32, 256, 264, 1024, 1056, 3100, 5000, 70000])
def test_embed_grad_one_token_for_all(T):
    # a run that is the whole batch, and one that starts off the partial rows' boundaries
    V, D = 6, 40
    g = torch.Generator().manual_seed(T)
    dy = rand(g, T, D)
    for lead in (0, 1, 29):
        ids = torch.full((T,), 4)
        ids[:lead] = 1
        grad = nan_like(V, D, dtype="f32")
        api.rar_embed_grad(V, D, api.F32, T, ids.to(DEV), dy.to(DEV), grad)
        want, bound = R.embed_grad(V, ids, dy, 1.0, "f32")
        R.check(grad, want, bound, f"lead {lead}")


def test_embed_grad_row_order_is_token_order():
    # three values whose sum depends on the order: the run is summed as the tokens come
    big = 2.0 ** 25
    vals = torch.tensor([big, 1.0, -big, 1.0, 0.5])
    ids = torch.tensor([3, 3, 3, 3, 0])
    grad = nan_like(4, 1, dtype="f32")
    api.rar_embed_grad(4, 1, api.F32, 5, ids.to(DEV), vals.reshape(-1, 1).to(DEV), grad)
    want = np.float32(0)
    for v in vals[:4].numpy():
        want = np.float32(want + v)
    assert grad.cpu().flatten().tolist() == [0.5, 0, 0, float(want)]


def test_embedding_offsets_past_32_bits():
    # a table of 4.4 GB: rows past 2^32 bytes and past 2^31 elements' half
    V, D, T = 1_100_000, 1000, 600
    ids = torch.randint(V - 1000, V, (T,), generator=torch.Generator().manual_seed(1))
    ids[0] = V - 1
    table = torch.zeros(V, D, device=DEV)
    rows = torch.randn(1000, D, generator=torch.Generator().manual_seed(2))
    table[V - 1000:] = rows.to(DEV)
    out = nan_like(T, D, dtype="f32")
    api.rar_embed_lookup(V, D, api.F32, table, T, ids.to(DEV), out)
    assert torch.equal(out.cpu(), rows[ids - (V - 1000)])
    api.rar_embed_grad(V, D, api.F32, T, ids.to(DEV), out, table)
    want, bound = R.embed_grad(1000, ids - (V - 1000), out.cpu(), 1.0, "f32")
    R.check(table[V - 1000:], want, bound, "grad")
    assert not table[:V - 1000].any()


# ---------------------------------------------------------------------------
# Largest sizes
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", BOTH)
def test_linear_most_rows(dtype):
    """2^24 rows that have to be packed.  Small integers: every sum is exact
    (|dw|, |db| <= 2^24) until its one rounding, so the results are compared
    with equality."""
    T, K, N = 1 << 24, 5, 3
    g = torch.Generator(device=DEV).manual_seed(5)
    x, w, dy = (torch.randint(-1, 2, s, device=DEV, generator=g, dtype=torch.int32) for s in ((T, K), (K, N), (T, N)))
    xf, wf, dyf = (t.to(R.DT[dtype]) for t in (x, w, dy))
    plan = api.rar_linear_plan(K, N, CODE[dtype])
    y, dx = nan_like(T, N, dtype=dtype), nan_like(T, K, dtype=dtype)
    dw, db = nan_like(K, N, dtype=dtype), nan_like(N, dtype=dtype)
    api.rar_linear_forward(plan, T, xf, wf, None, None, y)
    api.rar_linear_backward(plan, T, dyf, xf, wf, None, dx, dw, db)
    for k in range(K):
        assert torch.equal(dx[:, k], (dy * w[k]).sum(1).to(dx.dtype))
        assert torch.equal(dw[k], (x[:, k:k + 1] * dy).sum(0).float().to(dw.dtype))
    for n in range(N):
        assert torch.equal(y[:, n], (x * w[:, n]).sum(1).to(y.dtype))
    assert torch.equal(db, dy.sum(0).float().to(db.dtype))


@pytest.mark.parametrize("dtype", BOTH)
def test_linear_widest_rows(dtype):
    """Rows 2^22 elements apart, the most a call takes: offsets pass 2^31 bytes
    inside a tile's operand and 2^32 bytes behind it."""
    T, K, N, ld = 530, 40, 24, 1 << 22
    g = torch.Generator().manual_seed(6)
    big = torch.full((T * ld,), float("nan"), dtype=R.DT[dtype], device=DEV).view(T, ld)
    x, dy = rand(g, T, K, dtype=dtype), rand(g, T, N, dtype=dtype)
    w = rand(g, K, N, dtype=dtype, scale=K ** -0.5)
    plan = api.rar_linear_plan(K, N, CODE[dtype])
    vx, vdy, y, dx = big[:, 64:64 + K], big[:, ld - 128:ld - 128 + N], big[:, 256:256 + N], big[:, 320:320 + K]
    vx.copy_(x.to(DEV))
    vdy.copy_(dy.to(DEV))
    dw, db = nan_like(K, N, dtype=dtype), nan_like(N, dtype=dtype)
    api.rar_linear_forward(plan, T, vx, w.to(DEV), None, None, y)
    api.rar_linear_backward(plan, T, vdy, vx, w.to(DEV), None, dx, dw, db)
    (ry, ey), _ = R.forward(x, w, None, None, "none", dtype)
    R.check(y, ry, ey, "y")
    packed = [nan_like(T, K, dtype=dtype), nan_like(K, N, dtype=dtype), nan_like(N, dtype=dtype)]
    api.rar_linear_backward(plan, T, dy.to(DEV), x.to(DEV), w.to(DEV), None, *packed)
    for got, want in zip((dx, dw, db), packed):
        assert torch.equal(got, want)
    assert torch.isnan(big[:, 256 + N:320]).all() and torch.isnan(big[:, 320 + K:512]).all()


def test_lookup_of_more_elements_than_one_launch():
    T, D, V = 1 << 24, 1025, 7
    ids = torch.arange(T, device=DEV) % V
    table = torch.randn(V, D, device=DEV).bfloat16()
    out = torch.empty(T, D, dtype=torch.bfloat16, device=DEV)
    out[-9:] = float("nan")
    api.rar_embed_lookup(V, D, api.BF16, table, T, ids, out)
    at = torch.cat([torch.arange(0, T, 65537), torch.arange((1 << 33) // D - 5, (1 << 33) // D + 5),
                    torch.arange(T - 9, T)]).to(DEV)
    assert torch.equal(out[at], table[ids[at]])


@pytest.mark.parametrize("V", [5, 70_000])
def test_embed_grad_of_most_tokens(V):
    """2^24 tokens, some of them padding.  Small integers: every sum is exact."""
    T, D = 1 << 24, 2
    g = torch.Generator(device=DEV).manual_seed(8)
    ids = torch.randint(-1, V + 1, (T,), device=DEV, generator=g)
    dy = torch.randint(-1, 2, (T, D), device=DEV, generator=g)
    grad = nan_like(V, D, dtype="f32")
    api.rar_embed_grad(V, D, api.F32, T, ids, dy.float(), grad)
    ok = (ids >= 0) & (ids < V)
    want = torch.zeros(V, D, dtype=torch.int64, device=DEV).index_add_(0, ids[ok], dy[ok])
    assert torch.equal(grad, want.float())


def test_ckpt_offsets_past_32_bits():
    T, D = 4_200_000, 1025
    x = torch.zeros(T, D, dtype=torch.bfloat16, device=DEV)
    x[-100:] = torch.randn(100, D, device=DEV).bfloat16()
    pitch, groups = api.rar_ckpt_size(D)
    u8 = dict(dtype=torch.uint8, device=DEV)
    codes, scales = torch.empty(T, pitch, **u8), torch.empty(T, groups, **u8)
    api.rar_ckpt_store(T, D, api.BF16, x, codes, scales)
    c2, s2 = torch.empty(100, pitch, **u8), torch.empty(100, groups, **u8)
    api.rar_ckpt_store(100, D, api.BF16, x[-100:], c2, s2)
    assert torch.equal(codes[-100:, :D], c2[:, :D]) and torch.equal(scales[-100:], s2)
    y2 = torch.empty(100, D, dtype=torch.bfloat16, device=DEV)
    api.rar_ckpt_load(100, D, api.BF16, c2, s2, y2)
    api.rar_ckpt_load(T, D, api.BF16, codes, scales, x, api.ACT_RELU)
    assert torch.equal(x[-100:], y2.clamp_min(0)) and not x[:-100].any()


# ---------------------------------------------------------------------------
# Streams, graphs, repeatability
# ---------------------------------------------------------------------------

def _step(dtype):
    """A run of all operators on fixed inputs; returns (call, outputs)."""
    T, K, N, V = 700, 136, 264, 900
    g = torch.Generator().manual_seed(21)
    td = R.DT[dtype]
    ids = torch.randint(-1, 40, (T,), generator=g).to(DEV)
    table, w, b = (rand(g, *s, dtype=dtype, scale=0.3).to(DEV) for s in ((V, K), (K, N), (N,)))
    dy = rand(g, T, N, dtype=dtype).to(DEV)
    plan = api.rar_linear_plan(K, N, CODE[dtype], api.ACT_GELU)
    x, y, dx = (torch.zeros(T, n, dtype=td, device=DEV) for n in (K, N, K))
    (xp, xg), (zp, zg) = api.rar_ckpt_size(K), api.rar_ckpt_size(N)
    xc, xs, zc, zs = (torch.zeros(T, n, dtype=torch.uint8, device=DEV) for n in (xp, xg, zp, zg))
    dw, db, grad = (torch.zeros(*s, dtype=td, device=DEV) for s in ((K, N), (N,), (V, K)))

    def call(stream=None):
        c = CODE[dtype]
        api.rar_embed_lookup(V, K, c, table, T, ids, x, 2.0, stream=stream)
        api.rar_ckpt_store(T, K, c, x, xc, xs, stream=stream)
        api.rar_linear_forward(plan, T, x, w, b, None, y, pre=zc, pre_scales=zs, stream=stream)
        api.rar_linear_backward(plan, T, dy, xc, w, zc, dx, dw, db, x_scales=xs, pre_scales=zs, stream=stream)
        api.rar_embed_grad(V, K, c, T, ids, dx, grad, 2.0, stream=stream)

    return call, [x, xc, xs, y, zc, zs, dx, dw, db, grad]


def _bits(outs):
    return [t.clone() for t in outs]


def _same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", BOTH)
def test_repeated_calls_give_the_same_bits(dtype):
    call, outs = _step(dtype)
    call()
    torch.cuda.synchronize()
    first = _bits(outs)
    for _ in range(5):
        for t in outs:
            t.zero_()
        call()
        torch.cuda.synchronize()
        assert _same(outs, first)


@pytest.mark.parametrize("dtype", BOTH)
def test_other_streams_and_two_at_once(dtype):
    (call_a, a), (call_b, b) = _step(dtype), _step(dtype)
    call_a()
    torch.cuda.synchronize()
    want = _bits(a)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for t in a:
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        call_a(s1)                   # a torch stream, workspace allocated on another
        call_b(s2.cuda_stream)       # a raw stream handle
    torch.cuda.synchronize()
    assert _same(a, want) and _same(b, want)
    # the default stream by its handle, from inside another stream
    for t in a:
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        call_a(0)
    torch.cuda.synchronize()
    assert _same(a, want)


@pytest.mark.parametrize("dtype", BOTH)
def test_replays_from_graphs(dtype):
    # two graphs captured from two copies, replayed together, with eager work between the replays
    (call_a, a), (call_b, b) = _step(dtype), _step(dtype)
    call_a()
    call_b()
    torch.cuda.synchronize()
    want = _bits(a)
    graphs = []
    for call in (call_a, call_b):
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph):
            call()
        graphs.append(gph)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for rep in range(4):
        for t in a + b:
            t.zero_()
        _ = torch.randn(1000, device=DEV).sum().item()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert _same(a, want) and _same(b, want), f"replay {rep}"


# ---------------------------------------------------------------------------
# Differences, and a training step of several ranks
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
@pytest.mark.parametrize("shape", [(3, 5, 7), (40, 72, 33), (130, 96, 200)], ids=str)
def test_gradients_against_differences(shape, act):
    # along a direction v: (L(+h) - L(-h)) / 2h of the kernels' own forward pass, L = sum(c * y), against the
    # gradient's product with v.  Off by h^2 / 6 * |act'''| <= h^2 / 6 a term (gelu''' is below 0.8; the other
    # activations are linear away from 0), and by both passes' rounding over 2h.
    T, K, N = shape
    h = 2.0 ** -6
    g = torch.Generator().manual_seed(K)
    x, w, b, c = rand(g, T, K), rand(g, K, N, scale=K ** -0.5), rand(g, N), rand(g, T, N)
    vx, vw, vb = rand(g, T, K), rand(g, K, N, scale=K ** -0.5), rand(g, N)
    plan = api.rar_linear_plan(K, N, api.F32, R.ACTS[act])

    def forward(x, w, b):
        y, z = nan_like(T, N, dtype="f32"), nan_like(T, N, dtype="f32")
        api.rar_linear_forward(plan, T, x.to(DEV), w.to(DEV), b.to(DEV), None, y, pre=z)
        return y.double().cpu(), z, R.forward(x, w, b, None, act, "f32")[0][1]

    _, z, _ = forward(x, w, b)
    dx, dw, db = nan_like(T, K, dtype="f32"), nan_like(K, N, dtype="f32"), nan_like(N, dtype="f32")
    api.rar_linear_backward(plan, T, c.to(DEV), x.to(DEV), w.to(DEV), z, dx, dw, db)
    grads = R.backward(c, x, w, z.cpu(), act, "f32")
    zero = lambda t: torch.zeros_like(t)
    for k, (grad, v, d) in enumerate(((dx, vx, (vx, zero(w), zero(b))), (dw, vw, (zero(x), vw, zero(b))),
                                      (db, vb, (zero(x), zero(w), vb)))):
        at = lambda s: (x + s * h * d[0], w + s * h * d[1], b + s * h * d[2])
        yp, zp, ep = forward(*at(1))
        ym, zm, em = forward(*at(-1))
        # relu: keep to outputs whose z has one sign on both sides
        use = (torch.sign(zp) == torch.sign(zm)).cpu() if act == "relu" else torch.ones(T, N, dtype=torch.bool)
        step = ((zp - zm).double().cpu() / 2).abs()
        diff = ((yp - ym) * c.double())[use].sum() / (2 * h)
        cut = (c * use).to(torch.float32)
        if not use.all():
            api.rar_linear_backward(plan, T, cut.to(DEV), x.to(DEV), w.to(DEV), z, dx, dw, db)
            grads = R.backward(cut, x, w, z.cpu(), act, "f32")
        want = (grad.double().cpu() * v.double()).sum()
        bound = (cut.double().abs() * (ep + em)).sum() / (2 * h) + (grads[k][1] * v.double().abs()).sum()
        if act == "gelu":
            bound += (cut.double().abs() * step ** 3).sum() / (6 * h)
        # the operands of the two passes are rounded sums x + h v: half a step each
        moved = [2.0 ** -24 * (p.double().abs() + h * q.double().abs()) for p, q in zip((x, w, b), d)]
        drift = moved[0] @ w.double().abs() + x.double().abs() @ moved[1] + moved[2]
        bound += 1.3 * (cut.double().abs() * drift).sum() / h
        assert abs(diff - want) <= bound, (k, float(diff), float(want), float(bound))
        if not use.all():
            api.rar_linear_backward(plan, T, c.to(DEV), x.to(DEV), w.to(DEV), z, dx, dw, db)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("ckpt", [False, True])
def test_training_step_of_ranks(dtype, ckpt):
    """Embedding, two linear layers with a residual, their backward passes into per-rank arenas, and the bucketed
    all-reduce over them, each bucket behind the event that its last gradient records: the mean of the ranks'
    gradients."""
    ranks, T, V, d, h = 4, 200, 300, 48, 136
    code, td = CODE[dtype], R.DT[dtype]
    g = torch.Generator().manual_seed(8)
    table, w1, w2 = (rand(g, *s, dtype=dtype, scale=0.2) for s in ((V, d), (d, h), (h, d)))
    b1, b2 = rand(g, h, dtype=dtype), rand(g, d, dtype=dtype)
    ids = [torch.randint(-1, V, (T,), generator=g) for _ in range(ranks)]
    dys = [rand(g, T, d, dtype=dtype) for _ in range(ranks)]
    l1, l2 = api.rar_linear_plan(d, h, code, api.ACT_GELU), api.rar_linear_plan(h, d, code)
    # backward order: W2, b2, W1, b1, embedding
    shapes = [(h, d), (d,), (d, h), (h,), (V, d)]
    numel = [int(np.prod(s)) for s in shapes]
    total = sum(numel)
    buckets = api.rar_bucket_plan(numel, code, 16 * 512)
    n_buckets = api.rar_bucket_count(buckets)[0]
    arenas = [torch.full((total,), float("nan"), dtype=td, device=DEV) for _ in range(ranks)]
    ends = np.cumsum(numel)
    dev = lambda t: t.to(DEV)
    gt, gw1, gw2, gb1, gb2 = map(dev, (table, w1, w2, b1, b2))
    producer, comm = torch.cuda.Stream(), torch.cuda.Stream()
    want = [torch.zeros(s, dtype=torch.float64) for s in shapes]
    torch.cuda.synchronize()
    with torch.cuda.stream(producer):
        state = []
        for r in range(ranks):
            views, at = [], 0
            for s, n in zip(shapes, numel):
                views.append(arenas[r][at:at + n].view(s))
                at += n
            x, a, y = (torch.empty(T, n, dtype=td, device=DEV) for n in (d, h, d))
            api.rar_embed_lookup(V, d, code, gt, T, dev(ids[r]), x, 1.5)
            kw = {}
            if ckpt:
                (xp, xg), (zp, zg) = api.rar_ckpt_size(d), api.rar_ckpt_size(h)
                xk, xs, z, zs = (torch.empty(T, n, dtype=torch.uint8, device=DEV) for n in (xp, xg, zp, zg))
                api.rar_ckpt_store(T, d, code, x, xk, xs)
                api.rar_linear_forward(l1, T, x, gw1, gb1, None, a, pre=z, pre_scales=zs)
                kw = dict(x_scales=xs, pre_scales=zs)
            else:
                xk, z = x, torch.empty(T, h, dtype=td, device=DEV)
                api.rar_linear_forward(l1, T, x, gw1, gb1, None, a, pre=z)
            api.rar_linear_forward(l2, T, a, gw2, gb2, x, y)
            state.append((views, x, xk, a, z, kw, dev(ids[r]), dev(dys[r]), y))
        # layer by layer over the ranks, as their passes run side by side
        das = []
        for views, x, xk, a, z, kw, i, dy, y in state:
            if ckpt:
                api.rar_ckpt_load(T, h, code, z, kw["pre_scales"], a, act=api.ACT_GELU)
            da = torch.empty(T, h, dtype=td, device=DEV)
            api.rar_linear_backward(l2, T, dy, a, gw2, None, da, views[0], views[1])
            das.append(da)
        second = torch.cuda.Event()
        second.record(producer)
        dxs = []
        for (views, x, xk, a, z, kw, i, dy, y), da in zip(state, das):
            dx = torch.empty(T, d, dtype=td, device=DEV)
            api.rar_linear_backward(l1, T, da, xk, gw1, z, dx, views[2], views[3], **kw)
            dx += dy                                      # the residual's share
            dxs.append(dx)
        first = torch.cuda.Event()
        first.record(producer)
        for (views, x, xk, a, z, kw, i, dy, y), dx in zip(state, dxs):
            api.rar_embed_grad(V, d, code, T, i, dx, views[4], 1.5)
        last = torch.cuda.Event()
        last.record(producer)
    events = []
    for k in range(n_buckets):
        so, el, _ = api.rar_bucket_info(buckets, k)
        events.append(second if so + el <= ends[1] else first if so + el <= ends[3] else last)
    api.rar_bucket_allreduce_arena(buckets, arenas, events, stream=comm)
    torch.cuda.synchronize()
    # the same step in 64 bits, from what each operator reads; values kept in 8 bits from their codes
    bound = [torch.zeros(s, dtype=torch.float64) for s in shapes]
    for (views, x, xk, a, z, kw, i, dy, y), da, dx in zip(state, das, dxs):
        cpu = lambda t: t.detach().cpu()
        xv = R.values(cpu(xk).numpy(), cpu(kw["x_scales"]).numpy(), d) if ckpt else cpu(x)
        zv = R.values(cpu(z).numpy(), cpu(kw["pre_scales"]).numpy(), h) if ckpt else cpu(z)
        (_, _), (dw2, e2), (db2, f2) = R.backward(cpu(dy), cpu(a), w2, torch.zeros(T, d), "none", dtype)
        (_, _), (dw1, e1), (db1, f1) = R.backward(cpu(da), xv, w1, zv, "gelu", dtype)
        de, ee = R.embed_grad(V, cpu(i), cpu(dx), 1.5, dtype)
        for k, (t, e) in enumerate(((dw2, e2), (db2, f2), (dw1, e1), (db1, f1), (de, ee))):
            want[k] += t / ranks
            bound[k] += (e + 2 ** -22 * t.abs()) / ranks
        # and the forward pass
        if not ckpt:  # (with checkpoints `a` was made again since)
            (ry, ey), _ = R.forward(cpu(a), w2, b2, cpu(x), "none", dtype)
            R.check(y, ry, ey, "y")
    for r in range(ranks):
        at = 0
        for k, (s, n) in enumerate(zip(shapes, numel)):
            got = arenas[r][at:at + n].view(s)
            R.check(got, want[k], bound[k] * (1 + R.U[dtype]) + R.U[dtype] * want[k].abs(), f"rank {r} tensor {k}")
            at += n
        assert torch.equal(arenas[r], arenas[0])


# ---------------------------------------------------------------------------
# An error that an earlier HIP call left
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", BOTH)
def test_an_earlier_error_is_not_taken_for_the_calls_own(dtype):
    """A HIP call of the caller's that the host refused (no such device) leaves
    HIP's last error set: the calls after it run to their end and report their
    own status."""
    hip = ctypes.CDLL("libamdhip64.so")
    g = torch.Generator().manual_seed(17)
    T, K, N, V = 300, 60, 1001, 40
    code, td = CODE[dtype], R.DT[dtype]
    x, dy, w, b = (rand(g, *s, dtype=dtype).to(DEV) for s in ((T, K), (T, N), (K, N), (N,)))
    table, dt = (rand(g, n, K, dtype=dtype).to(DEV) for n in (V, 9000))
    ids = torch.randint(0, V, (9000,), generator=g).to(DEV)
    plan = api.rar_linear_plan(K, N, code, api.ACT_GELU)
    (xp, xg) = api.rar_ckpt_size(K)
    u8 = dict(dtype=torch.uint8, device=DEV)
    ws = torch.empty(max(*api.rar_linear_workspace(plan, T), api.rar_embed_grad_workspace(V, K, 9000)), **u8)
    outs = [torch.empty(*s, dtype=td, device=DEV) for s in
            ((T, K), (V, K), (V, K), (T, N), (T, N), (2, N), (T, K), (K, N), (N,), (T, K))]
    look, few, many, y, z, y2, dx, dw, db, back = outs
    codes, scales = torch.empty(T, xp, **u8), torch.empty(T, xg, **u8)
    calls = [lambda: api.rar_embed_lookup(V, K, code, table, T, ids[:T], look),
             lambda: api.rar_embed_grad(V, K, code, T, ids[:T], dt[:T], few, ws=ws),
             lambda: api.rar_embed_grad(V, K, code, 9000, ids, dt, many, ws=ws),
             lambda: api.rar_linear_forward(plan, T, x, w, b, None, y, pre=z, ws=ws),
             lambda: api.rar_linear_forward(plan, 2, x[:2], w, b, None, y2, ws=ws),
             lambda: api.rar_linear_backward(plan, T, dy, x, w, z, dx, dw, db, ws=ws),
             lambda: api.rar_ckpt_store(T, K, code, x, codes, scales),
             lambda: api.rar_ckpt_load(T, K, code, codes, scales, back)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs + [codes, scales]]
    for t in outs + [codes, scales]:
        t.zero_()
    torch.cuda.synchronize()
    try:
        for call in calls:
            assert hip.hipSetDevice(1 << 20) != 0
            call()
    finally:
        hip.hipGetLastError()
    torch.cuda.synchronize()
    assert all(torch.equal(t, v) for t, v in zip(outs + [codes, scales], want))
