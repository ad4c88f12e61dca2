"""The linear layer and the embedding's gradient on the GPU at sizes that take
the launch forms of large calls.  Which tile and split a size takes is
asserted from the host's own choice in test_linear_shape.py.  Bounds count
roundings (see ops_ref.py)."""
import pytest
import torch

import ops_ref as R
from ops_sizes import EMBED_32, LINEAR
from ring_all_reduce_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CODE = {"f32": api.F32, "bf16": api.BF16}
BOTH = ["f32", "bf16"]


def nan_like(*shape, dtype):
    return torch.full(shape, float("nan"), dtype=R.DT[dtype], device=DEV)


@pytest.mark.parametrize("K,N", [(32, 1025), (1025, 32)])
def test_most_rows_and_many_tiles(K, N):
    """2^24 binary32 rows: more 64-tiles than a launch shared by two products
    holds, in y and in dx.  Small integers: every sum is exact."""
    T = 1 << 24
    g = torch.Generator(device=DEV).manual_seed(5)
    x, w, y, dx = (torch.empty(*s, device=DEV) for s in ((T, K), (K, N), (T, N), (T, K)))
    w.random_(-1, 2, generator=g)
    x.random_(-1, 2, generator=g)
    y[-1] = dx[-1] = float("nan")
    plan = api.rar_linear_plan(K, N, api.F32)
    ws = torch.empty(max(api.rar_linear_workspace(plan, T)), dtype=torch.uint8, device=DEV)
    at = torch.cat([torch.arange(0, T, 65537), torch.arange(T - 70, T)]).to(DEV)
    api.rar_linear_forward(plan, T, x, w, None, None, y, ws=ws)
    assert torch.equal(y[at], x[at] @ w)
    y.random_(-1, 2, generator=g)
    api.rar_linear_backward(plan, T, y, None, w, None, dx, None, None, ws=ws)
    assert torch.equal(dx[at], y[at] @ w.T.contiguous())
    del x, y, dx, ws
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# Large tiles of the linear layer (LINEAR names the tile of every product)
# ---------------------------------------------------------------------------

def rand(gen, *shape, dtype="f32", scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(R.DT[dtype])


def strided(t, extra, offset):
    """t as a view of a wider matrix (rows t.shape[1] + extra apart), NaN around it."""
    big = torch.full((t.shape[0] + 1, t.shape[1] + extra), float("nan"), dtype=t.dtype, device=DEV)
    v = big[:t.shape[0], offset:offset + t.shape[1]]
    v.copy_(t)
    return v


def near(got, want, bound, what):
    """R.check on the GPU."""
    got = got.double()
    bad = ((got - want).abs() > bound + 1e-37) | (~torch.isfinite(got) & torch.isfinite(want))
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: got {got[i].item()!r}, "
                             f"want {want[i].item()!r} +- {bound[i].item():.3g}")


ALL = [(s, dt, a) for dt in BOTH for s in LINEAR[dt] for a in (("gelu", "none") if s[0] < 5000 else ("relu",))]


@pytest.mark.parametrize("shape,dtype,act", ALL, ids=str)
def test_large_forward(shape, dtype, act):
    T, K, N = shape
    g = torch.Generator(device=DEV).manual_seed(T + K + N)
    x, w = rand(g, T, K, dtype=dtype), rand(g, K, N, dtype=dtype, scale=K ** -0.5)
    b, r = rand(g, N, dtype=dtype), rand(g, T, N, dtype=dtype)
    plan = api.rar_linear_plan(K, N, CODE[dtype], R.ACTS[act])
    for bias, res in ((b, r), (None, None)):
        y, z = nan_like(T, N, dtype=dtype), nan_like(T, N, dtype=dtype)
        api.rar_linear_forward(plan, T, x, w, bias, res, y, pre=z)
        (ry, ey), (rz, ez) = R.forward(x, w, bias, res, act, dtype)
        near(z, rz, ez, "z")
        near(y, ry, ey, "y")
        # the residual in place, and z not kept: the same bits
        y2 = nan_like(T, N, dtype=dtype) if res is None else res.clone()
        api.rar_linear_forward(plan, T, x, w, bias, None if res is None else y2, y2)
        assert torch.equal(y, y2)


@pytest.mark.parametrize("shape,dtype,act", ALL, ids=str)
def test_large_backward(shape, dtype, act):
    T, K, N = shape
    g = torch.Generator(device=DEV).manual_seed(T + 2 * K + N)
    dy, x, z = (rand(g, T, n, dtype=dtype) for n in (N, K, N))
    w = rand(g, K, N, dtype=dtype, scale=K ** -0.5)
    dw0, db0 = rand(g, K, N, dtype=dtype), rand(g, N, dtype=dtype)
    plan = api.rar_linear_plan(K, N, CODE[dtype], R.ACTS[act])
    for acc in (False, True):
        dx = nan_like(T, K, dtype=dtype)
        dw = dw0.clone() if acc else nan_like(K, N, dtype=dtype)
        db = db0.clone() if acc else nan_like(N, dtype=dtype)
        api.rar_linear_backward(plan, T, dy, x, w, z, dx, dw, db, accumulate=acc)
        ref = R.backward(dy, x, w, z, act, dtype, *((dw0, db0) if acc else ()))
        for got, (want, bound), what in zip((dx, dw, db), ref, ("dx", "dw", "db")):
            near(got, want, bound, f"{what} accumulate={acc}")
        if not acc:
            whole = dx, dw, db
    for k, (xx, ww) in enumerate(((None, w), (x, None), (None, None))):   # each output alone: the same bits
        part = [None] * 3
        part[k] = torch.full_like(whole[k], float("nan"))
        api.rar_linear_backward(plan, T, dy, xx, ww, z, *part)
        assert torch.equal(part[k], whole[k])


def ckpt(x, dtype):
    T, D = x.shape
    pitch, groups = api.rar_ckpt_size(D)
    codes, scales = (torch.full((T, n), 0x55, dtype=torch.uint8, device=DEV) for n in (pitch, groups))
    api.rar_ckpt_store(T, D, CODE[dtype], x, codes, scales)
    return codes, scales


@pytest.mark.parametrize("shape,dtype", [(s, dt) for dt in BOTH for s in LINEAR[dt]
                                         if LINEAR[dt][s][0][0] == (256 if dt == "bf16" else 128)], ids=str)
def test_large_forward_writes_the_checkpoint_of_z(shape, dtype):
    T, K, N = shape
    g = torch.Generator(device=DEV).manual_seed(K)
    x, w = rand(g, T, K, dtype=dtype), rand(g, K, N, dtype=dtype, scale=K ** -0.5)
    b = rand(g, N, dtype=dtype)
    plan = api.rar_linear_plan(K, N, CODE[dtype], api.ACT_GELU)
    y, z, y2 = (nan_like(T, N, dtype=dtype) for _ in range(3))
    api.rar_linear_forward(plan, T, x, w, b, None, y, pre=z)
    want_c, want_s = ckpt(z, dtype)
    c, s = torch.full_like(want_c, 0x55), torch.full_like(want_s, 0x55)
    api.rar_linear_forward(plan, T, x, w, b, None, y2, pre=c, pre_scales=s)
    assert torch.equal(y, y2) and torch.equal(c, want_c) and torch.equal(s, want_s)


@pytest.mark.parametrize("shape,dtype", [((4001, 1032, 4104), "bf16"), ((900, 4232, 3613), "bf16"),
                                         ((2328, 5320, 592), "bf16"), ((4479, 256, 4352), "f32"),
                                         ((458, 2075, 3552), "f32"), ((3278, 736, 1357), "f32")], ids=str)
def test_large_backward_from_checkpoints(shape, dtype):
    T, K, N = shape
    g = torch.Generator(device=DEV).manual_seed(T)
    dy, x, z = (rand(g, T, n, dtype=dtype) for n in (N, K, N))
    w = rand(g, K, N, dtype=dtype, scale=K ** -0.5)
    plan = api.rar_linear_plan(K, N, CODE[dtype], api.ACT_GELU)
    (xc, xs), (zc, zs) = ckpt(x, dtype), ckpt(z, dtype)
    xv, zv = (R.values(c.cpu().numpy(), s.cpu().numpy(), n).to(DEV) for c, s, n in ((xc, xs, K), (zc, zs, N)))
    for use_x, use_z in ((True, True), (True, False), (False, True)):
        out = [nan_like(T, K, dtype=dtype), nan_like(K, N, dtype=dtype), nan_like(N, dtype=dtype)]
        api.rar_linear_backward(plan, T, dy, xc if use_x else x, w, zc if use_z else z, *out,
                                x_scales=xs if use_x else None, pre_scales=zs if use_z else None)
        ref = R.backward(dy, xv if use_x else x, w, zv if use_z else z, "gelu", dtype)
        for got, (want, bound), what in zip(out, ref, ("dx", "dw", "db")):
            near(got, want, bound, f"{what} x8={use_x} z8={use_z}")


@pytest.mark.parametrize("extra,offset", [(8, 8), (3, 1)])
@pytest.mark.parametrize("shape,dtype", [((4121, 603, 2960), "bf16"), ((4001, 1032, 4104), "bf16"),
                                         ((3054, 392, 2384), "f32"), ((4479, 256, 4352), "f32")], ids=str)
def test_large_strides_and_surroundings(shape, dtype, extra, offset):
    # every matrix a view of a wider one with NaN around it: nothing outside is read into a result or written
    T, K, N = shape
    g = torch.Generator(device=DEV).manual_seed(11)
    x, r, dy, z0 = (rand(g, T, n, dtype=dtype) for n in (K, N, N, N))
    w, b = rand(g, K, N, dtype=dtype, scale=K ** -0.5), rand(g, N, dtype=dtype)
    plan = api.rar_linear_plan(K, N, CODE[dtype], api.ACT_GELU)
    xs, rs, dys, zs = (strided(t, extra, offset) for t in (x, r, dy, z0))
    y, z, dx = (strided(torch.zeros(T, n, dtype=R.DT[dtype], device=DEV), extra, offset) for n in (N, N, K))
    api.rar_linear_forward(plan, T, xs, w, b, rs, y, pre=z)
    (ry, ey), (rz, ez) = R.forward(x, w, b, r, "gelu", dtype)
    near(y, ry, ey, "y")
    near(z, rz, ez, "z")
    dw, db = nan_like(K, N, dtype=dtype), nan_like(N, dtype=dtype)
    api.rar_linear_backward(plan, T, dys, xs, w, zs, dx, dw, db)
    for got, (want, bound), what in zip((dx, dw, db), R.backward(dy, x, w, z0, "gelu", dtype), ("dx", "dw", "db")):
        near(got, want, bound, what)
    for view in (y, z, dx):
        outside = torch.ones_like(view._base, dtype=torch.bool)
        outside[:T, offset:offset + view.shape[1]] = False
        assert torch.isnan(view._base[outside].float()).all()


@pytest.mark.parametrize("shape,dtype", [((4001, 1032, 4104), "bf16"), ((6592, 728, 1832), "bf16"),
                                         ((4479, 256, 4352), "f32"), ((3054, 392, 2384), "f32")], ids=str)
def test_large_calls_repeat_and_replay(shape, dtype):
    T, K, N = shape
    g = torch.Generator(device=DEV).manual_seed(13)
    dy, x, w = rand(g, T, N, dtype=dtype), rand(g, T, K, dtype=dtype), rand(g, K, N, dtype=dtype, scale=K ** -0.5)
    plan = api.rar_linear_plan(K, N, CODE[dtype], api.ACT_GELU)
    outs = [nan_like(*s, dtype=dtype) for s in ((T, N), (T, N), (T, K), (K, N), (N,))]
    y, z, dx, dw, db = outs

    def call():
        api.rar_linear_forward(plan, T, x, w, None, None, y, pre=z)
        api.rar_linear_backward(plan, T, dy, x, w, z, dx, dw, db)

    call()
    torch.cuda.synchronize()
    first = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rep in range(4):
        for t in outs:
            t.zero_()
        torch.randn(1000, device=DEV).sum().item()
        call() if rep == 1 else graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, first)), rep


# ---------------------------------------------------------------------------
# The embedding's gradient in chunks of 32 sorted positions
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,V,D", EMBED_32)
def test_embed_grad_of_a_batch(T, V, D, dtype):
    g = torch.Generator().manual_seed(T + V + D)
    ids = torch.randint(0, V, (T,), generator=g)
    ids[torch.rand(T, generator=g) < 0.5] = V // 2          # one frequent token: runs of whole groups of chunks
    ids[torch.rand(T, generator=g) < 0.05] = -1             # padding
    ids[3], ids[5], ids[6] = V, 2 ** 40, -2 ** 40           # outside
    dy, g0 = (torch.randn(n, D, generator=g).to(R.DT[dtype]) for n in (T, V))
    live = (ids >= 0) & (ids < V)
    scale, first = 1.7, None
    want, bound = R.embed_grad(V, ids, dy, scale, dtype)
    want_acc, bound_acc = R.embed_grad(V, ids, dy, scale, dtype, g0)
    for extra, offset in ((0, 0), (8, 8), (3, 1)):
        d = torch.full((T + 1, D + extra), float("nan"), dtype=R.DT[dtype], device=DEV)[:T, offset:offset + D]
        d.copy_(dy)
        d[(~live).to(DEV)] = float("nan")                   # rows that no sum takes
        grad = nan_like(V, D, dtype=dtype)
        api.rar_embed_grad(V, D, CODE[dtype], T, ids.to(DEV), d, grad, scale)
        R.check(grad, want, bound, f"stride {D + extra}")
        first = grad if first is None else first
        assert torch.equal(grad, first)                     # the order of the terms is the ids' alone
        acc = g0.to(DEV)
        api.rar_embed_grad(V, D, CODE[dtype], T, ids.to(DEV), d, acc, scale, accumulate=True)
        R.check(acc, want_acc, bound_acc, f"stride {D + extra}, accumulated")


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("lead", [0, 1, 31, 1000])
def test_embed_grad_one_token_for_a_batch(lead, dtype):
    # one run over all chunks, its start on and off the borders of chunks and of groups of chunks
    T, V, D = 22001, 6, 1544
    g = torch.Generator().manual_seed(lead)
    dy = torch.randn(T, D, generator=g).to(R.DT[dtype])
    ids = torch.full((T,), 4)
    ids[:lead] = 1
    grad = nan_like(V, D, dtype=dtype)
    api.rar_embed_grad(V, D, CODE[dtype], T, ids.to(DEV), dy.to(DEV), grad)
    want, bound = R.embed_grad(V, ids, dy, 1.0, dtype)
    R.check(grad, want, bound, f"lead {lead}")
