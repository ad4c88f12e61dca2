"""Log probabilities, alternatives and gradients of every kernel by the number of
logits, with more rows than its grid: rows of ties, masks, NaN and ordinary rows
follow one another in the same workgroups."""
import math

import pytest
import torch

import block_ref as R
from ring_all_reduce_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CODE = {"f32": api.F32, "bf16": api.BF16}
INF, NAN = math.inf, math.nan

# (T, V): rows on 64 and 256 lanes; more than 512 rows of up to four, six and eight eights on 512 lanes; rows on 1024
# lanes, in registers and, over 65536 (bf16: 131072), read again
SHAPES = [(9001, 300), (4300, 3000), (1103, 8200), (1103, 16384), (1103, 16385), (1103, 24576), (1103, 24577),
          (1103, 32768), (601, 40_000), (601, 60_003), (601, 100_000), (530, 140_000)]


def same_bits(a, b):
    i = {2: torch.int16, 4: torch.int32, 8: torch.int64}[a.element_size()]
    return bool((a.contiguous().view(i) == b.contiguous().view(i)).all())


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_behind_one_another(shape, dtype):
    T, V = shape
    K, N = 20, 23
    g = torch.Generator().manual_seed(V)
    z = (torch.randn(N, V, generator=g) * 3).to(R.DT[dtype])
    z[0] = 1.5                                        # all alike
    z[3] = torch.arange(V).float().to(z.dtype)        # rising (in bf16 with long runs of ties)
    z[5] = -torch.arange(V).float().to(z.dtype)
    z[8] = -INF
    z[8, 7], z[8, V - 1] = 0.0, -0.0                  # two are left, and they tie
    z[9] = -INF                                       # nothing is left
    z[12, ::2] = torch.finfo(z.dtype).min
    z[14, 1::3] = -INF
    z[17] = (z[17] / 4).round().clamp(-1, 1)          # three values
    z[19, 3] = NAN
    z[20, 4] = INF
    t = torch.randint(0, V, (N,), generator=g)
    t[6] = -1
    # (the number of rows that a grid takes at once is no multiple of 23: different rows follow one another)
    at = (torch.arange(T) % N).to(DEV)
    zs, ts = z.to(DEV)[at], t.to(DEV)[at]
    logp, ent, top = (torch.full(s, NAN, device=DEV) for s in ((T,), (T,), (T, K)))
    ids = torch.full((T, K), -7, device=DEV)
    api.rar_logprob(T, V, CODE[dtype], zs, ts, logp, ent, top_ids=ids, top_logp=top)
    dl, de = torch.randn(N, generator=g), torch.randn(N, generator=g)
    dz = torch.full_like(zs, NAN)
    api.rar_logprob_grad(T, V, CODE[dtype], zs, ts, dl.to(DEV)[at], de.to(DEV)[at], dz)
    # a row's results do not depend on where it stands
    for name, x in (("logp", logp), ("entropy", ent), ("ids", ids), ("top", top), ("dz", dz)):
        for first in range(0, T, 100):
            n = min(100, T - first)
            assert same_bits(x[first:first + n], x[at[first:first + n]]), (name, first)
    ok = torch.tensor([i for i in range(N) if i not in (9, 14, 19, 20)])
    logp, ent, ids, top, dz = (x[:N].cpu() for x in (logp, ent, ids, top, dz))
    good = torch.tensor([i for i in range(N) if i not in (19, 20)])
    ri, rt, et = R.top(z[good], 1.0, K)
    assert (ids[good] == ri).all()
    on = ri >= 0
    assert (top[good][~on] == -INF).all()
    R.check(torch.where(on, top[good], 0.0), torch.where(on, rt, 0.0), et, "alternatives")
    assert (ids[19:21] == -1).all() and torch.isnan(top[19:21]).all() and torch.isnan(logp[19:21]).all()
    assert logp[9] == -INF and ent[9] == 0 and (dz[9] == 0).all() and torch.isnan(dz[19:21]).all()
    (rl, el), (re, ee) = R.logprob(z[ok], t[ok], 1.0)
    R.check(logp[ok], rl, el, "logp")
    R.check(ent[ok], re, ee, "entropy")
    want, bound = R.logprob_grad(z[ok], t[ok], dl[ok], de[ok], 1.0, dtype)
    R.check(dz[ok], want, bound, "dz")
