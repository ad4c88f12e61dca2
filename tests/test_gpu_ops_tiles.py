"""The linear layer and the embedding's gradient on the GPU at sizes that take
the launch forms of large calls.  Which tile and split a size takes is
asserted from the host's own choice in test_linear_shape.py.  Bounds count
roundings (see ops_ref.py)."""
import pytest
import torch

import ops_ref as R
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
