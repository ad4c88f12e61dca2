"""Workspaces of the norms and of cross attention, without a GPU: what a call asks
for, and that a workspace for the largest call serves the smaller ones."""
import pytest

from ring_all_reduce_amd import api
from ring_all_reduce_amd._lib import lib

A = [(i + 1) << 40 for i in range(24)]   # addresses far apart; never dereferenced


def forward_bytes(p, *sizes):
    return api.rar_attn_workspace(p, *sizes)[0]


@pytest.mark.parametrize("dtype", [api.F32, api.BF16])
def test_a_token_needs_no_copy_of_its_cache(dtype):
    for H, Hkv, Tq in ((16, 16, 1), (16, 16, 4), (32, 16, 2), (64, 16, 1)):
        p = api.rar_attn_plan(H, Hkv, 128, dtype)
        # at most 64 parts of every row, and their maxima and sums
        for B, Tk in ((1, 100), (1, 1 << 20), (16, 2048), (64, 32768)):
            assert forward_bytes(p, B, Tq, Tk) <= 64 * B * H * Tq * (128 * 4 + 8) + 512
        assert forward_bytes(p, 64, Tq, 32768) <= 1 << 21          # of a cache of 8 GiB and more
        assert forward_bytes(p, 16, Tq, 300) == 0                  # too few keys to cut
        # no workspace is no error then: this call is refused for its address
        w, n = H * 128, Hkv * 128
        assert lib().rar_attn_forward(p.handle, 16, Tq, 300, A[0] + 1, w, A[1], n, A[2], n, 0, 0, A[3], w, 0, 0, 0,
                                      None) == api.EALIGN
    # one row more takes the matrix cores, which read copies of what is not aligned
    p = api.rar_attn_plan(16, 16, 128, dtype)
    es = 4 if dtype == api.F32 else 2
    assert forward_bytes(p, 16, 5, 2048) >= 2 * 16 * 2048 * 16 * 128 * es


def test_norm_workspace_serves_fewer_rows():
    for D in (40, 512, 520, 1024, 2048, 2056, 4096, 8192, 8200, 70_000, 1 << 20):
        p = api.rar_norm_plan(D, api.BF16, api.NORM_LAYER, api.NORM_LAYER)
        last = 0
        for T in [*range(1, 4000), *range(4000, 40_000, 7), 1 << 16, 1 << 20, 1 << 24]:
            n = api.rar_norm_workspace(p, T)
            assert n >= last, (D, T)
            last = n
