"""Tile and split of the linear layer's products, from the header that the
library is built from (host arithmetic, compiled here without HIP)."""
import ctypes
import pathlib
import random
import shutil
import subprocess

import pytest
import torch

import ops_sizes as S
from ring_all_reduce_amd import api
from ring_all_reduce_amd._lib import lib

ROOT = pathlib.Path(__file__).resolve().parents[1]
CODE = {"f32": api.F32, "bf16": api.BF16}


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    """shape(dtype, M, N, K) -> (tile, tiles along M, tiles along N, splits, steps of a split)."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("shape")
    (d / "s.cpp").write_text(
        '#include "linear_shape.h"\n'
        'extern "C" void shape(int dt, int64_t M, int64_t N, int64_t K, int64_t *o)\n'
        '{ const rar::Shape s = rar::shape_of((rar_dtype)dt, M, N, K);\n'
        '  o[0] = s.tile; o[1] = s.tiles_m; o[2] = s.tiles_n; o[3] = s.splits; o[4] = s.steps; }\n')
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{ROOT / 'include'}",
                    f"-I{ROOT / 'ring_all_reduce_amd' / 'csrc'}", str(d / "s.cpp"), "-o", str(d / "s.so")], check=True)
    fn = ctypes.CDLL(str(d / "s.so")).shape
    fn.argtypes = [ctypes.c_int] + [ctypes.c_int64] * 3 + [ctypes.POINTER(ctypes.c_int64)]
    fn.restype = None

    def call(dtype, M, N, K):
        out = (ctypes.c_int64 * 5)()
        fn(CODE[dtype], M, N, K, out)
        return tuple(out)

    return call


# (T, K, N) whose binary32 products of 64-tiles would not share a launch of 2^32 lanes
MANY = [((1 << 24), 32, n) for n in (1000, 1024, 1025, 1088, 1089, 1200, 1300, 1472, 1536)] + [((1 << 24), 1025, 32)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_product_fits_a_launch(shape, dtype):
    rng = random.Random(4)
    cases = [(T, N, K) for T, K, N in MANY] + [(T, K, N) for T, K, N in MANY]
    cases += [(1 << 24, 1 << 13, 1), (1 << 20, 1 << 17, 1 << 20), ((1 << 24) - 1, (1 << 13) + 0, 77), (1, 1, 1)]
    while len(cases) < 3000:
        M, N, K = (int(2 ** rng.uniform(0, b)) for b in (24, 20, 24))
        if M * N <= 1 << 37:
            cases.append((M, N, K))
    for M, N, K in cases:
        tile, tm, tn, splits, steps = shape(dtype, M, N, K)
        large = 256 if dtype == "bf16" else 128
        assert tile in (large, large // 2), (M, N, K)
        lanes = 512 if tile == 256 else 256
        assert tm * tn * splits * lanes < 1 << 32, (M, N, K)
        assert (tm - 1) * tile < M <= tm * tile and (tn - 1) * tile < N <= tn * tile
        step = 64 if dtype == "bf16" else 32
        assert (splits - 1) * steps * step < K <= splits * steps * step


@pytest.mark.skipif(torch.cuda.is_available(), reason="the accepted calls would run on made-up addresses")
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", MANY)
def test_calls_within_the_limits_are_accepted(T, K, N, dtype):
    # without a GPU an accepted call fails at its first launch
    a = [(i + 1) << 50 for i in range(8)]
    plan = api.rar_linear_plan(K, N, CODE[dtype])
    f, b = api.rar_linear_workspace(plan, T)
    assert lib().rar_linear_forward(plan.handle, T, a[0], K, a[1], None, None, N, a[2], N, None, N, None, a[3], f,
                                    None) == api.EHIP
    assert lib().rar_linear_backward(plan.handle, T, a[0], N, a[1], K, None, a[2], None, N, None, a[4], K, a[5], None,
                                     0, a[3], b, None) == api.EHIP


def test_layers_behind_the_limits_are_refused():
    a = [(i + 1) << 56 for i in range(8)]
    for K, N, T in (((1 << 20), (1 << 17) + 1, 1), ((1 << 13) + 1, 8, 1 << 24), (8, (1 << 13) + 1, 1 << 24)):
        for dt in (api.F32, api.BF16):
            plan = api.rar_linear_plan(K, N, dt)
            with pytest.raises(api.RarError) as e:
                api.rar_linear_workspace(plan, T)
            assert e.value.status == api.EINVAL
            assert lib().rar_linear_forward(plan.handle, T, a[0], K, a[1], None, None, N, a[2], N, None, N, None, a[3],
                                            1 << 60, None) == api.EINVAL
            assert lib().rar_linear_backward(plan.handle, T, a[0], N, a[1], K, None, a[2], None, N, None, a[4], K,
                                             a[5], None, 0, a[3], 1 << 60, None) == api.EINVAL
        if T > 1:
            api.rar_linear_workspace(plan, T - (1 << 23))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sizes_of_the_large_tiles(shape, dtype):
    # the GPU tests of the large tiles reach them only as long as this holds
    for (T, K, N), want in S.LINEAR[dtype].items():
        got = tuple(shape(dtype, *p)[::3] for p in ((T, N, K), (T, K, N), (K, N, T)))
        assert got == want, (T, K, N)
    # every large kernel with one and with several splits, and a pair of different tiles
    large = 256 if dtype == "bf16" else 128
    forms = S.LINEAR[dtype].values()
    assert {f[0][1] > 1 for f in forms if f[0][0] == large} == {False, True}
    for k in (1, 2):
        assert {f[k][1] > 1 for f in forms if f[k][0] == large} == {False, True}
    assert len({(f[1][0] == large, f[2][0] == large) for f in forms}) == 4
