"""Workspaces of the norms and of cross attention, without a GPU: what a call asks
for, and that a workspace for the largest call serves the smaller ones."""
import ctypes
import pathlib
import random
import shutil
import subprocess

import pytest

from ring_all_reduce_amd import api
from ring_all_reduce_amd._lib import lib

ROOT = pathlib.Path(__file__).resolve().parents[1]
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


def test_attention_workspace_serves_fewer_sequences_queries_and_keys():
    rng = random.Random(7)
    for H, Hkv, dh, dt in ((16, 4, 64, api.BF16), (8, 8, 128, api.F32), (6, 3, 60, api.F32), (16, 16, 128, api.BF16),
                           (1, 1, 8, api.BF16), (64, 1, 128, api.F32)):
        p = api.rar_attn_plan(H, Hkv, dh, dt)

        def grows(sizes):
            last = (0, 0)
            for size in sizes:
                n = api.rar_attn_workspace(p, *size)
                assert n[0] >= last[0] and n[1] >= last[1], (H, Hkv, dh, dt, size)
                last = n

        for Tq, Tk in ((512, 512), (1, 2048), (40, 300), (9, 4096), (2000, 64)):
            grows([(B, Tq, Tk) for B in range(1, 300)])
            grows([(3, n, Tk) for n in range(0, 1500)])
            grows([(3, Tq, n) for n in range(0, 3000, 3)])
        for _ in range(300):
            size = [1, 1, 1]
            walk = []
            while size[0] * max(size[1:]) < 1 << 16:
                walk.append(tuple(size))
                i = rng.randrange(3)
                size[i] += 1 + int(size[i] * rng.random())
            grows(walk)


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    """cut(H, Hkv, dh, dtype, B, Tq, Tk) -> rows that the parts of o, dq and dk (and dv) take, and room for each."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("cut")
    (d / "s.cpp").write_text(
        '#include "attn_shape.h"\n'
        'extern "C" void cut(int64_t H, int64_t Hkv, int64_t dh, int dt, int64_t B, int64_t Tq, int64_t Tk,\n'
        '                    int64_t *o)\n'
        '{ const rar::AttnShape s(H, Hkv, dh, (rar_dtype)dt, B, Tq, Tk);\n'
        '  o[0] = s.splits > 1 ? s.splits * s.part_rows() : 0; o[1] = s.part_room();\n'
        '  o[2] = s.q_splits > 1 ? s.q_splits * s.part_rows() : 0; o[3] = s.q_room();\n'
        '  o[4] = s.k_splits > 1 ? s.k_splits * B * Hkv * Tk : 0; o[5] = s.k_room(); }\n')
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{ROOT / 'include'}",
                    f"-I{ROOT / 'ring_all_reduce_amd' / 'csrc'}", str(d / "s.cpp"), "-o", str(d / "s.so")], check=True)
    fn = ctypes.CDLL(str(d / "s.so")).cut
    fn.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] + [ctypes.c_int64] * 3 + [ctypes.POINTER(ctypes.c_int64)]
    fn.restype = None

    def call(*a):
        out = (ctypes.c_int64 * 6)()
        fn(*a, out)
        return tuple(out)

    return call


def test_parts_stay_in_their_room(cut):
    rng = random.Random(8)
    cuts = 0
    for _ in range(200_000):
        Hkv = int(2 ** rng.uniform(0, 7))
        share = rng.choice([1, 1, 2, 3, 4, 8, 33])
        B, Tq, Tk = (int(2 ** rng.uniform(0, b)) for b in (9, 13, 18))
        size = (Hkv * share, Hkv, rng.randint(1, 128), rng.randint(0, 1), B, rng.choice([1, 2, Tq, Tq]), Tk)
        n = cut(*size)
        cuts += n[0] > 0
        assert n[0] <= n[1] and n[2] <= n[3] and n[4] <= n[5], (size, n)
    assert cuts > 10_000


def test_attention_takes_every_size_that_its_launches_do():
    def bytes_of(H, Hkv, dh, *size):
        p = api.rar_attn_plan(H, Hkv, dh, api.BF16)
        return api.rar_attn_workspace(p, *size)

    # caches of 32 GiB and more: copies of them would take lanes beyond 2^32 if each had one group
    assert bytes_of(16, 16, 128, 64, 1, 1 << 17)[0] <= 1 << 21
    assert bytes_of(64, 64, 128, 16, 1, 1 << 20)[0] <= 1 << 23
    assert bytes_of(16, 16, 128, 1, 5, 1 << 24)[0] >= 2 << 36
    # both sides of the limits that rar.h names
    for good, bad in (((128, 128, 8, 65535, 1, 1), (129, 129, 8, 65535, 1, 1)),
                      ((2048, 2048, 8, 4, 1 << 15, 1), (4096, 4096, 8, 4, 1 << 15, 1)),
                      ((127, 127, 8, 1, 1, 1 << 24), (128, 128, 8, 1, 1, 1 << 24)),
                      ((31, 1, 8, 1, 1 << 24, 1), (32, 1, 8, 1, 1 << 24, 1))):
        bytes_of(*good)
        with pytest.raises(api.RarError) as e:
            bytes_of(*bad)
        assert e.value.status == api.EINVAL
