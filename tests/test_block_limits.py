"""Limits of cross attention and log probabilities that keep their arithmetic in
range, without a GPU."""
import pytest

from ring_all_reduce_amd import api
from ring_all_reduce_amd._lib import lib

A = [(i + 1) << 40 for i in range(8)]   # addresses far apart; never dereferenced


@pytest.mark.parametrize("dtype", [api.F32, api.BF16])
def test_scales_that_overflow_are_refused(dtype):
    # log 64 / 1e-38 is more than binary32 holds: every weight of the bf16 gradients would be zero; 3e38 log2 e is too
    for scale in (1e-38, 2.0 ** -101, 2.0 ** 101, 3e38):
        with pytest.raises(api.RarError) as e:
            api.rar_attn_plan(2, 1, 8, dtype, scale)
        assert e.value.status == api.EINVAL
    for scale in (2.0 ** -100, 2.0 ** 100):
        api.rar_attn_plan(2, 1, 8, dtype, scale)
    L = lib()
    for scale, status in ((3e38, api.EINVAL), (2.0 ** 127, api.EINVAL), (2.0 ** 126, api.OK), (1e-45, api.OK)):
        assert L.rar_logprob(0, 100, dtype, A[0], 100, scale, A[1], A[2], 0, 0, 0, 0, None) == status
        assert L.rar_logprob_grad(0, 100, dtype, A[0], 100, scale, A[1], A[2], 0, 0, 0, A[3], 100, None) == status
