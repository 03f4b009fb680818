"""dspark_attend over values of any size: an exponential that has passed its row's reference
times a large value stays finite.  At the tolerance that test_gpu_cache.py derives."""

import pytest

from test_gpu_attend_moves import grown
from test_gpu_cache import FMT, quantise

pytestmark = pytest.mark.gpu


@FMT
@pytest.mark.parametrize("rows,ctx", [([1, 1], [2900, 700]), ([8, 5], [1500, 400]), ([40], [900])])
@pytest.mark.parametrize("size", [1e15, 1e25])
def test_large_values_under_growing_scores(lib, size, rows, ctx, e4m3):
    b = grown(rows, ctx, 4, 32, False, octaves=9, seed=7)
    b.v = (b.v.float() * size).bfloat16()
    if e4m3:
        b.e4m3 = True
        b.k, b.k_exp = quantise(b.k)
        b.v, b.v_exp = quantise(b.v)
    b.upload()
    b.check(*b.attend())
