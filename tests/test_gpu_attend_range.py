"""dspark_attend over values of any size: an exponential that has passed its row's reference
times a large value stays finite, and queries of any size keep their bits.  At the tolerance
that test_gpu_cache.py derives."""

import pytest
import torch

from test_gpu_attend_moves import grown
from test_gpu_cache import FMT, Batch, quantise

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


@FMT
@pytest.mark.parametrize("rows,ctx", [([1, 3], [300, 40]), ([8], [200]), ([40], [50])])
@pytest.mark.parametrize("octaves", [-118, -105, 60])
def test_queries_and_keys_far_apart(lib, octaves, rows, ctx, e4m3):
    """q times 2^octaves, k divided by it: the scores are those of ordinary sizes."""
    b = Batch(rows, ctx, e4m3=False, seed=11)
    b.q = (b.q.double() * 2.0 ** octaves).bfloat16()
    b.k = (b.k.double() * 2.0 ** -octaves).bfloat16()
    assert torch.isfinite(b.k).all() and (b.q != 0).float().mean() > 0.9
    if e4m3:
        b.e4m3 = True
        b.k, b.k_exp = quantise(b.k)
        b.v, b.v_exp = quantise(b.v)
    b.upload()
    b.check(*b.attend())
