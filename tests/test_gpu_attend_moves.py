"""dspark_attend where the scores grow along the context: the softmax's references
move again and again, by far more than the range of the probabilities' type, in both
kernels and both cache formats.  Compared with the plain 64-bit form, at the tolerance
that test_gpu_cache.py derives."""

import pytest
import torch

from test_gpu_cache import Batch, quantise

pytestmark = pytest.mark.gpu


def grown(rows, ctx, G, page, e4m3, octaves, seed):
    """A batch whose keys grow by 2^octaves from each request's first position to its
    last, from 2^-6 on (the largest scores then differ by hundreds of powers of two)."""
    b = Batch(rows, ctx, G=G, page=page, seed=seed)
    for n in range(b.R):
        p = torch.arange(b.end[n])
        at, slot = b.tab[n, p // page].long(), p % page
        f = torch.exp2(-6 + octaves * p / max(1, b.end[n] - 1)).bfloat16()
        b.k[at, :, slot] = b.k[at, :, slot] * f.view(-1, 1, 1)
    if e4m3:
        b.e4m3 = True
        b.k, b.k_exp = quantise(b.k)
        b.v, b.v_exp = quantise(b.v)
    return b.upload()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows,ctx,G,page", [
    ([1, 1, 1], [2900, 700, 5], 4, 16),     # one eight of rows
    ([4, 3], [1500, 130], 4, 32),           # two
    ([8, 8, 2, 5], [3000, 260, 40, 0], 4, 64),  # four
    ([40, 9], [1700, 300], 4, 128),         # more than 32 rows a head, both modes
    ([70], [900], 4, 16),
])
def test_scores_that_grow(lib, rows, ctx, G, page, e4m3):
    b = grown(rows, ctx, G, page, e4m3, octaves=11, seed=len(rows))
    b.check(*b.attend())
    assert b.cache.status(b.ws) == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows", [[6, 8, 1], [50]])
def test_growth_seen_through_a_window(lib, rows, e4m3):
    b = grown(rows, [1000, 333, 2000][: len(rows)], 4, 32, e4m3, octaves=11, seed=9)
    b.check(*b.attend(window=200), window=200)


def test_results_repeat(lib):
    """Moved references and split items: the same bits every time."""
    b = grown([8, 8, 8], [3000, 2000, 1000], 4, 16, True, octaves=11, seed=2)
    first = b.attend()
    for _ in range(10):
        again = b.attend()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_equal_scores(lib):
    """Queries of zeros: every visible position counts the same."""
    b = Batch([3, 40], [200, 300], seed=4)
    b.q[:] = 0
    b.upload()
    b.check(*b.attend())
