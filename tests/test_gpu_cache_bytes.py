"""Exponent bytes that dspark_cache_append never writes (0, 254, 255): the read and both
attention kernels take them as the nearest of 1 .. 253."""

import math

import pytest
import torch

from test_gpu_cache import DEV, Batch, code_values

pytestmark = pytest.mark.gpu


def pools(rows, ctx):
    b = Batch(rows, ctx, e4m3=True, seed=1)
    b.q.zero_()  # equal scores: the values' average
    g = torch.Generator().manual_seed(2)
    for pool, exp in ((b.k, b.k_exp), (b.v, b.v_exp)):
        pool[:] = torch.randint(0, 4, pool.shape, generator=g).to(torch.uint8)  # up to 3 * 2^-9
        exp[:] = torch.tensor([0, 1, 253, 254, 255], dtype=torch.uint8)[
            torch.randint(0, 5, exp.shape, generator=g)]
    return b


def clamped(b, n, pool, exp):
    p = torch.arange(b.end[n])
    page, slot = b.tab[n, p // b.page].long(), p % b.page
    return code_values(pool[page, :, slot], exp[page, :, slot].clamp(1, 253))


def test_read(lib):
    b = pools([40, 3], [0, 9]).upload()
    ko, vo = (torch.empty(b.T, b.Hkv, b.D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    b.cache.read(b.d_off, b.d_ctx, b.d_tab, ko, vo, b.ws)
    for out, pool, exp in ((ko, b.k, b.k_exp), (vo, b.v, b.v_exp)):
        for n in range(b.R):
            want = clamped(b, n, pool, exp)[b.ctx[n]:]
            got = out[b.off[n]:b.off[n + 1]].cpu().double()
            # 2^-126 times a small code is below bf16's subnormals: at most half of one off
            assert ((got == want) | ((want < 2.0 ** -126) & ((got - want).abs() <= 2.0 ** -134))
                    ).all()


@pytest.mark.parametrize("rows,ctx", [([1, 3], [5, 30]), ([40], [9])])
def test_attention(lib, rows, ctx):
    b = pools(rows, ctx).upload()
    out, lse = b.attend()
    for n in range(b.R):
        v = clamped(b, n, b.v, b.v_exp).repeat_interleave(b.G, 1)
        for j in range(b.rows[n]):
            seen = b.ctx[n] + j + 1
            want = v[:seen].mean(0)
            got = out[b.off[n] + j].cpu().double()
            # bf16's rounding, and fp32 sums of a few positive terms
            assert ((got - want).abs() <= 2.0 ** -7 * want + 1e-30).all()
            assert (lse[b.off[n] + j].cpu().double() - math.log(seen)).abs().max() < 1e-5
