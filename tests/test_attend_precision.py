"""How exact dspark_attend is: probabilities of 16 bits however small they are, sums that
lose nothing.

Tolerances, derived from the formula.  With p the exact probabilities, w = sum_c p_c |v_c|,
and d_c what the score of position c may be off by:
  * the result is rounded once to bf16 (8 bits):          2^-8 |o|
  * each p_c enters its product with 16 bits:             2^-16 w
  * a score is an fp32 sum of D exact products, off by at most d_c = 2^-22 D scale
    max|q| max|k_c| (2^-22 a term: a tensor core may truncate; twice that over e4m3, where
    q is two codes, down to 2^-21 of its row's largest).  That moves p_c by the factor
    1 +- d_c, and the sum of exponentials by sum p_c d_c:  sum p_c d_c |v_c| + |o| sum p_c d_c
  * O is an fp32 sum of L / 16 products of 16 positions, each addition off by 2^-23 of a
    partial sum at most, and of the sixteen's own; the exponentials' sum likewise:
    (L / 16 + 64) 2^-23 w
lse: sum p_c d_c, the sums' (L / 16 + 64) 2^-23, and 2^-20 of its size or of 1."""

import math

import pytest
import torch

from test_gpu_cache import FMT, Batch, quantise


def bounds(q, k, v, at, causal, scale, e4m3):
    """One request in 64 bits, q [m, Hq, D], k, v [L, Hkv, D]: o, lse, their tolerances, and
    p [Hq][m, L]."""
    m, Hq, D = q.shape
    L, Hkv, _ = k.shape
    see = torch.ones(m, L, dtype=torch.bool)
    if causal:
        see = torch.arange(L) <= at + torch.arange(m).view(-1, 1)
    sums = (L / 16 + 64) * 2.0 ** -23
    o, tol, lse, lse_tol, ps = [], [], [], [], []
    for h in range(Hq):
        kh, vh, qh = k[:, h // (Hq // Hkv)], v[:, h // (Hq // Hkv)], q[:, h]
        x = (qh @ kh.T * scale).masked_fill(~see, -math.inf)
        z = torch.logsumexp(x, 1, keepdim=True)
        p = torch.exp(x - z)
        d = (2.0 ** -22 * D * scale * (2 if e4m3 else 1)) * (
            qh.abs().amax(1, keepdim=True) * kh.abs().amax(1))
        pd = (p * d).sum(1, keepdim=True)
        oh, w = p @ vh, p @ vh.abs()
        o.append(oh)
        tol.append(2.0 ** -8 * oh.abs() + (2.0 ** -16 + sums) * w + (p * d) @ vh.abs()
                   + oh.abs() * pd + 1e-30)
        lse.append(z[:, 0])
        lse_tol.append(pd[:, 0] + sums + 2.0 ** -20 * z[:, 0].abs().clamp(min=1))
        ps.append(p)
    return *(torch.stack(t, 1) for t in (o, tol, lse, lse_tol)), ps


def check(b, out, lse, causal=True):
    out, lse = out.cpu().double(), lse.cpu().double()
    for n in range(b.R):
        a, m = b.off[n], b.rows[n]
        o, tol, z, z_tol, _ = bounds(b.q[a:a + m].double(), b.values(n, b.k, b.k_exp),
                                     b.values(n, b.v, b.v_exp), b.ctx[n], causal,
                                     1 / math.sqrt(b.D), b.e4m3)
        worst = ((out[a:a + m] - o).abs() / tol).max().item()
        assert worst <= 1, (n, m, b.ctx[n], worst)
        worst = ((lse[a:a + m] - z).abs() / z_tol).max().item()
        assert worst <= 1, ("lse", n, m, b.ctx[n], worst)


def to_codes(b):
    b.e4m3 = True
    b.k, b.k_exp = quantise(b.k)
    b.v, b.v_exp = quantise(b.v)
    return b


def opposed(rows, ctx, e4m3, G=4, seed=0):
    """Few positions, all of about the same weight, whose values nearly cancel: the
    probabilities' own rounding is what is left."""
    b = Batch(rows, ctx, G=G, e4m3=False, seed=seed, q_gain=0.3)
    g = torch.Generator().manual_seed(seed + 1)
    for n in range(b.R):
        p = torch.arange(b.end[n])
        page, slot = b.tab[n, p // b.page].long(), p % b.page
        b.k[page, :, slot] = (0.3 * torch.randn(len(p), b.Hkv, b.D, generator=g)).bfloat16()
        sign = 1.0 - 2.0 * (p % 2).view(-1, 1, 1)
        b.v[page, :, slot] = (sign * (1 + 0.05 * torch.randn(len(p), b.Hkv, b.D, generator=g))
                              ).bfloat16()
    return to_codes(b) if e4m3 else b


OPPOSED = [([1, 1, 1, 2], [3, 5, 9, 6]), ([6, 8], [0, 2]), ([12, 16], [0, 4])]


@pytest.mark.gpu
@FMT
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("rows,ctx", OPPOSED)
def test_probabilities_have_sixteen_bits(lib, rows, ctx, causal, e4m3):
    b = opposed(rows, ctx, e4m3).upload()
    check(b, *b.attend(causal=causal), causal=causal)


@pytest.mark.parametrize("rows,ctx", OPPOSED)
def test_one_rounding_of_the_probabilities_would_show(rows, ctx):
    """The tolerance tells one bf16 rounding of P from two terms (plain form, no GPU)."""
    b = opposed(rows, ctx, False)
    worst = {1: 0.0, 2: 0.0}
    for n in range(b.R):
        a, m = b.off[n], b.rows[n]
        v = b.values(n, b.v, None)
        o, tol, _, _, ps = bounds(b.q[a:a + m].double(), b.values(n, b.k, None), v, b.ctx[n],
                                  False, 1 / math.sqrt(b.D), False)
        for terms in worst:
            for h, p in enumerate(ps):
                x = p / p.amax(1, keepdim=True)
                r = torch.zeros_like(x)
                for _ in range(terms):
                    r = r + (x - r).float().bfloat16().double()
                got = ((r @ v[:, h // b.G]) / x.sum(1, keepdim=True)).float().bfloat16().double()
                worst[terms] = max(worst[terms],
                                   ((got - o[:, h]).abs() / tol[:, h]).max().item())
    assert worst[2] <= 1 and worst[1] > 2, worst


@pytest.mark.gpu
@FMT
@pytest.mark.parametrize("rows,ctx", [([1, 1], [700, 2100]), ([8, 3], [900, 2000]), ([40], [600]),
                                      ([300], [100])])
def test_ordinary_rows(lib, rows, ctx, e4m3):
    b = Batch(rows, ctx, q_gain=0.5, e4m3=e4m3, page=32, seed=3).upload()
    check(b, *b.attend())


@pytest.mark.gpu
@FMT
@pytest.mark.parametrize("rows", [1, 8, 12])
@pytest.mark.parametrize("L,nats", [(8192, 16.0), (65536, 15.0), (65536, 17.0)])
def test_a_tail_far_below_one_position(lib, L, nats, rows, e4m3):
    """The first position takes nearly all of the weight but has values in eight of the
    dimensions only: the others' outputs are the sum of all the small probabilities.  As many
    requests as blocks hold whole items, all over the same pages."""
    b = Batch([rows], [L - rows], Hkv=1, G=4, page=64, seed=rows, spare_pages=0)
    g = torch.Generator().manual_seed(L)
    n, D = 160, b.D
    q = 0.5 * torch.randn(n * rows, b.Hq, D, generator=g)
    q[..., 0] = 8.0
    b.q = q.bfloat16()
    k = 0.3 * torch.randn(L, 1, D, generator=g)
    k[:, :, 0] = 0.0
    k[0, 0, 0] = nats * math.sqrt(D) / 8.0
    v = 1 + 0.5 * torch.randn(L, 1, D, generator=g)
    v[0] = 0.0
    v[0, :, :8] = 1.0
    p = torch.arange(L)
    page, slot = b.tab[0, p // b.page].long(), p % b.page
    b.k[page, :, slot], b.v[page, :, slot] = k.bfloat16(), v.bfloat16()
    if e4m3:
        to_codes(b)
    b.R, b.T, b.rows, b.ctx, b.end = n, n * rows, [rows] * n, [L - rows] * n, [L] * n
    b.off = [rows * i for i in range(n + 1)]
    b.tab = b.tab.repeat(n, 1)
    b.upload()
    out, lse = b.attend()
    b.R = 20  # of the same kind, the rest
    check(b, out, lse)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


@pytest.mark.gpu
@FMT
@pytest.mark.parametrize("rows,ctx", [([1, 3], [20, 300]), ([40], [200])])
def test_values_of_very_different_sizes(lib, rows, ctx, e4m3):
    """Rows of zeros beside rows of 1e11, equal scores: every position counts in the sum."""
    b = Batch(rows, ctx, e4m3=False, seed=5)
    b.q.zero_()
    b.v[:] = (b.v.float() * 1e11).bfloat16()
    b.v[:, :, ::2] = 0
    if e4m3:
        to_codes(b)
    b.upload()
    check(b, *b.attend())
