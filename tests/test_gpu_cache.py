"""The paged key/value cache and its attention against plain 64-bit forms, at
the sizes, lengths and masks where they can go wrong.

Tolerances of the attention, from the formula.  With w = sum_c p_c |v_c| and p
the exact probabilities:
  * the result is rounded once to bf16:           2^-9 |o|
  * each p_c is rounded to 16 bits (bf16 at the coarsest): at most 2^-9 w
  * a score is an fp32 sum of D exact products; with 2^-22 a term (a tensor
    core may truncate) it is off by at most d = 2^-22 D scale max|q| max|k|,
    which moves p_c by at most the factor 1 +- 2d (numerator and sum): 2 d w
  * exponentials and fp32 sums of up to 2^15 terms: 2^-14 w
lse: d, and 2^-20 of its size or of 1 for the sum and the logarithm."""

import ctypes
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


# ---------------------------------------------------------------- plain forms


def pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def code_values(codes, exp):
    """64-bit values of e4m3 codes (uint8) with exponent bytes."""
    u = codes.long()
    e, f = (u >> 3) & 15, (u & 7).double()
    mag = torch.where(e == 0, f / 512, (1 + f / 8) * pow2(e - 7))
    return torch.where(u >= 128, -mag, mag) * pow2(exp.long() - 127).unsqueeze(-1)


def quantise(x):
    """(codes, exponent bytes) of rows of finite values, by search for the nearest code."""
    x = x.double()
    amax = x.abs().amax(-1)
    e = torch.full_like(amax, -100)
    for k in range(-100, 121):  # the smallest exponent that holds the row
        e = torch.where((448 * 2.0 ** k < amax) & (e == k), torch.full_like(e, k + 1), e)
    y = x / pow2(e).unsqueeze(-1)
    grid = code_values(torch.arange(127).to(torch.uint8).view(1, -1),
                       torch.tensor([127])).reshape(-1)
    i = torch.searchsorted(grid, y.abs().contiguous()).clamp(1, 126)
    lo, hi = grid[i - 1], grid[i]
    up = (y.abs() - lo > hi - y.abs()) | ((y.abs() - lo == hi - y.abs()) & (i % 2 == 0))
    code = torch.where(up, i, i - 1)
    sign = torch.signbit(y)
    return (code + 128 * sign).to(torch.uint8), (e + 127).to(torch.uint8)


def attention(q, k, v, at, causal, window, scale):
    """One request: q [m, Hq, D], k, v [L, Hkv, D] (64 bits), first position at.
    Returns o, lse, and w = sum p |v| (the scale of its error)."""
    m, Hq, D = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    pos = at + torch.arange(m).view(-1, 1)
    c = torch.arange(L).view(1, -1)
    see = torch.ones(m, L, dtype=torch.bool)
    if causal:
        see = c <= pos
        if window:
            see &= c > pos - window
    o, lse, w = (torch.zeros(m, Hq, D, dtype=torch.float64),
                 torch.full((m, Hq), -math.inf, dtype=torch.float64),
                 torch.zeros(m, Hq, D, dtype=torch.float64))
    rows = see.any(1)
    for h in range(Hq):
        x = (q[:, h] @ k[:, h // G].T * scale).masked_fill(~see, -math.inf)[rows]
        if x.numel() == 0:
            continue
        z = torch.logsumexp(x, 1, keepdim=True)
        p = torch.exp(x - z)
        # positions that a row does not see are no part of its sum
        o[rows, h] = p @ v[:, h // G].nan_to_num(0.0)
        w[rows, h] = p @ v[:, h // G].nan_to_num(0.0).abs()
        lse[rows, h] = z[:, 0]
    return o, lse, w


# ---------------------------------------------------------------- fixtures


class Batch:
    """A batch of requests on a cache of scattered pages, inputs on the CPU and the GPU."""

    def __init__(self, rows, ctx, Hkv=2, G=4, D=128, page=16, e4m3=False, seed=0, spare_pages=3,
                 q_gain=1.5):
        from draft_sampling_lossless_gb300.cache import PagedCache

        g = torch.Generator().manual_seed(seed)
        self.rows, self.ctx, self.Hkv, self.G, self.D, self.page, self.e4m3 = (
            rows, ctx, Hkv, G, D, page, e4m3)
        self.R, self.T, self.Hq = len(rows), sum(rows), Hkv * G
        self.end = [max(0, c + m) for c, m in zip(ctx, rows)]
        need = [-(-e // page) for e in self.end]
        self.n_pages = sum(need) + spare_pages
        ids = torch.randperm(self.n_pages, generator=g).tolist()
        self.tab = torch.full((self.R, max(1, max(need))), -1, dtype=torch.int32)
        for n in range(self.R):
            for i in range(need[n]):
                self.tab[n, i] = ids.pop()
        off = [0]
        for m in rows:
            off.append(off[-1] + m)
        self.off = off
        shape = (self.n_pages, Hkv, page, D)
        size = torch.exp(0.5 * torch.randn((2,) + shape[:3] + (1,), generator=g))
        self.k, self.v = (torch.randn(shape, generator=g).mul(x).bfloat16() for x in size)
        self.k_exp = self.v_exp = None
        if e4m3:
            self.k, self.k_exp = quantise(self.k)
            self.v, self.v_exp = quantise(self.v)
        self.q = (torch.randn(max(1, self.T), self.Hq, D, generator=g) * q_gain).bfloat16()[: self.T]
        self._cls = PagedCache

    def upload(self):
        to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        self.cache = self._cls(to(self.k), to(self.v), to(self.k_exp), to(self.v_exp))
        self.d_off = torch.tensor(self.off, dtype=torch.int32, device=DEV)
        self.d_ctx = torch.tensor(self.ctx, dtype=torch.int32, device=DEV)
        self.d_tab = self.tab.to(DEV)
        self.ws = self.cache.workspace(self.R, self.T, self.Hq)
        return self

    def values(self, n, pool, exp):
        """64-bit cached values of request n, [end, Hkv, D]."""
        p = torch.arange(self.end[n])
        page, slot = self.tab[n, p // self.page].long(), p % self.page
        x = pool[page, :, slot]
        return x.double() if exp is None else code_values(x, exp[page, :, slot])

    def attend(self, causal=True, window=0, q=None, max_rows=None, **kw):
        q = self.q.to(DEV) if q is None else q
        out = torch.full((self.T, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((self.T, self.Hq), 7.0, dtype=torch.float32, device=DEV)
        self.cache.attend(q, self.d_off, self.d_ctx, self.d_tab, out, lse=lse, causal=causal,
                          window=window, max_rows=max(self.rows) if max_rows is None else max_rows,
                          ws=self.ws, **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, causal=True, window=0):
        out, lse = out.cpu().double(), lse.cpu().double()
        scale = 1 / math.sqrt(self.D)
        for n in range(self.R):
            a, m = self.off[n], self.rows[n]
            if m == 0:
                continue
            k, v = self.values(n, self.k, self.k_exp), self.values(n, self.v, self.v_exp)
            o, z, w = attention(self.q[a:a + m].double(), k, v, self.ctx[n], causal, window, scale)
            kmax = k.nan_to_num(0.0).abs().max().item() if k.numel() else 0.0
            d = 2.0 ** -22 * self.D * scale * self.q.abs().max().item() * kmax
            tol = 2.0 ** -9 * o.abs() + (2.0 ** -9 + 2 * d + 2.0 ** -14) * w + 1e-30
            bad = (out[a:a + m] - o).abs() > tol
            assert not bad.any(), (n, m, self.ctx[n], int(bad.sum()),
                                   ((out[a:a + m] - o).abs() / tol).max().item())
            empty = z == -math.inf
            assert (lse[a:a + m][empty] == -math.inf).all()
            assert (out[a:a + m][empty] == 0).all()
            off = (lse[a:a + m] - z)[~empty].abs()
            assert (off <= d + 2.0 ** -20 * z[~empty].abs().clamp(min=1)).all(), (n, off.max())


def ragged(seed, R, rows, ctx):
    r = random.Random(seed)
    return [r.randint(*rows) for _ in range(R)], [r.randint(*ctx) for _ in range(R)]


FMT = pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])

# ---------------------------------------------------------------- attention


@FMT
@pytest.mark.parametrize("D", [16, 48, 64, 80, 128])
def test_single_tokens_of_every_length(lib, D, e4m3):
    """One row a request, around the edges of pages (16) and of tiles (powers of two)."""
    ctx = [0, 1, 14, 15, 16, 31, 62, 63, 64, 126, 127, 128, 129, 255, 256, 383, 500, 1023]
    b = Batch([1] * len(ctx), ctx, D=D, e4m3=e4m3).upload()
    b.check(*b.attend())
    assert b.cache.status(b.ws) == 0


@FMT
@pytest.mark.parametrize("G,rows", [(1, (1, 8)), (3, (1, 8)), (4, (0, 8)), (5, (2, 13)), (7, (1, 17)),
                                    (8, (8, 8)), (16, (1, 8)), (32, (1, 4)), (128, (1, 1)),
                                    (128, (1, 3))])
def test_verify_rows_for_every_group(lib, G, rows, e4m3):
    """Ragged rows of 7 requests (some without any), 1 to 384 packed rows a head."""
    m, ctx = ragged(G, 7, rows, (0, 700))
    b = Batch(m, ctx, Hkv=2, G=G, page=32, e4m3=e4m3, seed=G).upload()
    b.check(*b.attend(max_rows=rows[1]))
    assert b.cache.status(b.ws) == 0


@FMT
@pytest.mark.parametrize("rows,ctx,page,G,D", [
    ([65], [0], 16, 1, 64), ([129], [3], 16, 1, 128), ([300], [0], 64, 4, 128),
    ([257, 1, 40], [100, 900, 0], 128, 3, 96), ([511], [1000], 256, 2, 128), ([77, 350], [5, 130], 1024, 5, 64)])
def test_chunks(lib, rows, ctx, page, G, D, e4m3):
    """More packed rows than a tile has, beside short requests in the same batch."""
    b = Batch(rows, ctx, Hkv=2, G=G, D=D, page=page, e4m3=e4m3, seed=sum(rows)).upload()
    b.check(*b.attend())


@FMT
@pytest.mark.parametrize("rows", [(7, 7), (1, 9), (90, 200)])
def test_blocks_that_see_each_other(lib, rows, e4m3):
    m, ctx = ragged(3, 5, rows, (0, 300))
    b = Batch(m, ctx, e4m3=e4m3, page=64, seed=5).upload()
    b.check(*b.attend(causal=False), causal=False)


@FMT
@pytest.mark.parametrize("window", [1, 2, 17, 128, 200, 5000])
def test_windows(lib, window, e4m3):
    m, ctx = ragged(window, 6, (1, 60), (0, 900))
    b = Batch(m + [150], ctx + [40], e4m3=e4m3, seed=window).upload()
    b.check(*b.attend(window=window), window=window)


@FMT
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing(lib, causal, e4m3):
    """Padding rows (negative positions), wholly or partly; requests without rows
    or without anything cached."""
    rows, ctx = [5, 4, 0, 3, 0, 40, 2], [-2, -4, 0, -9, 50, -39, 0]
    b = Batch(rows, ctx, e4m3=e4m3, spare_pages=2).upload()
    b.check(*b.attend(causal=causal), causal=causal)
    assert b.cache.status(b.ws) == 0


@FMT
@pytest.mark.parametrize("rows,Hkv", [([1], 1), ([8], 2), ([3, 1], 1)])
def test_long_contexts_are_split_and_joined(lib, rows, Hkv, e4m3):
    ctx = [20011, 9001][: len(rows)]
    b = Batch(rows, ctx, Hkv=Hkv, page=128, e4m3=e4m3, seed=9).upload()
    b.check(*b.attend())


@FMT
def test_long_chunk_is_split_and_joined(lib, e4m3):
    """256-row tiles shared between blocks: few tiles, a long axis."""
    b = Batch([120], [9000], Hkv=1, G=4, page=64, e4m3=e4m3, seed=2).upload()
    b.check(*b.attend())


@FMT
def test_peaked_scores_and_growing_maxima(lib, e4m3):
    """Large scores that grow along the context, so that the running maximum moves often."""
    b = Batch([8, 100], [900, 300], e4m3=e4m3, q_gain=12.0, seed=4)
    if not e4m3:
        for n in range(2):
            for i in range(b.end[n] // b.page):
                b.k[b.tab[n, i].long()] *= 0.2 + 0.05 * i
    b.upload()
    b.check(*b.attend())


@FMT
def test_equal_scores_average_the_values(lib, e4m3):
    b = Batch([4, 70], [333, 60], e4m3=e4m3, seed=6)
    b.q.zero_()
    b.upload()
    out, lse = b.attend()
    b.check(out, lse)
    n_seen = torch.tensor([334 + i for i in range(4)]).double().log()
    assert (lse[:4, 0].cpu().double() - n_seen).abs().max() < 1e-5


@FMT
@pytest.mark.parametrize("rows,window", [([1, 8, 3], 0), ([100, 300, 1], 0), ([20, 9, 1], 33)])
def test_what_no_row_sees_is_never_used(lib, rows, window, e4m3):
    """NaN and infinities in every slot that no row of its request sees: other pages,
    the rest of the last page, what lies before the window."""
    b = Batch(rows, [130, 77, 1000], page=32, e4m3=e4m3, seed=8)
    keep = torch.zeros(b.n_pages, b.page, dtype=torch.bool)
    for n in range(b.R):
        lo = max(0, b.ctx[n] + 1 - window) if window else 0
        p = torch.arange(lo, b.end[n])
        keep[b.tab[n, p // b.page].long(), p % b.page] = True
    hide = ~keep.unsqueeze(1).expand(-1, b.Hkv, -1)
    if e4m3:
        for pool, exp in ((b.k, b.k_exp), (b.v, b.v_exp)):
            pool[hide] = 0x7F
            exp[hide] = 255
    else:
        b.k[hide] = math.nan
        b.v[hide] = math.inf
        b.v[:, :, ::3][hide[:, :, ::3]] = math.nan
    b.upload()
    out, lse = b.attend(window=window)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    if e4m3:  # the plain form masks, but 0 * NaN is NaN there
        b.k_exp[hide], b.v_exp[hide] = 127, 127
        b.k[hide], b.v[hide] = 0, 0
    else:
        b.k[hide], b.v[hide] = 0, 0
    b.check(out, lse, window=window)


def test_nan_at_a_visible_position_reaches_the_rows_that_see_it(lib):
    b = Batch([1, 2], [100, 50], seed=3)
    b.k[b.tab[0, 3].long(), 0, 5, 7] = math.nan
    b.upload()
    out, lse = b.attend()
    assert out[0, : b.G].isnan().all() and lse[0, : b.G].isnan().all()
    assert torch.isfinite(out[0, b.G:]).all() and torch.isfinite(out[1:]).all()


@FMT
def test_rows_apart_and_a_batch_larger_than_its_rows(lib, e4m3):
    """q as a slice of a projection's output; the rows past row_off[R] stay as they are."""
    b = Batch([3, 8], [40, 200], e4m3=e4m3, seed=12).upload()
    T = b.T + 5
    wide = torch.full((T, b.Hq + 6, b.D), math.nan, dtype=torch.bfloat16, device=DEV)
    wide[: b.T, 2:2 + b.Hq] = b.q.to(DEV)
    q = wide[:, 2:2 + b.Hq]
    out = torch.full((T, b.Hq, b.D), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, b.Hq), 7.0, device=DEV)
    ws = b.cache.workspace(b.R, T, b.Hq)
    for max_rows in (8, 0):
        b.cache.attend(q, b.d_off, b.d_ctx, b.d_tab, out, lse=lse, max_rows=max_rows, ws=ws)
        torch.cuda.synchronize()
        b.check(out[: b.T], lse[: b.T])
        assert (out[b.T:] == 7).all() and (lse[b.T:] == 7).all()


@FMT
def test_bits_repeat_on_streams_and_in_graphs(lib, e4m3):
    b = Batch([8, 1, 3, 130], [5000, 90, 700, 20], e4m3=e4m3, seed=13).upload()
    out, lse = b.attend()
    side = torch.cuda.Stream()
    q = b.q.to(DEV)
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    args = (q, b.d_off, b.d_ctx, b.d_tab, o2)
    kw = dict(lse=l2, max_rows=130, ws=b.ws)
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        for _ in range(3):
            o2.zero_()
            torch.cuda.synchronize()
            b.cache.attend(*args, stream=stream, **kw)
            torch.cuda.synchronize()
            assert torch.equal(o2, out) and torch.equal(l2, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.cache.attend(*args, **kw)
    for _ in range(2):
        o2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    # the workspace is at rest again: nothing but the (clear) status word and counters
    assert (b.ws[:8192] == 0).all() if b.ws.numel() >= 8192 else (b.ws == 0).all()


def test_lse_is_optional(lib):
    b = Batch([2, 140], [30, 10], seed=1).upload()
    out, _ = b.attend()
    o2 = torch.zeros_like(out)
    b.cache.attend(b.q.to(DEV), b.d_off, b.d_ctx, b.d_tab, o2, max_rows=140, ws=b.ws)
    torch.cuda.synchronize()
    assert torch.equal(out, o2)


@FMT
def test_bad_pages_and_lengths_are_flagged_and_read_as_zeros(lib, e4m3):
    from draft_sampling_lossless_gb300 import binding as B

    b = Batch([2, 3], [60, 100], e4m3=e4m3, seed=2)
    b.tab[0, 1] = b.n_pages  # one past the pool
    b.tab[1, 0] = -5
    b.upload()
    out, lse = b.attend()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert b.cache.status(b.ws, clear=True) == B.DEVFLAG_PAGE_RANGE
    # what such a page holds reads as zeros: the same rows over a zeroed page
    b1 = Batch([2, 3], [60, 100], e4m3=e4m3, seed=2)
    for n, i in ((0, 1), (1, 0)):
        b1.k[b1.tab[n, i].long()] = 0
        b1.v[b1.tab[n, i].long()] = 0
    b1.check(out, lse)
    # a context past the table: the positions it does not cover read as zeros
    b2 = Batch([1, 2], [60, 100], e4m3=e4m3, seed=2).upload()
    b2.d_ctx[0] = 2 ** 31 - 1
    out, lse = b2.attend()
    assert torch.isfinite(out).all()
    assert b2.cache.status(b2.ws, clear=True) & B.DEVFLAG_PAGE_RANGE
    # more rows than max_rows says
    b3 = Batch([4, 1], [60, 100], e4m3=e4m3, seed=2).upload()
    out, lse = b3.attend(max_rows=3)
    assert b3.cache.status(b3.ws, clear=True) == B.DEVFLAG_ROW_RANGE
    assert (out[3] == 7).all() and torch.isfinite(out).all()


@FMT
def test_offsets_past_32_bits(lib, e4m3):
    """Pages beyond element 2^31 of a pool (k and v share one: it is only read)."""
    from draft_sampling_lossless_gb300.cache import PagedCache

    small = Batch([8, 2], [300, 90], Hkv=8, page=128, e4m3=e4m3, seed=21)
    n_pages = 2 ** 31 // (8 * 128 * 128) + 10
    pool = torch.empty((n_pages, 8, 128, 128), dtype=small.k.dtype, device=DEV)
    exp = torch.empty(pool.shape[:3], dtype=torch.uint8, device=DEV) if e4m3 else None
    at = n_pages - small.n_pages
    pool[at:] = small.k.to(DEV)
    if e4m3:
        exp[at:] = small.k_exp.to(DEV)
    small.v, small.v_exp = small.k, small.k_exp
    small.upload()
    small.cache = PagedCache(pool, pool, exp, exp)
    small.d_tab = torch.where(small.d_tab >= 0, small.d_tab + at, small.d_tab)
    small.check(*small.attend())
    ko, vo = (torch.empty((small.T, 8, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    small.cache.read(small.d_off, small.d_ctx, small.d_tab, ko, vo, small.ws)
    k_new = torch.randn(small.T, 8, 128, device=DEV).bfloat16()
    small.cache.append(k_new, k_new, small.d_off, small.d_ctx, small.d_tab, small.ws)
    ka, va = torch.empty_like(ko), torch.empty_like(vo)
    small.cache.read(small.d_off, small.d_ctx, small.d_tab, ka, va, small.ws)
    torch.cuda.synchronize()
    for n in range(2):
        a, m = small.off[n], small.rows[n]
        want = small.values(n, small.k, small.k_exp)[-m:]
        assert torch.equal(ko[a:a + m].cpu().double(), want)
    if e4m3:
        assert torch.equal(ka.cpu().double(), code_values(*quantise(k_new.cpu())))
    else:
        assert torch.equal(ka, k_new) and torch.equal(va, k_new)
    assert small.cache.status(small.ws) == 0


# ---------------------------------------------------------------- writing and reading


def special_rows(D):
    """Rows where the exponent or the rounding is on an edge."""
    x = torch.zeros(12, D)
    x[1, 0] = 448.0  # the largest code at exponent 0
    x[2, 0] = 450.0  # bf16's next value: exponent 1
    x[3] = torch.linspace(-1, 1, D)
    x[4, :8] = torch.tensor([448.0, 17.0, 19.0, 21.0, 1.0625, -1.1875, 2 ** -9, 3 * 2 ** -10])  # ties
    x[5, 3] = 2.0 ** -133  # bf16's smallest
    x[6, 1] = 2.0 ** -95
    x[7, 2] = 1.0e38
    x[7, 3] = -3.0
    x[8, :4] = torch.tensor([-0.0, 1e-30, 2.0, -2.0])
    x[9] = 1.75
    x[10] = -1.7578125  # just over 1.75
    x[11, D - 1] = -0.013
    return x.bfloat16()


@FMT
@pytest.mark.parametrize("D,Hkv", [(16, 1), (64, 3), (80, 2), (128, 8), (128, 21)])
def test_write_and_read_back(lib, D, Hkv, e4m3):
    """Every slot that a row was written to holds its value, every other slot what it held."""
    m, ctx = ragged(D, 6, (0, 9), (0, 60))
    m, ctx = m + [5, 12, 2], ctx + [-3, 0, -2]
    b = Batch(m, ctx, Hkv=Hkv, G=1, D=D, page=16, e4m3=e4m3, seed=D).upload()
    g = torch.Generator().manual_seed(D)
    new = torch.randn(b.T, Hkv * 2 + 1, D, generator=g).bfloat16()
    new[b.off[7]:b.off[8], :Hkv] = special_rows(D).unsqueeze(1)
    wide = new.to(DEV)
    b.cache.append(wide[:, :Hkv], wide[:, Hkv:2 * Hkv], b.d_off, b.d_ctx, b.d_tab, b.ws)
    ko, vo = (torch.full((b.T + 2, Hkv, D), 7.0, dtype=torch.bfloat16, device=DEV)
              for _ in range(2))
    b.cache.read(b.d_off, b.d_ctx, b.d_tab, ko, vo, b.ws)
    torch.cuda.synchronize()
    assert b.cache.status(b.ws) == 0
    assert (ko[b.T:] == 7).all() and (vo[b.T:] == 7).all()
    for pool, exp, dev, dexp, out, part in (
            (b.k, b.k_exp, b.cache.k, b.cache.k_exp, ko, new[:, :Hkv]),
            (b.v, b.v_exp, b.cache.v, b.cache.v_exp, vo, new[:, Hkv:2 * Hkv])):
        codes, byte = quantise(part) if e4m3 else (part, None)
        for n in range(b.R):
            for j in range(b.rows[n]):
                t, p = b.off[n] + j, b.ctx[n] + j
                if p < 0:
                    assert (out[t] == 0).all()
                    continue
                page, slot = b.tab[n, p // 16].long(), p % 16
                pool[page, :, slot] = codes[t]
                want = part[t].double()
                if e4m3:
                    exp[page, :, slot] = byte[t]
                    want = code_values(codes[t], byte[t])
                got = out[t].cpu().double()
                ok = (got == want) | ((want.abs() < 2.0 ** -126) & ((got - want).abs() <= 2.0 ** -134))
                assert ok.all(), (n, j)
        assert torch.equal(dev.cpu().view(torch.uint8), pool.view(torch.uint8))
        if e4m3:
            assert torch.equal(dexp.cpu(), exp)


def test_non_finite_values_are_flagged_and_kept(lib):
    from draft_sampling_lossless_gb300 import binding as B

    b = Batch([1], [3], Hkv=1, G=1, D=16, e4m3=True).upload()
    x = torch.zeros(1, 1, 16)
    x[0, 0, :5] = torch.tensor([math.inf, -math.inf, math.nan, 1.75, -0.5])
    x = x.bfloat16().to(DEV)
    b.cache.append(x, x, b.d_off, b.d_ctx, b.d_tab, b.ws)
    out = torch.empty(1, 1, 16, dtype=torch.bfloat16, device=DEV)
    b.cache.read(b.d_off, b.d_ctx, b.d_tab, out, torch.empty_like(out), b.ws)
    torch.cuda.synchronize()
    assert b.cache.status(b.ws) == B.DEVFLAG_NONFINITE
    got = out[0, 0, :5].tolist()  # 1.75 = 448 * 2^-8 is the largest finite value
    assert got[0] == 1.75 and got[1] == -1.75 and math.isnan(got[2]) and got[3:] == [1.75, -0.5]


@FMT
def test_writes_and_reads_with_bad_pages(lib, e4m3):
    from draft_sampling_lossless_gb300 import binding as B

    b = Batch([20, 2], [0, 5], e4m3=e4m3, seed=1)
    b.tab[0, 1] = -1
    b.upload()
    before = [t.clone() for t in (b.cache.k, b.cache.v)]
    new = torch.ones(b.T, b.Hkv, b.D, dtype=torch.bfloat16, device=DEV)
    b.cache.append(new, new, b.d_off, b.d_ctx, b.d_tab, b.ws)
    torch.cuda.synchronize()
    assert b.cache.status(b.ws, clear=True) == B.DEVFLAG_PAGE_RANGE
    used = {int(b.tab[0, 0]), int(b.tab[1, 0])}
    for was, pool in zip(before, (b.cache.k, b.cache.v)):
        for page in range(b.n_pages):
            if page not in used:
                assert torch.equal(was[page], pool[page])
    out = torch.full((b.T, b.Hkv, b.D), 7.0, dtype=torch.bfloat16, device=DEV)
    b.cache.read(b.d_off, b.d_ctx, b.d_tab, out, torch.empty_like(out), b.ws)
    torch.cuda.synchronize()
    assert b.cache.status(b.ws) == B.DEVFLAG_PAGE_RANGE
    assert (out[:16] == 1).all() and (out[16:20] == 0).all() and (out[20:] == 1).all()


@pytest.mark.parametrize("R", [1, 3, 127, 128, 129, 1000, 20000])
def test_rows_find_their_request(lib, R):
    """Batches around the lookup's 128-way passes, many requests without rows."""
    r = random.Random(R)
    rows = [r.choice([0, 0, 1, 2]) for _ in range(R)]
    rows[r.randrange(R)] = 5
    b = Batch(rows, [r.randint(0, 11) for _ in range(R)], Hkv=1, G=1, D=16, seed=R).upload()
    out = torch.empty(b.T, 1, 16, dtype=torch.bfloat16, device=DEV)
    b.cache.read(b.d_off, b.d_ctx, b.d_tab, out, torch.empty_like(out), b.ws)
    torch.cuda.synchronize()
    n = torch.repeat_interleave(torch.arange(R), torch.tensor(rows))
    p = torch.tensor(b.ctx)[n] + torch.arange(b.T) - torch.tensor(b.off)[n]
    assert torch.equal(out[:, 0].cpu(), b.k[b.tab[n, p // 16].long(), 0, p % 16])
    b.check(*b.attend())


# ---------------------------------------------------------------- refusals


def test_refusals(lib):
    from draft_sampling_lossless_gb300.cache import PagedCache

    L = lib.lib()
    b = Batch([2, 1], [5, 9]).upload()
    c, ws, st = ctypes.byref(b.cache.desc), b.ws.data_ptr(), None
    q = b.q.to(DEV)
    p = q.data_ptr()
    off, ctx, tab = b.d_off.data_ptr(), b.d_ctx.data_ptr(), b.d_tab.data_ptr()
    W = b.tab.shape[1]

    def attend(c=c, R=2, T=3, Hq=8, max_rows=2, scale=0.1, causal=1, window=0, q=p, qs=8 * 128,
               off=off, ctx=ctx, tab=tab, W=W, out=p, ws=ws, n=b.ws.numel()):
        return L.dspark_attend(c, R, T, Hq, max_rows, scale, causal, window, q, qs, off, ctx, tab,
                               W, out, None, ws, n, st)

    launches = lib.launch_count()
    blank = lib.KVCache()
    for kw in (dict(c=None), dict(c=ctypes.byref(blank)), dict(R=0), dict(T=-1), dict(Hq=7),
               dict(Hq=0), dict(Hq=2 * 129), dict(max_rows=-1), dict(scale=0.0),
               dict(scale=math.nan), dict(scale=math.inf), dict(window=-1),
               dict(window=4, causal=0), dict(q=None), dict(q=p + 2), dict(qs=8 * 128 - 8),
               dict(qs=8 * 128 + 4), dict(off=None), dict(ctx=None), dict(tab=None), dict(W=0),
               dict(W=1 << 28), dict(out=None), dict(out=p + 8), dict(ws=None), dict(ws=ws + 16)):
        assert attend(**kw) == 1, kw
        assert L.dspark_last_error()
    assert attend(n=255) == 4
    assert attend(T=0, q=None, out=None) == 0  # no rows: nothing to do

    def append(k=p, ks=256, v=p, vs=256, T=3, n=b.ws.numel()):
        return L.dspark_cache_append(c, 2, T, k, ks, v, vs, off, ctx, tab, W, ws, n, st)

    for kw in (dict(k=None), dict(v=p + 4), dict(ks=248), dict(vs=260), dict(T=(1 << 24) + 1)):
        assert append(**kw) == 1, kw
    assert append(n=100) == 4
    assert append(T=0) == 0
    assert L.dspark_cache_read(c, 2, 3, off, ctx, tab, W, None, p, ws, 256, st) == 1
    assert L.dspark_cache_read(c, 2, 0, off, ctx, tab, W, None, None, ws, 256, st) == 0
    assert L.dspark_cache_workspace_bytes(c, 2, 3, 7) == 0
    assert lib.launch_count() == launches  # nothing was launched

    # the binding's own checks
    out = torch.empty_like(q)
    with pytest.raises(ValueError):
        b.cache.attend(q, b.d_off, b.d_ctx, b.d_tab, out)  # no workspace
    with pytest.raises(ValueError):
        b.cache.attend(q, b.d_off[:2], b.d_ctx, b.d_tab, out, ws=b.ws)
    with pytest.raises(ValueError):
        b.cache.attend(q.float(), b.d_off, b.d_ctx, b.d_tab, out, ws=b.ws)
    with pytest.raises(ValueError):
        b.cache.attend(q.transpose(0, 1), b.d_off, b.d_ctx, b.d_tab, out, ws=b.ws)
    with pytest.raises(ValueError):
        b.cache.attend(q, b.d_off.long(), b.d_ctx, b.d_tab, out, ws=b.ws)
    with pytest.raises(ValueError):
        PagedCache(b.cache.k, b.cache.v[:1])
    with pytest.raises(ValueError):
        PagedCache(b.cache.k.float(), b.cache.v.float())
    with pytest.raises(ValueError):
        PagedCache(b.cache.k, b.cache.v, b.cache.k[..., 0], None)
