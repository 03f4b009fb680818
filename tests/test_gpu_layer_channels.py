"""4-bit products of rows with a channel far above its neighbours: where its weight is zero, the
neighbours' products are all there is, and each of their bits counts.

The neighbours are whole numbers of 8 bits, the weights' partial sums whole numbers of halves that
fp32 holds (as in test_gpu_layer_cuts), and the channels' weights are zero, so a product is
the exact one, rounded once, whatever the channels hold."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

from test_gpu_layer import DEV, act64, bound_of, run_gated, run_linear  # noqa: E402
from test_gpu_layer_cuts import Codes, rows  # noqa: E402

# rows of few and many, clusters of 1 to 8 blocks, x split by the blocks and before, several tiles
SIZES = ((3, 200, 512), (20, 300, 2560), (33, 131, 32), (33, 138, 704), (34, 140, 5440),
         (17, 139, 5056), (18, 131, 7200), (61, 20053, 160), (64, 30000, 640), (122, 2560, 4096),
         (165, 13159, 288), (300, 1000, 2080), (700, 6144, 640), (2092, 131, 7104))


def channels(x, K, far, seed, row_share=1.0):
    """One channel of every group of 32 becomes 2^far times its neighbours (in a share of the rows);
    the channels, as columns."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    at = torch.randint(0, 32, (K // 32,), generator=g, device=DEV) + 32 * torch.arange(
        K // 32, device=DEV)
    pick = torch.rand((x.shape[0], 1), generator=g, device=DEV) < row_share
    x[:, at] = torch.where(pick, (x[:, at].double() * 2.0 ** far).bfloat16(), x[:, at])
    return at


@pytest.mark.parametrize("far", (9, 14, 17, 24, 60, 110))
@pytest.mark.parametrize("T,N,K", SIZES)
def test_the_neighbours_of_a_far_channel_keep_their_bits(T, N, K, far):
    for share in (1.0, 0.05):
        w = Codes(N, K, T + N)
        x = rows(T, K, 8 * (T % 3), T + K)
        w.c[:, channels(x, K, far, far, share)] = 0
        if share < 1:  # ordinary rows too lie apart: an infinity in one of them
            x[T // 2, 1] = math.inf
        near = torch.where(x.abs() > 255, 0, x)
        o = w.product(near)
        got = run_linear(x, w.load(), apart=T % 4)
        ok = torch.ones(T, dtype=torch.bool, device=DEV)
        if share < 1:
            ok[T // 2] = False
            assert not got[T // 2].isfinite().any()
        assert torch.equal(got[ok], o.float().bfloat16()[ok])


@pytest.mark.parametrize("T,N,K", SIZES)
def test_channels_further_away_than_fp32_reaches(T, N, K):
    """2^127 beside numbers of 2^-23: the neighbours in the channel's scale are below 2^-126."""
    w = Codes(N, K, T + N)
    x = rows(T, K, 0, T + K) * 2.0 ** -30
    at = channels(x, K, 1, 4)
    w.c[:, at] = 0
    x[:, at] = 0
    o = w.product(x)
    x[:, at] = 2.0 ** 127
    assert torch.equal(run_linear(x, w.load(), apart=T % 4), o.float().bfloat16())


@pytest.mark.parametrize("T,N,K", SIZES)
def test_gated(T, N, K):
    shift = round(math.log2(470 * math.sqrt(K)))
    g, u = Codes(N, K, T + N, shift), Codes(N, K, T + N + 1, shift)
    x = rows(T, K, 0, T + K)
    at = channels(x, K, 20, 1, 0.5)
    g.c[:, at], u.c[:, at] = 0, 8  # a zero with a sign
    near = torch.where(x.abs() > 255, 0, x)
    want = act64("silu", g.product(near)) * u.product(near)
    got = run_gated(x, g.load(), u.load(), "silu", apart=T % 4)
    assert ((got.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -14) * want.abs() + 1e-36).all()


@pytest.mark.parametrize("T,N,K", SIZES)
def test_channels_with_weights(T, N, K):
    """With other weights on the channels the sums are as far off as fp32's: K 2^-25 of the
    products' magnitudes (as in test_gpu_layer), no group's rounding on top."""
    w = Codes(N, K, T + N)
    x = rows(T, K, 0, T + K)
    channels(x, K, 16, 2)
    m = torch.eye(K, dtype=torch.bfloat16, device=DEV)
    a, _ = bound_of(x, w.product(m).T)
    o = w.product(x)
    off = (run_linear(x, w.load()).double() - o).abs()
    assert (off <= 2.0 ** -8 * o.abs() + K * 2.0 ** -25 * a).all()


def test_sparse_rows_and_smallest_numbers():
    """Few values a group, the rest zeros; numbers down to bf16's smallest beside one of 1; the
    smallest alone."""
    T, N, K = 64, 160, 96
    w = Codes(N, K, 5)
    w.c[:, 0::32] = 0
    for low in (-20, -60, -125, -133):
        x = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
        x[:, 0::32] = 1.0
        x[:, 7::32] = 2.0 ** low
        x[::2, 9::32] = -3 * 2.0 ** low
        o = w.product(x)
        got = run_linear(x, w.load())
        # below the smallest normal numbers sums may end: near enough there
        assert ((got.double() - o).abs() <= 2.0 ** -9 * o.abs() + (low < -100) * 2.0 ** -126).all()
        if low > -100:
            assert torch.equal(got, o.float().bfloat16())


def test_a_rows_result_does_not_depend_on_its_neighbours():
    T, N, K = 300, 260, 1280
    w = Codes(N, K, 1)
    q = w.load()
    x = rows(T, K, 0, 2)
    clean = run_linear(x, q).clone()
    bad = x.clone()
    channels(bad[::7], K, 18, 3)
    bad[::7] = torch.where(torch.arange(K, device=DEV) % 32 == 5, 2.0 ** 25, bad[::7])
    got = run_linear(bad, q)
    rest = torch.arange(T, device=DEV) % 7 != 0
    assert torch.equal(got[rest], clean[rest])
    for _ in range(3):
        assert torch.equal(run_linear(bad, q), got)
