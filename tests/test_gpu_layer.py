"""The layers' operators (4-bit products, the gated product, the norms) against plain
64-bit forms, at the sizes and values where they can go wrong.

Products of whole numbers are exact: where every partial sum is a whole number of
halves below 2^23, the result is the exact one, rounded once to bf16.

Otherwise, with A = sum_k |x_k w_k| of an output value, from the formula:
  * the result is rounded once to bf16:                     2^-8 |o|
  * x may lose what lies below 2^-21 of its group's largest: 2^-21 sum_g max|x_g| sum|w_g|
  * fp32 sums of K terms, 2^-22 a term where it may truncate, over chains of K / 8
    terms at most (every kernel adds at least 8 products or partial sums side by side):
                                                            K 2^-25 A"""

import ctypes
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

from draft_sampling_lossless_gb300 import binding as B  # noqa: E402
from draft_sampling_lossless_gb300 import layer  # noqa: E402

DEV = "cuda"
VALUES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                      dtype=torch.float64)


class Matrix:
    """Random codes and scales, their 64-bit values and the library's copy of them."""

    def __init__(self, N, K, seed=0, lo=120, hi=126, codes=None, scales=None):
        g = torch.Generator().manual_seed(seed + 1000 * N + K)
        self.N, self.K = N, K
        c = torch.randint(0, 16, (N, K), generator=g) if codes is None else codes
        self.scales = (torch.randint(lo, hi + 1, (N, K // 32), generator=g).to(torch.uint8)
                       if scales is None else scales)
        self.codes = (c[:, 0::2] | (c[:, 1::2] << 4)).to(torch.uint8)
        e = self.scales.long().clamp(1, 252) - 127
        self.m = torch.ldexp(VALUES[c], e.repeat_interleave(32, 1)).to(DEV)

    def load(self):
        return layer.Weights4.load(self.codes.to(DEV), self.scales.to(DEV))


def activations(T, K, seed=0, apart=0):
    g = torch.Generator().manual_seed(seed + 77 * T + K)
    x = torch.randn(T, K + apart, generator=g) * torch.exp(torch.randn(K + apart, generator=g))
    return x.bfloat16().to(DEV)[:, :K]


def bound_of(x, m):
    """(sum |x w|, sum over groups of max |x| sum |w|) of every output value."""
    x, m = x.double().abs(), m.abs()
    g = x.view(x.shape[0], -1, 32).amax(2).repeat_interleave(32, 1)
    return x @ m.T, g @ m.T


def check_linear(x, w, got):
    o = x.double() @ w.m.T
    a, g = bound_of(x, w.m)
    tol = 2.0 ** -8 * o.abs() + 2.0 ** -21 * g + w.K * 2.0 ** -25 * a + 1e-38
    off = (got.double() - o).abs()
    assert (off <= tol).all(), (off / tol).max().item()


def act64(name, a):
    if name == "silu":
        return a * torch.sigmoid(a)
    # 0.5 (1 + tanh y) = 1 / (1 + exp(-2 y)), which 64 bits hold where 1 + tanh y cancels
    return a * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3))


def check_gated(x, g, u, act, got):
    """|act'| <= 1.2 and |act(a)| <= |a|: the products' errors, 2^-20 for the fp32
    arithmetic on top of each factor, one rounding."""
    a, b = x.double() @ g.m.T, x.double() @ u.m.T
    (aa, ga), (ab, gb) = bound_of(x, g.m), bound_of(x, u.m)
    ea = 2.0 ** -21 * ga + g.K * 2.0 ** -25 * aa
    eb = 2.0 ** -21 * gb + g.K * 2.0 ** -25 * ab
    o = act64(act, a) * b
    tol = (2.0 ** -8 + 2.0 ** -20) * o.abs() + 1e-38 + (
        (1.2 * ea + 2.0 ** -20 * a.abs()) * (b.abs() + eb) + a.abs() * eb)
    off = (got.double() - o).abs()
    assert (off <= tol).all(), (off / tol).max().item()


def run_linear(x, w, apart=0, ws=None):
    T = x.shape[0]
    out = torch.full((T, w.N + apart), -7.0, dtype=torch.bfloat16, device=DEV)
    ws = layer.workspace(T, w.K) if ws is None else ws
    layer.linear4(x, w, out[:, :w.N], ws)
    assert layer.status(ws) == 0
    assert (out[:, w.N:] == -7).all()
    return out[:, :w.N]


def run_gated(x, g, u, act, apart=0):
    T = x.shape[0]
    out = torch.full((T, g.N + apart), -7.0, dtype=torch.bfloat16, device=DEV)
    ws = layer.workspace(T, g.K)
    layer.gated4(x, g, u, out[:, :g.N], ws, act=act)
    assert layer.status(ws) == 0
    assert (out[:, g.N:] == -7).all()
    return out[:, :g.N]


ROWS = (1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 49, 64, 65, 96, 97, 127, 128, 129,
        191, 192, 193, 257, 300, 511, 700)
SHAPES = ((1, 32), (3, 64), (16, 96), (17, 128), (127, 160), (128, 256), (129, 512), (300, 1056),
          (520, 2560), (2560, 4096))


# ---------------------------------------------------------------- 4-bit weights


def test_quantize_and_load_agree_with_a_search():
    """Codes by search over the values (ties to the even code), scales by the rule; the
    store that quantize fills is the one that load fills from them."""
    for N, K, dt in ((1, 32, torch.float32), (5, 96, torch.bfloat16), (131, 160, torch.float32),
                     (64, 256, torch.bfloat16)):
        g = torch.Generator().manual_seed(N + K)
        w = torch.randn(N, K, generator=g) * torch.exp2(
            torch.randint(-140, 120, (N, K // 32), generator=g).float()).repeat_interleave(32, 1)
        w[0, :32] = 0
        w[0, 3] = 6.0  # a full group of ties and borders
        w[0, 4:20] = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 0.2500001, -.25, -.75, -1.25,
                                   -1.75, -2.5, -3.5, -5, 5.0000005])
        if N > 2:
            w[2, :32] = 0
            w[1, :32] = 6.0000005
        w = w.to(dt)
        v = w.double().view(N, -1, 32)
        amax = v.abs().amax(-1)
        e = torch.full_like(amax, -100)
        for k in range(-100, 128):
            e = torch.where((6 * 2.0 ** k < amax) & (e == k), torch.full_like(e, k + 1), e)
        y = (v / torch.exp2(e).unsqueeze(-1)).view(N, K)
        mag = VALUES[:8]
        near = (y.abs().unsqueeze(-1) - mag).abs()
        best = near == near.amin(-1, keepdim=True)
        even = torch.tensor([0, 0, 0, 0, 0, 0, 0, 0]) + (torch.arange(8) % 2)
        code = torch.argmin(torch.where(best, even, 9), dim=-1)
        code = code + 8 * torch.signbit(w).long().view(N, K)
        ref = Matrix(N, K, codes=code, scales=(e + 127).to(torch.uint8))
        a, b = ref.load(), layer.Weights4.quantize(w.to(DEV))
        assert torch.equal(a.store, b.store), (N, K)


def test_quantize_takes_what_is_not_finite():
    w = torch.ones(2, 64)
    w[0, 5], w[0, 6], w[0, 7] = math.inf, -math.inf, math.nan
    q = layer.Weights4.quantize(w.to(DEV))
    eye = torch.zeros(64, 64, dtype=torch.bfloat16, device=DEV)
    eye.fill_diagonal_(1.0)
    got = run_linear(eye, q).cpu().T
    # the finite maximum is 1 = 4 * 2^-2: an infinity is 6 * 2^-2
    assert got[0, 5] == 1.5 and got[0, 6] == -1.5 and got[0, 7] == 0
    assert (got[1] == 1).all() and got[0, 4] == 1


def test_every_code_and_scale():
    """A matrix that holds every code at every scale, one column at a time."""
    for e in (1, 20, 100, 127, 150, 230):
        codes = (torch.arange(32).view(1, -1) + torch.arange(16).view(-1, 1)) % 16
        w = Matrix(16, 32, codes=codes, scales=torch.full((16, 1), e, dtype=torch.uint8))
        eye = torch.zeros(32, 32, dtype=torch.bfloat16, device=DEV)
        eye.fill_diagonal_(1.0)
        got = run_linear(eye, w.load())
        want = w.m.T.float().bfloat16()
        if e == 1:  # below bf16's and fp32's normal numbers: near enough
            assert (got.double() - w.m.T).abs().max() <= 2.0 ** -126
        else:
            assert torch.equal(got, want), e


def test_scale_bytes_outside_the_range_count_as_the_nearest():
    codes = torch.randint(0, 16, (8, 64), generator=torch.Generator().manual_seed(0))
    a = torch.full((8, 2), 127, dtype=torch.uint8)
    b = a.clone()
    a[1, 0], b[1, 0], a[2, 1], b[2, 1] = 0, 1, 255, 254
    x = activations(4, 64)
    # row 2's products pass fp32's range: NaN or infinite, but the same
    got = [run_linear(x, Matrix(8, 64, codes=codes, scales=s).load()) for s in (a, b)]
    assert torch.equal(got[0].isnan(), got[1].isnan())
    assert torch.equal(got[0].nan_to_num(), got[1].nan_to_num())
    assert got[0][:, [0, 1, 3, 4, 5, 6, 7]].isfinite().all()


# ---------------------------------------------------------------- products


@pytest.mark.parametrize("N,K", SHAPES)
def test_linear_sizes(N, K):
    w = Matrix(N, K)
    q = w.load()
    for T in ROWS:
        check_linear(activations(T, K), w, run_linear(activations(T, K), q))


@pytest.mark.parametrize("T", (1, 5, 16, 23, 64, 130, 260, 1000))
@pytest.mark.parametrize("N,K", ((37, 160), (300, 2560), (1030, 640)))
def test_whole_numbers_are_exact(N, K, T):
    """Values of 8 bits need both halves of every activation; partial sums stay below 2^22."""
    g = torch.Generator().manual_seed(T + N)
    x = (2 * torch.randint(64, 128, (T, K), generator=g) + 1).float()
    x *= torch.randint(0, 2, (T, K), generator=g) * 2 - 1
    x = x.bfloat16().to(DEV)
    w = Matrix(N, K, lo=127, hi=127)
    got = run_linear(x, w.load())
    o = x.double() @ w.m.T
    assert torch.equal(got, o.float().bfloat16())


@pytest.mark.parametrize("T", (3, 40, 200))
def test_activations_of_very_different_sizes(T):
    """Within a group of 32 the small values keep their bits down to 2^-21 of the largest;
    other groups keep all of theirs."""
    K = 256
    g = torch.Generator().manual_seed(T)
    e = torch.randint(-24, 1, (T, K), generator=g) + 30 * torch.randint(-2, 3, (T, 8),
                                                                       generator=g).repeat_interleave(32, 1)
    x = torch.ldexp(torch.randn(T, K, generator=g), e).bfloat16().to(DEV)
    eye = torch.full((K, K), 0)
    eye.fill_diagonal_(2)
    w = Matrix(K, K, codes=eye, scales=torch.full((K, 8), 127, dtype=torch.uint8))
    got = run_linear(x, w.load())
    top = x.double().abs().view(T, -1, 32).amax(2).repeat_interleave(32, 1)
    off = (got.double() - x.double()).abs()
    assert (off <= 2.0 ** -8 * x.double().abs() * (x.double().abs() < 2.0 ** -12 * top)
            + 2.0 ** -21 * top).all()
    big = x.double().abs() >= 2.0 ** -12 * top
    assert torch.equal(got[big], x[big])


@pytest.mark.parametrize("T", (1, 20, 150))
def test_rows_lie_apart(T):
    w = Matrix(200, 96)
    x = activations(T, 96, apart=40)
    got = run_linear(x, w.load(), apart=7)
    check_linear(x, w, got)
    u = Matrix(200, 96, seed=5)
    check_gated(x, w, u, "silu", run_gated(x, w.load(), u.load(), "silu", apart=9))


@pytest.mark.parametrize("act", ("silu", "gelu"))
@pytest.mark.parametrize("N,K", ((1, 32), (33, 160), (128, 256), (300, 1056), (1000, 2080)))
def test_gated_sizes(N, K, act):
    g, u = Matrix(N, K, lo=119, hi=123), Matrix(N, K, seed=9, lo=119, hi=123)
    qg, qu = g.load(), u.load()
    for T in ROWS:
        x = activations(T, K)
        check_gated(x, g, u, act, run_gated(x, qg, qu, act))


@pytest.mark.parametrize("T", (1, 40, 200))
def test_gated_far_values(T):
    """Activations of large arguments: silu and gelu go to a or to 0, not to NaN."""
    K = 32
    codes = torch.zeros(64, K, dtype=torch.int64)
    codes[:, 0] = 2
    g = Matrix(64, K, codes=codes, scales=torch.full((64, 1), 127, dtype=torch.uint8))
    x = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = torch.linspace(-500, 500, T).bfloat16().to(DEV) if T > 1 else -500.0
    for act in ("silu", "gelu"):
        got = run_gated(x, g.load(), g.load(), act)
        a = x[:, :1].double().expand(T, 64)
        want = act64(act, a) * a
        assert ((got.double() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-30).all()


@pytest.mark.parametrize("T", (2, 24, 150, 300))
def test_rows_that_are_not_finite_stay_alone(T):
    w = Matrix(150, 288)
    q = w.load()
    x = activations(T, 288)
    clean = run_linear(x, q).clone()
    bad = x.clone()
    bad[T // 2, 40] = math.nan
    bad[T - 1, 200] = math.inf
    got = run_linear(bad, q)
    rows = [t for t in range(T) if t not in (T // 2, T - 1)]
    assert torch.equal(got[rows], clean[rows])
    assert got[T // 2].isnan().all()
    assert not got[T - 1].isfinite().any()


def test_zero_rows_and_zeros():
    w = Matrix(70, 64)
    q = w.load()
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV)
    assert run_linear(x, q).shape == (0, 70)
    for T in (1, 30, 200):
        x = torch.zeros(T, 64, dtype=torch.bfloat16, device=DEV)
        assert (run_linear(x, q) == 0).all()
        assert (run_gated(x, q, q, "silu") == 0).all()


def test_same_results_every_time_and_with_a_larger_workspace():
    w = Matrix(1030, 2560)
    q = w.load()
    ws = layer.workspace(5000, 2560)
    for T in (1, 7, 16, 60, 130, 400):
        x = activations(T, 2560)
        a = run_linear(x, q).clone()
        for _ in range(3):
            assert torch.equal(run_linear(x, q, ws=ws), a)


def test_a_rows_result_does_not_depend_on_the_others():
    """The rows of a call are independent: a padded batch changes nothing."""
    w = Matrix(140, 320)
    q = w.load()
    x = activations(600, 320)
    full = run_linear(x, q)
    x2 = x.clone()
    x2[1::2] = 0
    half = run_linear(x2, q)
    assert torch.equal(full[0::2], half[0::2])


# ---------------------------------------------------------------- norms


def norm64(x, y, post, gate, alpha, pre, eps):
    x = x.double()
    if y is not None:
        u = y.double()
        if post is not None:
            u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps) * post.double()
        if gate is not None:
            u = u * gate.double()
        x = x + alpha * u
    return x, None if pre is None else (
        x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * pre.double())


@pytest.mark.parametrize("dt", (torch.bfloat16, torch.float32))
@pytest.mark.parametrize("d", (8, 16, 64, 248, 1000, 2560, 7168, 8200, 16392, 32768))
def test_norm_sizes(d, dt):
    """Per value: u carries at most 8 fp32 roundings and its norm's (a sum of d squares
    of one sign, at most d / 8 + 16 roundings in a row, halved by the root), x' two more."""
    for T in (1, 2, 33):
        g = torch.Generator().manual_seed(d + T)
        x = torch.randn(T, d + 8, generator=g).mul(3).to(dt).to(DEV)[:, :d]
        y = torch.randn(T, d + 16, generator=g).bfloat16().to(DEV)[:, :d]
        post, pre = (1 + 0.3 * torch.randn(d, generator=g).to(DEV) for _ in range(2))
        for use_y, use_post, gate_rows, store, use_h in (
                (False, False, 0, False, True), (True, False, 0, True, True),
                (True, True, T, True, True), (True, True, 1, False, True),
                (True, False, 1, True, False), (True, True, 0, True, True)):
            gate = None
            if gate_rows:
                gate = torch.rand(gate_rows, d, generator=g).bfloat16().to(DEV)
            h = torch.full((T + 1, d + 8), -7.0, dtype=torch.bfloat16, device=DEV)
            xo = torch.full((T + 1, d + 24), -7.0, dtype=dt, device=DEV)
            yy, pp = (y if use_y else None), (post if use_post else None)
            layer.norm(x, h[:T, :d] if use_h else None, pre if use_h else None, y=yy,
                       x_out=xo[:T, :d] if store else None, post=pp, gate=gate, alpha=0.75,
                       eps=1e-5)
            want_x, want_h = norm64(x, yy, pp, gate, 0.75, pre if use_h else None, 1e-5)
            sums = (d / 8 + 16) * 2.0 ** -24
            err = 0.0 if not use_y else (
                (want_x - x.double()).abs() * (8 * 2.0 ** -24 + sums) + 2.0 ** -23 * want_x.abs()
                + 2.0 ** -23 * x.double().abs())
            half = torch.finfo(dt).eps / 2
            if store:
                assert ((xo[:T, :d].double() - want_x).abs() <= err + half * want_x.abs()).all()
                assert (xo[T:] == -7).all() and (xo[:, d:] == -7).all()
            if use_h:
                rms = torch.sqrt((want_x ** 2).mean(-1, keepdim=True) + 1e-5)
                rel = 8 * 2.0 ** -24 + sums + 2.0 ** -8
                if use_y:
                    rel = rel + torch.sqrt((err ** 2).mean(-1, keepdim=True)) / rms
                tol = rel * want_h.abs() + err / rms * pre.double().abs() * 1.01
                assert ((h[:T, :d].double() - want_h).abs() <= tol).all()
                assert (h[T:] == -7).all() and (h[:, d:] == -7).all()
            else:
                assert (h == -7).all()


@pytest.mark.parametrize("dt", (torch.bfloat16, torch.float32))
def test_norm_in_place(dt):
    T, d = 19, 1032
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, d, generator=g).to(dt).to(DEV)
    y = torch.randn(T, d, generator=g).bfloat16().to(DEV)
    pre = torch.rand(d, generator=g).to(DEV)
    h, xo = torch.empty_like(y), torch.empty_like(x)
    layer.norm(x, h, pre, y=y, x_out=xo, post=pre, alpha=-1.5)
    layer.norm(x, y, pre, y=y, x_out=x, post=pre, alpha=-1.5)
    assert torch.equal(x, xo) and torch.equal(y, h)


def test_norm_of_zeros_and_of_what_is_not_finite():
    d = 64
    x = torch.zeros(4, d, device=DEV)
    x[1, 3], x[2, 5] = math.nan, math.inf
    x[3] = 1.0
    h = torch.empty(4, d, dtype=torch.bfloat16, device=DEV)
    layer.norm(x, h, torch.ones(d, device=DEV), eps=1e-6)
    assert (h[0] == 0).all()
    assert h[1].isnan().all()
    assert h[2, 5].isnan() and (h[2, :5] == 0).all()  # as the formula: inf / inf, 1 / inf
    assert (h[3] == 1).all()
    layer.norm(x[:0], h[:0], torch.ones(d, device=DEV))  # no rows


# ---------------------------------------------------------------- calls


def test_one_block_of_a_model():
    """The operators one after the other as a feed-forward block uses them."""
    T, d, F = 45, 256, 640
    g, u, dn = Matrix(F, d), Matrix(F, d, seed=1), Matrix(d, F, seed=2)
    x = torch.randn(T, d, generator=torch.Generator().manual_seed(1)).to(DEV)
    pre = torch.ones(d, device=DEV)
    h, y = (torch.empty(T, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    m = torch.empty(T, F, dtype=torch.bfloat16, device=DEV)
    ws = layer.workspace(T, F)
    layer.norm(x, h, pre)
    qg, qu, qd = g.load(), u.load(), dn.load()
    layer.gated4(h, qg, qu, m, ws)
    layer.linear4(m, qd, y, ws)
    check_gated(h, g, u, "silu", m)
    check_linear(m, dn, y)
    x2, h2 = torch.empty_like(x), torch.empty_like(h)
    layer.norm(x, h2, pre, y=y, x_out=x2, post=pre, alpha=0.5)
    want_x, want_h = norm64(x, y, pre, None, 0.5, pre, 1e-6)
    assert (x2.double() - want_x).abs().max() <= 2.0 ** -20 * want_x.abs().max()
    assert ((h2.double() - want_h).abs() <= 2.0 ** -7 * want_h.abs() + 1e-5).all()


@pytest.mark.parametrize("T", (1, 13, 100, 300))
def test_captured_and_replayed(T):
    w, u = Matrix(300, 512), Matrix(300, 512, seed=4)
    q, qu = w.load(), u.load()
    x = activations(T, 512).contiguous()
    out, out2 = (torch.empty(T, 300, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    h = torch.empty(T, 512, dtype=torch.bfloat16, device=DEV)
    pre = torch.ones(512, device=DEV)
    ws = layer.workspace(T, 512)

    def calls():
        layer.norm(x, h, pre)
        layer.linear4(h, q, out, ws)
        layer.gated4(h, q, qu, out2, ws)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed in (1, 2):
        x.copy_(activations(T, 512, seed=seed))
        out.zero_(), out2.zero_()
        graph.replay()
        a, b = out.clone(), out2.clone()
        calls()
        assert torch.equal(a, out) and torch.equal(b, out2)
        check_linear(h, w, out)
    assert layer.status(ws) == 0


def test_two_streams_with_a_workspace_each():
    w = Matrix(900, 1024)
    q = w.load()
    xs = [activations(T, 1024) for T in (11, 90, 400)]
    want = [run_linear(x, q).clone() for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    wss = [layer.workspace(x.shape[0], 1024) for x in xs]
    outs = [torch.empty_like(o) for o in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, s, ws, o in zip(xs, streams, wss, outs):
            layer.linear4(x, q, o, ws, stream=s)
    torch.cuda.synchronize()
    for o, r in zip(outs, want):
        assert torch.equal(o, r)


def test_refusals_that_need_tensors():
    w = Matrix(64, 96)
    q = w.load()
    x = activations(300, 96)
    out = torch.empty(300, 64, dtype=torch.bfloat16, device=DEV)
    ws = layer.workspace(300, 96)
    n = B.launch_count()
    with pytest.raises(B.DSparkError, match="workspace"):
        layer.linear4(x, q, out, ws[:256 if B.linear4_workspace_bytes(300, 96) > 256 else 128])
    with pytest.raises(B.DSparkError, match="aligned"):
        layer.linear4(x, q, out, ws[16:])
    wide = torch.zeros(300, 101, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(B.DSparkError, match="x_stride"):
        layer.linear4(wide[:, :96], q, out, ws)
    with pytest.raises(B.DSparkError, match="aligned"):
        layer.linear4(torch.zeros(300, 104, dtype=torch.bfloat16, device=DEV)[:, 4:100], q, out, ws)
    with pytest.raises(ValueError, match="shape"):
        layer.gated4(x, q, Matrix(64, 128).load(), out, ws)
    bad = B.Weights4Desc.from_buffer_copy(q.desc)
    other = Matrix(32, 96).load()
    assert B.lib().dspark_gated4(ctypes.byref(bad), other._ref, 0, 1, x.data_ptr(), 96,
                                 out.data_ptr(), 64, ws.data_ptr(), ws.numel(), None) == 1
    assert B.lib().dspark_gated4(q._ref, q._ref, 2, 1, x.data_ptr(), 96, out.data_ptr(), 64,
                                 ws.data_ptr(), ws.numel(), None) == 1
    for t in (x.cpu(), ):
        with pytest.raises(ValueError, match="CUDA"):
            layer.linear4(t, q, out, ws)
    with pytest.raises(ValueError, match="CUDA"):
        layer.linear4(x, q, out, ws.cpu())
    with pytest.raises(ValueError, match="CUDA"):
        layer.norm(x, out[:, :1].expand(300, 96).contiguous().cpu(), torch.ones(96, device=DEV))
    assert B.launch_count() - n == 2  # the two matrices loaded in between


# ---------------------------------------------------------------- large sizes, first calls


@pytest.mark.parametrize("T,N,K", ((64, 151936, 2560), (4100, 6144, 2560), (1500, 2560, 10240),
                                   (9, 32000, 2560), (33, 151936, 640), (5, 130, 65280),
                                   (40, 130, 65280), (200, 130, 65280)))
def test_large_sizes(T, N, K):
    """Against the 64-bit form in some of the columns; every value is finite."""
    g = torch.Generator(device=DEV).manual_seed(T)
    q = layer.Weights4.quantize(torch.randn((N, K), generator=g, device=DEV).bfloat16())
    x = (torch.randn((T, K), generator=g, device=DEV) * 2).bfloat16()
    got = run_linear(x, q)
    assert got.isfinite().all()
    # the matrix's values: unit rows of some columns' groups would need K rows; take the
    # columns' codes back through a product with whole blocks of unit rows
    cols = torch.randint(0, N, (40,), generator=torch.Generator().manual_seed(1)).to(DEV)
    m = torch.empty(len(cols), K, dtype=torch.float64, device=DEV)
    for k in range(0, K, 640):
        unit = torch.zeros(640, K, dtype=torch.bfloat16, device=DEV)
        unit[torch.arange(640), torch.arange(k, k + 640)] = 1.0
        m[:, k:k + 640] = run_linear(unit, q)[:, cols].double().T

    class W:
        pass

    w = W()
    w.K, w.m = K, m
    check_linear(x, w, got[:, cols])


def test_gated_prompts():
    T, N, K = 2300, 10240, 640
    g = torch.Generator(device=DEV).manual_seed(2)
    ws = [torch.randn((N, K), generator=g, device=DEV).mul_(0.05) for _ in range(2)]
    qs = [layer.Weights4.quantize(w) for w in ws]
    x = torch.randn((T, K), generator=g, device=DEV).bfloat16()
    got = run_gated(x, *qs, "silu")
    cols = torch.randint(0, N, (64,), generator=torch.Generator().manual_seed(1)).to(DEV)
    unit = torch.eye(K, dtype=torch.bfloat16, device=DEV)
    mats = []
    for q in qs:
        w = type("W", (), {})()
        w.K, w.m = K, run_linear(unit, q)[:, cols].double().T
        mats.append(w)
    check_gated(x, *mats, "silu", got[:, cols])


FIRST = """
import torch
from draft_sampling_lossless_gb300 import layer
x = torch.randn({T}, 512, device="cuda").bfloat16()
q = layer.Weights4.quantize(torch.randn(300, 512, device="cuda"))
h, pre = torch.empty_like(x), torch.ones(512, device="cuda")
out = torch.zeros({T}, 300, dtype=torch.bfloat16, device="cuda")
ws = layer.workspace({T}, 512)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    layer.norm(x, h, pre)
    layer.linear4(h, q, out, ws)
g.replay()
a = out.clone()
layer.linear4(h, q, out, ws)
assert torch.equal(a, out) and a.abs().max() > 0
print("same")
"""


@pytest.mark.parametrize("T", (2, 60, 300))
def test_first_call_of_a_process_may_be_captured(T):
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(T=T)], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-800:]


def test_two_graphs_one_after_the_other_may_share_a_workspace():
    w = Matrix(260, 384)
    q = w.load()
    xs = [activations(T, 384) for T in (40, 300)]
    want = [run_linear(x, q).clone() for x in xs]
    ws = layer.workspace(300, 384)
    outs = [torch.empty_like(o) for o in want]
    graphs = []
    for x, o in zip(xs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.linear4(x, q, o, ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, r in zip(outs, want):
        assert torch.equal(o, r)
    assert layer.status(ws) == 0


def test_one_matrix_for_gate_and_up_and_outputs_into_a_wider_buffer():
    w = Matrix(96, 64, lo=120, hi=123)
    q = w.load()
    for T in (5, 50, 200):
        x = activations(T, 64)
        wide = torch.full((T, 300), 3.0, dtype=torch.bfloat16, device=DEV)
        layer.gated4(x, q, q, wide[:, 101:197], layer.workspace(T, 64))
        check_gated(x, w, w, "silu", wide[:, 101:197])
        assert (wide[:, :101] == 3).all() and (wide[:, 197:] == 3).all()


def test_devices_and_streams():
    """Tensors of a call are on one device, the current one; a call given a stream runs there."""
    w = Matrix(64, 96)
    q = w.load()
    x = activations(7, 96)
    want = run_linear(x, q)
    out = torch.zeros_like(want)
    ws = layer.workspace(7, 96)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    layer.linear4(x, q, out, ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want)
    with pytest.raises(ValueError, match="device"):
        B.dspark_linear4(q._ref, 64, 96, x, out, ws, None, (1,))


@pytest.mark.parametrize("T", (3, 40, 200))
def test_the_longest_rows(T):
    """K = 65536, whole numbers: every partial sum is a whole number of halves below 2^23."""
    K = 65536
    g = torch.Generator().manual_seed(T)
    x = torch.randint(-3, 4, (T, K), generator=g).float().bfloat16().to(DEV)
    w = Matrix(150, K, lo=127, hi=127)
    got = run_linear(x, w.load())
    assert torch.equal(got, (x.double() @ w.m.T).float().bfloat16())


def test_weights_made_on_another_stream():
    s = torch.cuda.Stream()
    m = Matrix(200, 320)
    codes, scales = m.codes.to(DEV), m.scales.to(DEV)
    torch.cuda.synchronize()
    q = layer.Weights4.load(codes, scales, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for T in (4, 100):
        x = activations(T, 320)
        check_linear(x, m, run_linear(x, q))


def test_weights_written_just_before_they_are_used():
    """A product queued behind the call that writes its weights uses the new ones."""
    a, b = Matrix(300, 640), Matrix(300, 640, seed=8)
    q = a.load()
    cb = b.codes.to(DEV), b.scales.to(DEV)
    for T in (2, 50, 300):
        x = activations(T, 640)
        ws = layer.workspace(T, 640)
        outs = [torch.empty(T, 300, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        ca = a.codes.to(DEV), a.scales.to(DEV)
        torch.cuda.synchronize()
        for (c, s), o in ((ca, outs[0]), (cb, outs[1])):
            B.dspark_weights4_load(q._ref, 300, 640, c, s)
            layer.linear4(x, q, o, ws)
        check_linear(x, a, outs[0])
        check_linear(x, b, outs[1])


@pytest.mark.parametrize("d", (64, 2560, 12000))
@pytest.mark.parametrize("size,eps", ((2.0 ** 100, 1e-6), (2.0 ** 126, 1e-6), (2.0 ** 66, 0.0),
                                      (2.0 ** -70, 0.0), (2.0 ** -120, 0.0), (2.0 ** -20, 0.0),
                                      (2.0 ** -70, 1e-6)))
def test_norm_of_far_values(d, size, eps):
    """Rows whose squares leave fp32's range are normed like others (as in test_norm_sizes: the
    sum, a root, a quotient and products in fp32, bf16's rounding)."""
    for T in (3, 200):
        g = torch.Generator().manual_seed(d + T)
        x = (torch.rand(T, d, generator=g) + 0.5).mul(size).to(DEV)
        x[1] = torch.rand(d, generator=g).to(DEV)  # an ordinary row among them
        pre = (1 + 0.3 * torch.randn(d, generator=g)).to(DEV)
        h = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
        layer.norm(x, h, pre, eps=eps)
        _, want = norm64(x, None, None, None, 1.0, pre, eps)
        rel = 8 * 2.0 ** -24 + (d / 8 + 16) * 2.0 ** -24 + 2.0 ** -8
        assert ((h.double() - want).abs() <= rel * want.abs() + 1e-38).all()
        y = x.bfloat16()  # the block's own norm brings its output back to ordinary sizes
        s = torch.ones(T, d, device=DEV)
        xo = torch.empty_like(s)
        layer.norm(s, h, pre, y=y, x_out=xo, post=pre, eps=eps)
        want_x, _ = norm64(s, y, pre, None, 1.0, None, eps)
        err = (want_x - 1).abs() * (16 * 2.0 ** -24 + (d / 8 + 16) * 2.0 ** -24) + 2.0 ** -23 * (
            want_x.abs() + 1)
        assert ((xo.double() - want_x).abs() <= err).all()
