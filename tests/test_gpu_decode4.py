"""Speculative decoding of a target with 4-bit projections, gated feed-forward blocks and
the norms between blocks (draft_sampling_lossless_gb300.decode.Target4): every call of a run
against its 64-bit form on that call's own inputs."""

import pytest
import torch

pytestmark = pytest.mark.gpu

from draft_sampling_lossless_gb300 import layer  # noqa: E402
from draft_sampling_lossless_gb300.decode import Decoder, Target4  # noqa: E402
from test_gpu_layer import Matrix, check_gated, check_linear, norm64  # noqa: E402


class Values:
    """A loaded matrix's 64-bit values, read back as products with unit rows (exact: a value
    of 4 bits times a power of two is a bf16)."""

    def __init__(self, w):
        eye = torch.eye(w.K, dtype=torch.bfloat16, device="cuda")
        out = torch.empty(w.K, w.N, dtype=torch.bfloat16, device="cuda")
        layer.linear4(eye, w, out, layer.workspace(w.K, w.K))
        self.N, self.K, self.m = w.N, w.K, out.double().T


@pytest.fixture
def checked(monkeypatch):
    """Every call of the layers checked as it is made; counts by name."""
    real = {n: getattr(layer, n) for n in ("linear4", "gated4", "norm")}
    seen, values = dict(linear4=0, gated4=0, norm=0), {}

    def value(w):
        if id(w) not in values:
            values[id(w)] = (w, None)
            busy.append(1)
            values[id(w)] = (w, Values(w))
            busy.pop()
        return values[id(w)][1]

    busy = []

    def linear4(x, w, out, ws, stream=None):
        real["linear4"](x, w, out, ws, stream)
        if not busy:
            seen["linear4"] += 1
            check_linear(x, value(w), out)

    def gated4(x, gate, up, out, ws, act="silu", stream=None):
        real["gated4"](x, gate, up, out, ws, act, stream)
        seen["gated4"] += 1
        check_gated(x, value(gate), value(up), act, out)

    def norm(x, h=None, pre=None, y=None, x_out=None, post=None, gate=None, alpha=1.0, eps=1e-6,
             stream=None):
        before = x.clone()
        real["norm"](x, h, pre, y, x_out, post, gate, alpha, eps, stream)
        seen["norm"] += 1
        want_x, want_h = norm64(before, y, post, gate, alpha, pre, eps)
        if x_out is not None:  # one product and one sum in fp32
            scale = want_x.abs() + before.double().abs()
            assert ((x_out.double() - want_x).abs() <= 2.0 ** -22 * scale).all()
        # the sum of squares, a root, a quotient and two products in fp32; bf16's rounding; what
        # x's own roundings are against the row's size
        rms = want_x.square().mean(-1, keepdim=True).sqrt()
        tol = (2.0 ** -8 + 2.0 ** -16) * want_h.abs() + 2.0 ** -20 * (
            before.double().abs() + want_x.abs()).amax(-1, keepdim=True) / rms
        assert ((h.double() - want_h).abs() <= tol).all()

    for n, f in (("linear4", linear4), ("gated4", gated4), ("norm", norm)):
        monkeypatch.setattr(layer, n, f)
    return seen


@pytest.mark.parametrize("T,e4m3", ((0.0, False), (0.0, True), (1.0, False)))
def test_every_call_of_a_run(checked, T, e4m3):
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, 512, (n,), generator=g).tolist() for n in (1, 2, 33, 150)]
    d = Decoder(Target4(seed=3), prompts, T=T, e4m3=e4m3)
    steps = 5
    gained = sum(len(x) for _ in range(steps) for x in d.step())
    assert steps * len(prompts) <= gained <= steps * len(prompts) * 8
    calls = steps + 1  # the prompts' pass is one more
    assert checked == dict(linear4=calls * (2 * 3 + 1), gated4=calls * 2, norm=calls * 5)
    assert d.t.status() == 0


def test_the_values_read_back():
    m = Matrix(40, 96)
    assert torch.equal(Values(m.load()).m, m.m)


def test_tokens_repeat():
    """Greedy runs of the same prompts give the same tokens; the drafter is of use."""
    prompts = [[i, 7 * i + 1] for i in range(8)]
    a, b = (Decoder(Target4(seed=1), prompts) for _ in range(2))
    for _ in range(4):
        assert a.step() == b.step()
    b.move(e4m3=True)
    b.step()
