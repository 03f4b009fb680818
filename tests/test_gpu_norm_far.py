"""Norms at the ends of the number ranges: not only the sums of squares but the products around
them pass fp32's range where the formula's value does not."""

import pytest
import torch

pytestmark = pytest.mark.gpu

from draft_sampling_lossless_gb300 import layer  # noqa: E402
from test_gpu_layer import DEV, norm64  # noqa: E402


def norm_error(d):
    """Relative: a sum of d squares (at most d / 8 + 16 roundings in a row, halved by the root),
    the root, the factor, four products."""
    return (d / 8 + 16) * 2.0 ** -24 + 8 * 2.0 ** -24


@pytest.mark.parametrize("d", (64, 2560, 12000, 20000))
def test_norm_of_a_blocks_largest_output(d):
    """y near bf16's largest, a post (and gate) above 1: rms(y) * post is of ordinary size."""
    for T in (2, 200):
        g = torch.Generator().manual_seed(d + T)
        y = (torch.rand(T, d, generator=g) * 0.4 + 1.5).mul(2.0 ** 127).bfloat16().to(DEV)
        post = (2 + torch.rand(d, generator=g)).to(DEV)
        gate = (1 + torch.rand(T, d, generator=g)).bfloat16().to(DEV)
        x, xo = torch.ones(T, d, device=DEV), torch.empty(T, d, device=DEV)
        for gt in (None, gate, gate[:1]):
            layer.norm(x, y=y, x_out=xo, post=post, gate=gt, alpha=0.5)
            want, _ = norm64(x, y, post, gt, 0.5, None, 1e-6)
            err = (want - 1).abs() * norm_error(d) + 2.0 ** -23 * (want.abs() + 1)
            assert ((xo.double() - want).abs() <= err).all()


def test_norm_with_a_gate_and_a_small_alpha():
    """alpha * gate * y without post: gate * y alone is past fp32's largest."""
    T, d = 3, 256
    g = torch.Generator().manual_seed(1)
    y = (torch.rand(T, d, generator=g) * 0.4 + 1.5).mul(2.0 ** 127).bfloat16().to(DEV)
    gate = (4 + torch.rand(T, d, generator=g)).bfloat16().to(DEV)
    x, xo = torch.zeros(T, d, device=DEV), torch.empty(T, d, device=DEV)
    layer.norm(x, y=y, x_out=xo, gate=gate, alpha=2.0 ** -10)
    want, _ = norm64(x, y, None, gate, 2.0 ** -10, None, 1e-6)
    assert ((xo.double() - want).abs() <= 3 * 2.0 ** -24 * want.abs()).all()


@pytest.mark.parametrize("d", (64, 2560, 12000, 20000))
@pytest.mark.parametrize("size", (2.0 ** -126, 2.0 ** -130, 2.0 ** -140, 2.0 ** -148))
def test_norm_of_the_smallest_rows(d, size):
    """eps = 0 and rows below fp32's smallest normal number: each value is what fp32 (and, for y,
    bf16) holds of it, and is normed like any other."""
    for T in (2, 200):
        g = torch.Generator().manual_seed(d + T)
        x = (torch.rand(T, d, generator=g, dtype=torch.float64) + 1).mul(size).float().to(DEV)
        assert (x > 0).all()
        pre = (1 + 0.3 * torch.randn(d, generator=g)).to(DEV)
        h = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
        layer.norm(x, h, pre, eps=0.0)
        _, want = norm64(x, None, None, None, 1.0, pre, 0.0)
        assert ((h.double() - want).abs() <= (norm_error(d) + 2.0 ** -8) * want.abs()).all()
        y = x.bfloat16()
        if not (y > 0).all():  # below half of bf16's smallest
            continue
        s, xo = torch.ones(T, d, device=DEV), torch.empty(T, d, device=DEV)
        layer.norm(s, y=y, x_out=xo, post=pre, eps=0.0)
        want, _ = norm64(s, y, pre, None, 1.0, None, 0.0)
        err = (want - 1).abs() * norm_error(d) + 2.0 ** -23 * (want.abs() + 1)
        assert ((xo.double() - want).abs() <= err).all()
