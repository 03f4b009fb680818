"""Activations of the gated product far below zero, and of what is not finite."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

from test_gpu_layer import DEV, Matrix, act64, run_gated  # noqa: E402


@pytest.mark.parametrize("T", (1, 40, 200))
@pytest.mark.parametrize("act", ("silu", "gelu"))
def test_activations_far_below_zero(act, T):
    """act(a) near the smallest normal number, times a factor that brings the product back to
    ordinary sizes.  The exponential's argument, at most 96, is off by 5 roundings (a cube, a sum,
    two products): 96 * 5 * 2^-24 < 2^-15, the quick exponential and quotient below as much;
    exp and act are fp32, so what they have below 2^-149 is lost; bf16's rounding."""
    K, N = 64, 64
    codes = torch.zeros(N, K, dtype=torch.int64)
    codes[:, 0] = 2  # a = x[0]
    one = torch.full((N, 2), 127, dtype=torch.uint8)
    g = Matrix(N, K, codes=codes, scales=one)
    ucodes = torch.zeros(N, K, dtype=torch.int64)
    ucodes[:, 32] = 2  # b = x[32] * 2^64
    u = Matrix(N, K, codes=ucodes, scales=one + 64)
    top = -92.0 if act == "silu" else -10.25
    x = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = torch.linspace(top, top + 5, T).bfloat16().to(DEV) if T > 1 else top
    x[:, 32] = 2.0 ** 40
    got = run_gated(x, g.load(), u.load(), act)
    a = x[:, :1].double().expand(T, N)
    want = act64(act, a) * 2.0 ** 104
    assert want.abs().min() > 0
    assert ((got.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -14) * want.abs()
            + 96 * 2.0 ** -149 * 2.0 ** 104).all()


def test_activations_of_what_is_not_finite():
    """A row with an infinity or a NaN is not finite; act of the largest numbers is a or 0."""
    K, N = 32, 8
    codes = torch.zeros(N, K, dtype=torch.int64)
    codes[:, 0] = 2
    w = Matrix(N, K, codes=codes, scales=torch.full((N, 1), 127, dtype=torch.uint8))
    q = w.load()
    for T in (6, 60):
        x = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
        for i, v in enumerate((math.inf, -math.inf, math.nan, 2.0 ** 60, -2.0 ** 60)):
            x[i, 0] = v
        for act in ("silu", "gelu"):
            got = run_gated(x, q, q, act)
            assert not got[:3].isfinite().any()
            assert (got[3] == 2.0 ** 120).all() and (got[4] == 0).all()
            assert (got[5:] == 0).all()
