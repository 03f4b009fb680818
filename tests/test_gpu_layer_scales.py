"""Every code and scale byte through the 4-bit products' kernel on the tensor cores."""

import pytest
import torch

pytestmark = pytest.mark.gpu

from test_gpu_layer import DEV, Matrix, run_linear  # noqa: E402


@pytest.mark.parametrize("T", (40, 300, 900))
@pytest.mark.parametrize("e", (1, 2, 20, 100, 127, 128, 129, 150, 230, 251, 252))
def test_every_code_and_scale_with_many_rows(e, T):
    """As test_every_code_and_scale, through the kernel on the tensor cores: unit rows among
    others, of 1 and of sizes that use both of an activation's terms."""
    codes = (torch.arange(32).view(1, -1) + torch.arange(16).view(-1, 1)) % 16
    for N in (16, 300):
        c = codes.repeat(-(-N // 16), 1)[:N]
        w = Matrix(N, 32, codes=c, scales=torch.full((N, 1), e, dtype=torch.uint8))
        q = w.load()
        for v in (1.0, 1.9921875) if e < 252 else (1.0,):
            unit = torch.zeros(T, 32, dtype=torch.bfloat16, device=DEV)
            unit[torch.arange(T), torch.arange(T) % 32] = v
            got = run_linear(unit, q)
            exact = v * w.m.T[torch.arange(T) % 32]
            if e <= 2:  # below bf16's and fp32's normal numbers: near enough
                assert (got.double() - exact).abs().max() <= 2.0 ** -126
            else:
                assert torch.equal(got, exact.float().bfloat16())


@pytest.mark.parametrize("T", (4, 40, 300))
def test_bytes_outside_the_range_are_the_nearest_of_it(T):
    """0 counts as 1, 253 to 255 as 252: on unit rows every weight is the same number."""
    codes = torch.randint(0, 16, (8, 64), generator=torch.Generator().manual_seed(0))
    unit = torch.zeros(T, 64, dtype=torch.bfloat16, device=DEV)
    unit[torch.arange(T), torch.arange(T) % 64] = 1.0
    for byte, near in ((0, 1), (253, 252), (254, 252), (255, 252)):
        a, b = (torch.full((8, 2), v, dtype=torch.uint8) for v in (byte, near))
        got = [run_linear(unit, Matrix(8, 64, codes=codes, scales=s).load()) for s in (a, b)]
        assert torch.equal(got[0], got[1]) and got[0].isfinite().all()
        if near == 252:
            m = Matrix(8, 64, codes=codes, scales=b).m.T[torch.arange(T) % 64]
            assert torch.equal(got[0], m.float().bfloat16())
