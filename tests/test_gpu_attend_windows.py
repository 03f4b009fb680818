"""dspark_attend with windows that no context reaches and rows at negative positions: the
window's start lies below -2^31 there, and every row sees what it sees without a window."""

import pytest

from test_gpu_cache import FMT, Batch

pytestmark = pytest.mark.gpu


@FMT
@pytest.mark.parametrize("rows,ctx", [([8, 5, 1, 7], [-3, -2, 400, -7]),
                                      ([40, 90, 3], [-3, -39, 130])])
@pytest.mark.parametrize("window", [1 << 30, (1 << 30) + (1 << 24), (1 << 31) - 1])
def test_windows_past_every_position(lib, window, rows, ctx, e4m3):
    b = Batch(rows, ctx, e4m3=e4m3, page=32, seed=window % 97).upload()
    b.check(*b.attend(window=window), window=window)
    assert b.cache.status(b.ws) == 0


@FMT
@pytest.mark.parametrize("window", [5, 60])
def test_windows_and_padding_rows(lib, window, e4m3):
    b = Batch([8, 30, 90], [-3, -12, -39], e4m3=e4m3, seed=window).upload()
    b.check(*b.attend(window=window), window=window)
