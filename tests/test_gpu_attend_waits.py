"""The attention kernels' bounded wait: on a barrier that nothing completes it gives up near
its limit and tells its block, and the device stays usable."""

import pytest
import torch

from test_gpu_cache import Batch

pytestmark = pytest.mark.gpu


def test_a_wait_that_runs_out(lib):
    ws = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    ws[136:144] = 255
    t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    t[0].record()
    lib.dspark_check_wait_timeout(2000, ws)  # 2 ms each
    t[1].record()
    torch.cuda.synchronize()
    assert lib.device_status(ws) & lib.DEVFLAG_TIMEOUT
    assert ws[136:144].view(torch.int32).tolist() == [0, 1]  # no success, block told to stop
    assert 5.0 < t[0].elapsed_time(t[1]) < 1000.0
    b = Batch([2, 40], [30, 10], seed=1).upload()
    b.check(*b.attend())
