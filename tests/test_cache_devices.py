"""The paged cache's calls take CUDA tensors only: a host tensor is refused before anything is
launched (its address would be followed on the GPU).  No GPU needed."""

import ctypes

import pytest
import torch


def test_host_tensors_are_refused(lib):
    cache = ctypes.byref(lib.KVCache())
    rows = torch.zeros(3, 2, 16, dtype=torch.bfloat16)
    off, ctx = torch.tensor([0, 3], dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    pages, ws = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        lib.dspark_cache_append(cache, 2, 16, rows, rows, off, ctx, pages, ws, stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        lib.dspark_cache_read(cache, 2, 16, off, ctx, pages, rows, rows, ws, stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        lib.dspark_attend(cache, 16, rows, off, ctx, pages, rows, None, 1.0, True, 0, 0, ws,
                          stream=0)


def test_host_pools_are_refused(lib):
    k = torch.zeros(4, 2, 16, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        lib.cache_init(k, k)
    c, e = torch.zeros(4, 2, 16, 16, dtype=torch.uint8), torch.zeros(4, 2, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        lib.cache_init(c, c, e, e)


@pytest.mark.gpu
def test_one_host_tensor_among_the_others(lib):
    from test_gpu_cache import Batch

    b = Batch([2, 1], [5, 9]).upload()
    q, out = b.q.cuda(), torch.empty(b.q.shape, dtype=torch.bfloat16, device="cuda")
    good = dict(q=q, row_off=b.d_off, ctx=b.d_ctx, pages=b.d_tab, out=out, ws=b.ws)
    launches = lib.launch_count()
    for name in good:
        with pytest.raises(ValueError, match="CUDA"):
            b.cache.attend(**{**good, name: good[name].cpu()})
    kv = torch.zeros(3, b.Hkv, b.D, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="CUDA"):
        b.cache.append(kv, kv.cpu(), b.d_off, b.d_ctx, b.d_tab, b.ws)
    with pytest.raises(ValueError, match="CUDA"):
        b.cache.read(b.d_off, b.d_ctx, b.d_tab, kv, kv.cpu(), b.ws)
    assert lib.launch_count() == launches
