"""The checks of the layers' calls that need no GPU: bad arguments and host tensors
are refused before anything is launched."""

import ctypes

import pytest
import torch

F = 0x10000  # a non-null pointer that is never dereferenced
WS = 1 << 30


def test_store_sizes(lib):
    # tiles of 128 x 128: 64 bytes of codes a row, 512 bytes of scales
    assert lib.weights4_bytes(1, 32) == 128 * 64 + 512
    assert lib.weights4_bytes(129, 2560) == 2 * 20 * (128 * 64 + 512)
    for N, K in ((0, 32), (-1, 32), (1, 0), (1, 16), (1, 33), (1, 1 << 17), ((1 << 24) + 1, 32)):
        assert lib.weights4_bytes(N, K) == 0, (N, K)


def test_workspace_sizes(lib):
    assert lib.linear4_workspace_bytes(0, 32) >= 256
    assert lib.linear4_workspace_bytes(4096, 2560) >= lib.linear4_workspace_bytes(1, 2560)
    for T, K in ((-1, 64), ((1 << 24) + 1, 64), (1, 0), (1, 40)):
        assert lib.linear4_workspace_bytes(T, K) == 0, (T, K)


def test_init_rejects_bad_descriptions(lib):
    L = lib.lib()
    d = lib.Weights4Desc()
    ref = ctypes.byref(d)
    for kw in (dict(w=None), dict(N=0), dict(N=(1 << 24) + 1), dict(K=0), dict(K=48),
               dict(K=65568), dict(store=None), dict(store=F + 128)):
        a = dict(dict(w=ref, N=4, K=64, store=F), **kw)
        assert L.dspark_weights4_init(a["w"], a["N"], a["K"], a["store"]) == 1, kw
        assert L.dspark_last_error()


def test_calls_reject_weights_that_were_not_initialised(lib):
    L = lib.lib()
    w = ctypes.byref(lib.Weights4Desc())
    for p in (w, None):
        assert L.dspark_weights4_load(p, F, F, None) == 1
        assert L.dspark_weights4_quantize(p, F, 0, 64, None) == 1
        assert L.dspark_linear4(p, 1, F, 64, F, 4, F, WS, None) == 1
        assert L.dspark_gated4(p, p, 0, 1, F, 64, F, 4, F, WS, None) == 1


def test_norm_rejects_bad_arguments(lib):
    L = lib.lib()

    def norm(T=2, d=64, dt=0, x=F, xs=64, y=F, ys=64, post=F, gate=F, gs=64, alpha=1.0, pre=F,
             eps=1e-6, xo=F, xos=64, h=F, hs=64):
        return L.dspark_norm(T, d, dt, x, xs, y, ys, post, gate, gs, alpha, pre, eps, xo, xos, h,
                             hs, None)

    nan = float("nan")
    for kw in (dict(T=-1), dict(T=(1 << 24) + 1), dict(d=0), dict(d=4), dict(d=68),
               dict(d=1 << 16), dict(dt=2), dict(dt=-1), dict(x=None), dict(x=F + 8), dict(xs=56),
               dict(xs=65), dict(y=F + 2), dict(ys=63), dict(ys=8), dict(post=F + 4),
               dict(gate=F + 2), dict(gs=8), dict(gs=68), dict(gs=-64), dict(alpha=nan),
               dict(alpha=float("inf")), dict(eps=-1.0), dict(eps=nan), dict(eps=float("inf")),
               dict(pre=None), dict(pre=F + 4), dict(xo=F + 8), dict(xos=0), dict(h=F + 8),
               dict(hs=0), dict(h=None), dict(h=None, pre=None, xo=None), dict(y=None),
               dict(y=None, post=None, gate=None), dict(y=None, xo=None, gate=None),
               dict(y=None, xo=None, post=None)):
        assert norm(**kw) == 1, kw
        assert L.dspark_last_error()
    assert norm(T=0) == 0  # nothing to do


def test_the_python_calls_refuse_host_tensors_and_wrong_types(lib):
    b = torch.bfloat16
    x, out = torch.zeros(3, 64, dtype=b), torch.zeros(3, 8, dtype=b)
    ws = torch.zeros(4096, dtype=torch.uint8)
    w = ctypes.byref(lib.Weights4Desc())
    with pytest.raises(ValueError, match="CUDA"):
        lib.dspark_linear4(w, 8, 64, x, out, ws, stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        lib.dspark_gated4(w, w, 8, 64, 0, x, out, ws, stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        lib.dspark_norm(x, None, None, None, 1.0, torch.ones(64), 1e-6, None, x.clone(), stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        lib.weights4_init(8, 64, torch.zeros(16384, dtype=torch.uint8))
    with pytest.raises(ValueError, match="store"):
        lib.weights4_init(8, 64, torch.zeros(16, dtype=torch.uint8))
    for bad in (x.float(), x[:, :32], x[0], x.T.contiguous().T):
        with pytest.raises(ValueError):
            lib.dspark_linear4(w, 8, 64, bad, out, ws, stream=0)
    for bad in (out.float(), out[:2], out[:, :4]):
        with pytest.raises(ValueError):
            lib.dspark_linear4(w, 8, 64, x, bad, ws, stream=0)


def test_layer_refuses_shapes(lib):
    from draft_sampling_lossless_gb300 import layer

    with pytest.raises(ValueError, match="sizes"):
        layer.Weights4(4, 40, device="cpu")
    with pytest.raises(ValueError, match="sizes"):
        layer.workspace(-1, 64, device="cpu")
    with pytest.raises(ValueError, match="act"):
        layer.gated4(None, None, None, None, None, act="relu")
