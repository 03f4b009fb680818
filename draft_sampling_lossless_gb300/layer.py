"""The target's layers around its attention: products with 4-bit weights, the
gated product of a feed-forward block, the norms between blocks (libdspark's
dspark_linear4, dspark_gated4, dspark_norm), enqueued on one stream.  Marshalling
only -- every operator runs in the CUDA library.

Tensors are on the current device; rows may lie apart (slices of wider tensors).  A
call given a stream runs there: its tensors have to be ready on that stream, and their
memory must not be reused before it has passed the call (as for any use of a tensor on
another stream; Tensor.record_stream says so to torch).  Weights see to that themselves."""

from __future__ import annotations

import ctypes

import torch

from . import binding as B


class Weights4:
    """A matrix [N, K] in 4 bits: codes 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign, a
    power-of-two scale for 32 columns, in the library's layout."""

    def __init__(self, N, K, device="cuda"):
        n = B.weights4_bytes(N, K)
        if n == 0:
            raise ValueError(f"sizes out of range (N={N}, K={K}; K a multiple of 32)")
        self.N, self.K = N, K
        self.store = torch.empty(n, dtype=torch.uint8, device=device)
        self.desc = B.weights4_init(N, K, self.store)
        self._ref = ctypes.byref(self.desc)
        self._on = (self.store.get_device(),)
        # the handles of the streams that torch knows the store to be in use on
        self._streams = {torch._C._cuda_getCurrentRawStream(self._on[0])}

    def _used_on(self, handle, stream):
        """The store's memory is reused only after what `stream` does with it."""
        self.store.record_stream(torch.cuda.current_stream() if stream is None else stream)
        self._streams.add(handle)

    @classmethod
    def load(cls, codes, scales, stream=None):
        """From codes [N, K / 2] (two a byte, the even column in the low half) and
        scale bytes [N, K / 32] (b for 2^(b - 127)), uint8."""
        with torch.cuda.stream(stream):  # the store's memory is that stream's
            w = cls(codes.shape[0], 2 * codes.shape[1], codes.device)
        B.dspark_weights4_load(w._ref, w.N, w.K, codes, scales, stream)
        if stream is not None:
            codes.record_stream(stream)
            scales.record_stream(stream)
        return w

    @classmethod
    def quantize(cls, src, stream=None):
        """From a bf16 or fp32 matrix [N, K]: to nearest, scales that hold each
        group's largest value."""
        with torch.cuda.stream(stream):
            w = cls(src.shape[0], src.shape[1], src.device)
        B.dspark_weights4_quantize(w._ref, w.N, w.K, src, stream)
        if stream is not None:
            src.record_stream(stream)
        return w


def workspace_bytes(T, K) -> int:
    """Bytes of a workspace for products of up to T rows of up to K columns."""
    n = B.linear4_workspace_bytes(T, K)
    if n == 0:
        raise ValueError("sizes out of range")
    return n


def workspace(T, K, device="cuda", stream=None):
    """A zeroed workspace (uint8) for products of up to T rows of up to K columns;
    calls in flight at the same time need one each.  It is zeroed on `stream`, which
    its memory belongs to; calls on another one have to wait for that."""
    n = workspace_bytes(T, K)
    with torch.cuda.stream(stream):
        return torch.zeros(n, dtype=torch.uint8, device=device)


def linear4(x, w, out, ws, stream=None):
    """out = x w^T: x [T, K], out [T, N] bf16.  (dspark.h says what small values of x
    among larger ones may lose.)"""
    h = B.dspark_linear4(w._ref, w.N, w.K, x, out, ws, stream, w._on)
    if h not in w._streams:
        w._used_on(h, stream)


def gated4(x, gate, up, out, ws, act="silu", stream=None):
    """out = act(x gate^T) * (x up^T): x [T, K], out [T, N] bf16, act "silu" or
    "gelu" (the tanh form)."""
    if act not in B.ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(B.ACTIVATIONS)}, got {act!r}")
    if (up.N, up.K) != (gate.N, gate.K):
        raise ValueError("gate and up differ in shape")
    h = B.dspark_gated4(gate._ref, up._ref, gate.N, gate.K, B.ACTIVATIONS[act], x, out, ws,
                        stream, (*gate._on, *up._on))
    for w in (gate, up):
        if h not in w._streams:
            w._used_on(h, stream)


def norm(x, h=None, pre=None, y=None, x_out=None, post=None, gate=None, alpha=1.0, eps=1e-6,
         stream=None):
    """x' = x + alpha * gate * rms(y) * post into x_out, rms(x') * pre into h.

    x and x_out [T, d] bf16 or fp32, y and h [T, d] bf16, gate [T, d] or [1, d]
    bf16, post and pre [d] fp32.  Without post y is taken as it is, without gate as
    1, without y x' = x.  x_out may be x, h may be y."""
    B.dspark_norm(x, y, post, gate, alpha, pre, eps, x_out, h, stream)


def status(ws, clear=False) -> int:
    """The device status word of a workspace."""
    return B.device_status(ws, clear)
