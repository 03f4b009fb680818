"""A layer's paged key/value cache on the GPU and the attention over it:
tensors, page bookkeeping and libdspark calls (dspark_cache_append,
dspark_cache_read, dspark_attend), enqueued on one stream.  Marshalling only
-- every operator runs in the CUDA library."""

from __future__ import annotations

import ctypes
import math

import torch

from . import binding as B


class PagedCache:
    """Pools k, v [n_pages, Hkv, page, D] that the caller made: bf16, or e4m3
    codes with exponent bytes k_exp, v_exp [n_pages, Hkv, page].

    Rows are packed as the scheduler lays them out: request n's are
    row_off[n] .. row_off[n+1]-1, its row j at position ctx[n] + j; position p
    is in slot p % page of page pages[n, p // page].  row_off [R+1], ctx [R]
    and pages [R, max_pages] are int32 device tensors."""

    def __init__(self, k, v, k_exp=None, v_exp=None):
        self.k, self.v, self.k_exp, self.v_exp = k, v, k_exp, v_exp
        self.n_pages, self.Hkv, self.page, self.D = k.shape
        self.desc = B.cache_init(k, v, k_exp, v_exp)
        self._ref = ctypes.byref(self.desc)

    @classmethod
    def empty(cls, n_pages, Hkv, page, D, e4m3=False, device="cuda"):
        """A cache with its own zeroed pools."""
        dev = torch.device(device)
        shape = (n_pages, Hkv, page, D)
        if not e4m3:
            return cls(*(torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in range(2)))
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=dev) for _ in range(2))
        return cls(k, v, *(torch.zeros(shape[:3], dtype=torch.uint8, device=dev)
                           for _ in range(2)))

    def workspace(self, R, T, Hq):
        """A zeroed workspace (uint8) for up to R requests, T rows and Hq query
        heads; calls in flight at the same time need one each."""
        n = B.cache_workspace_bytes(self.desc, R, T, Hq)
        if n == 0:
            raise ValueError("sizes out of range")
        return torch.zeros(n, dtype=torch.uint8, device=self.k.device)

    def append(self, k, v, row_off, ctx, pages, ws, stream=None):
        """Writes the rows' keys and values, [T, Hkv, D] bf16 (rows may lie apart)."""
        B.dspark_cache_append(self._ref, self.Hkv, self.D, k, v, row_off, ctx, pages, ws, stream)

    def read(self, row_off, start, pages, k_out, v_out, ws, stream=None):
        """Request n's positions start[n], start[n]+1, .. as rows of k_out and
        v_out, [T, Hkv, D] bf16."""
        B.dspark_cache_read(self._ref, self.Hkv, self.D, row_off, start, pages, k_out, v_out, ws,
                            stream)

    def attend(self, q, row_off, ctx, pages, out, lse=None, scale=None, causal=True, window=0,
               max_rows=0, ws=None, stream=None):
        """The rows' attention, q and out [T, Hq, D] bf16, over positions
        0 .. ctx[n] + rows - 1 (their own included: append first).  lse [T, Hq]
        fp32 takes ln of each row's sum of exponentials.  scale: 1 / sqrt(D) when
        None; max_rows: the most rows a request has (0: q's rows)."""
        if ws is None:
            raise ValueError("attend needs a workspace (PagedCache.workspace)")
        B.dspark_attend(self._ref, self.D, q, row_off, ctx, pages, out, lse,
                        1.0 / math.sqrt(self.D) if scale is None else scale, causal, window,
                        max_rows, ws, stream)

    def status(self, ws, clear=False) -> int:
        """The device status word of a workspace."""
        return B.device_status(ws, clear)
