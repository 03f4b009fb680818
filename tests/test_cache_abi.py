"""The paged cache's host-side checks that need no GPU."""

import ctypes


def test_cache_init_rejects_bad_descriptions(lib):
    L = lib.lib()
    c = lib.KVCache()
    ref = ctypes.byref(c)
    f = 0x10000  # a non-null pointer that is never dereferenced

    def init(cache=ref, fmt=0, n=4, Hkv=2, page=16, D=128, k=f, v=f, ke=None, ve=None):
        return L.dspark_cache_init(cache, fmt, n, Hkv, page, D, k, v, ke, ve)

    for kw in (dict(cache=None), dict(fmt=2), dict(fmt=-1), dict(D=0), dict(D=136), dict(D=144),
               dict(D=24), dict(page=8), dict(page=48), dict(page=2048), dict(n=0), dict(Hkv=0),
               dict(n=1 << 27), dict(n=1 << 62), dict(k=None), dict(v=None), dict(k=f + 8),
               dict(ke=f), dict(fmt=1), dict(fmt=1, ke=f), dict(fmt=1, ke=f, ve=f + 1)):
        assert init(**kw) == 1, kw
        assert L.dspark_last_error()


def test_calls_reject_a_cache_that_was_not_initialised(lib):
    L = lib.lib()
    c = ctypes.byref(lib.KVCache())
    f = 0x10000
    assert L.dspark_cache_append(c, 1, 1, f, 256, f, 256, f, f, f, 1, f, 1 << 20, None) == 1
    assert b"dspark_cache_init" in L.dspark_last_error()
    assert L.dspark_cache_read(c, 1, 1, f, f, f, 1, f, f, f, 1 << 20, None) == 1
    assert L.dspark_attend(c, 1, 1, 2, 1, 1.0, 1, 0, f, 256, f, f, f, 1, f, None, f, 1 << 20,
                           None) == 1
    assert L.dspark_cache_workspace_bytes(c, 1, 1, 2) == 0
    assert L.dspark_cache_append(None, 1, 1, f, 256, f, 256, f, f, f, 1, f, 1 << 20, None) == 1
