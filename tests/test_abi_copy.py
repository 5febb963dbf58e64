"""Host-side argument checks of the block copy by bytes (no GPU: fake pointers that are never
dereferenced)."""
import ctypes

import pytest
import torch

import __graft_entry__
from paged_kv_cache_221_gb300 import _lib

E = {v: k for k, v in _lib.STATUS_NAMES.items()}
OK, INVALID, UNSUPPORTED = (E[n] for n in ("PA_OK", "PA_ERR_INVALID_ARG", "PA_ERR_UNSUPPORTED"))
vp = ctypes.c_void_p
P = vp(256)


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return _lib.load()


@pytest.mark.skipif(torch.cuda.is_available(),
                    reason="fake device pointers: host-only argument checks")
def test_copy_block_bytes_arguments(lib):
    def call(k=P, v=P, pairs=P, n=2, NB=4, size=544):
        return lib.pa_copy_block_bytes(k, v, pairs, n, NB, size, None)
    assert call(n=0) == OK
    for kw in (dict(n=-1), dict(NB=0), dict(size=0), dict(size=-16), dict(size=552), dict(k=None),
               dict(v=None), dict(pairs=None), dict(k=vp(264)), dict(v=vp(264))):
        assert call(**kw) == INVALID, kw
    assert call(n=65536) == UNSUPPORTED
