"""Host-side argument checks of prompt attention, the batch's block tables and the log
probabilities (no GPU: fake pointers that are never dereferenced)."""
import ctypes

import pytest
import torch

import __graft_entry__
from paged_kv_cache_221_gb300 import _lib

E = {v: k for k, v in _lib.STATUS_NAMES.items()}
OK, INVALID, UNSUPPORTED, WORKSPACE = (E[n] for n in ("PA_OK", "PA_ERR_INVALID_ARG",
                                                       "PA_ERR_UNSUPPORTED",
                                                       "PA_ERR_WORKSPACE"))
vp = ctypes.c_void_p
P, Z = vp(256), vp(512)
host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="fake device pointers: host-only argument checks")


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return _lib.load()


@host_only
def test_prompt_arguments(lib):
    def call(**kw):
        a = dict(out=P, q=P, k=P, v=P, ks=None, vs=None, dtype=0, window=0, tables=P, mbs=8, lens=P,
                 mcl=128, starts=P, N=20, B=2, NB=4, hq=4, hkv=4, D=64, BS=16, scale=0.125, psize=0,
                 ws=None, wsb=0)
        a.update(kw)
        return lib.pa_prompt_attention(*a.values(), None)
    assert call(N=0) == OK
    assert call(B=0) == OK
    for name in ("out", "q", "k", "v", "tables", "lens", "starts"):
        assert call(**{name: None}) == INVALID
    for name in ("out", "q", "k", "v"):
        assert call(**{name: vp(264)}) == INVALID
    for kw in (dict(N=-1), dict(B=-1), dict(NB=0), dict(hq=0), dict(hkv=0), dict(mbs=0),
               dict(window=-1), dict(psize=-128), dict(psize=100), dict(dtype=2), dict(dtype=-1),
               dict(dtype=1), dict(dtype=1, ks=P), dict(hq=6), dict(mcl=0), dict(mcl=129)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=96), dict(BS=32), dict(hq=129, hkv=1), dict(NB=2 ** 25),
               dict(mcl=2 ** 30 + 1, mbs=2 ** 27)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(N=2 ** 31 - 1, hq=128, hkv=1) == UNSUPPORTED          # units past 32 bits
    long = dict(mcl=4096, mbs=256, psize=128)
    assert call(**long) == WORKSPACE
    need = lib.pa_prompt_workspace_size(20, 2, 4, 4, 4096, 64, 16, 128, 0)
    assert call(**long, ws=P, wsb=need - 1) == WORKSPACE
    assert call(**long, ws=vp(264), wsb=need) == INVALID


def test_prompt_workspace(lib):
    def size(N=20, B=2, hq=4, hkv=4, mcl=4096, D=64, BS=16, psize=128, window=0):
        return lib.pa_prompt_workspace_size(N, B, hq, hkv, mcl, D, BS, psize, window)

    def r256(x):
        return (x + 255) // 256 * 256

    rows = 20 * 4 * 32                                   # 32 partitions
    assert size() == r256(rows * 64 * 4) + r256(rows * 8)
    assert size(psize=4096) == 0
    assert size(mcl=128) == 0
    assert size(window=4096) == size() and size(window=100) < size()
    assert size(N=12000, mcl=512, psize=0) == 0          # enough query tiles: nothing is cut
    assert size(N=200000, psize=0) == 256                # many: a counter to take them by
    assert size(N=1, B=1, psize=0) > 0
    for kw in (dict(N=0), dict(B=0), dict(hq=5), dict(psize=100), dict(psize=-1), dict(BS=8),
               dict(window=-1), dict(mcl=0), dict(hq=129, hkv=1)):
        assert size(**kw) == 0, kw


@host_only
def test_extend_arguments(lib):
    def call(**kw):
        a = dict(tables=P, mbs=4, lens=P, refs=P, new=P, B=2, N=5, NB=8, BS=16, starts=P, slots=P,
                 pos=P, copies=P)
        a.update(kw)
        return lib.pa_extend_sequences(*a.values(), None)
    for name in ("tables", "lens", "refs", "new", "starts", "slots", "pos", "copies"):
        assert call(**{name: None}) == INVALID, name
    for kw in (dict(B=-1), dict(N=-1), dict(NB=0), dict(mbs=0)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(BS=8), dict(B=12289), dict(mbs=2 ** 26 + 1), dict(NB=2 ** 30 + 1),
               dict(N=2 ** 30 + 1)):
        assert call(**kw) == UNSUPPORTED, kw


@host_only
def test_truncate_arguments(lib):
    def call(**kw):
        a = dict(tables=P, mbs=4, lens=P, refs=P, keep=Z, B=2, NB=8, BS=16)
        a.update(kw)
        return lib.pa_truncate_sequences(*a.values(), None)
    assert call(B=0) == OK
    for name in ("tables", "lens", "refs", "keep"):
        assert call(**{name: None}) == INVALID, name
    assert call(keep=P) == INVALID                       # the lengths themselves
    for kw in (dict(B=-1), dict(NB=0), dict(mbs=0)):
        assert call(**kw) == INVALID, kw
    assert call(BS=32) == UNSUPPORTED


@host_only
def test_logprob_arguments(lib):
    def call(**kw):
        a = dict(lp=P, h=P, top=P, tok=P, x=P, stride=100, dtype=0, tokens=P, N=3, V=100, k=2)
        a.update(kw)
        return lib.pa_token_logprobs(*a.values(), None)
    assert call(N=0) == OK
    for name in ("lp", "h", "top", "tok", "x", "tokens"):
        assert call(**{name: None}) == INVALID, name
    for kw in (dict(N=-1), dict(V=0), dict(k=-1), dict(k=101), dict(stride=99), dict(dtype=3),
               dict(dtype=-1), dict(x=vp(258)), dict(x=vp(257), dtype=1)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(V=2 ** 19 + 1, stride=2 ** 20), dict(k=33), dict(N=2 ** 27 + 1)):
        assert call(**kw) == UNSUPPORTED, kw
