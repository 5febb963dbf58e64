"""Host-side argument checks of the INT4-page and bounded-cache entry points, and the block
manager's truncate (no GPU: fake pointers that are never dereferenced)."""
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
P, Z = vp(256), vp(512)                  # fake 256-byte aligned device pointers
host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="fake device pointers: host-only argument checks")


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return _lib.load()


@host_only
@pytest.mark.parametrize("fn", ["pa_reshape_and_cache_int4", "pa_gather_cache_int4"])
def test_store_and_gather_arguments(lib, fn):
    def call(**kw):
        a = dict(k=P, v=P, kc=P, vc=P, slots=P, ks=P, vs=P, n=4, NB=4, hkv=2, D=64, BS=16)
        a.update(kw)
        return getattr(lib, fn)(*a.values(), None)
    assert call(n=0) == OK
    assert call(n=-1) == INVALID
    assert call(D=96) == UNSUPPORTED
    assert call(D=8) == UNSUPPORTED
    assert call(BS=8) == UNSUPPORTED
    assert call(NB=0) == INVALID
    assert call(hkv=0) == INVALID
    assert call(n=2 ** 31 - 1, hkv=64) == UNSUPPORTED                 # past the grid's extent
    for name in ("k", "v", "kc", "vc", "slots", "ks", "vs"):
        assert call(**{name: None}) == INVALID
    for name in ("k", "v", "kc", "vc"):
        assert call(**{name: vp(264)}) == INVALID                     # misaligned


@host_only
def test_attention_arguments(lib):
    def call(**kw):
        a = dict(out=P, q=P, nk=None, nv=None, k=P, v=P, ks=P, vs=P, window=0, tables=P, mbs=4,
                 lens=P, mcl=64, B=1, T=1, NB=4, hq=4, hkv=4, D=64, BS=16, scale=0.125, psize=0,
                 ws=None, wsb=0)
        a.update(kw)
        return lib.pa_attention_int4(*a.values(), None)
    assert call(B=0) == OK
    for name in ("out", "q", "k", "v", "ks", "vs", "tables", "lens"):
        assert call(**{name: None}) == INVALID
    for name in ("out", "q", "k", "v"):
        assert call(**{name: vp(264)}) == INVALID
    assert call(nk=P) == INVALID and call(nv=P) == INVALID
    assert call(nk=vp(264), nv=P) == INVALID
    assert call(T=0) == INVALID and call(window=-1) == INVALID
    assert call(T=5, mcl=4) == INVALID
    assert call(mcl=65) == INVALID                                    # above the table's reach
    assert call(hq=6, hkv=4) == INVALID
    assert call(D=96) == UNSUPPORTED and call(BS=32) == UNSUPPORTED
    assert call(hq=64, hkv=1, T=2) == UNSUPPORTED                     # 128 rows per kv head
    assert call(psize=24) == INVALID and call(psize=-16) == INVALID
    assert call(psize=16) == WORKSPACE                                # split without scratch
    need = lib.pa_int4_workspace_size(1, 4, 4, 1, 64, 64, 16, 16, 0)
    assert need > 0
    assert call(psize=16, ws=P, wsb=need - 1) == WORKSPACE
    assert call(psize=16, ws=vp(272), wsb=need) == INVALID            # scratch misaligned
    assert call(B=65536) == UNSUPPORTED


def test_workspace_sizes(lib):
    size = lib.pa_int4_workspace_size
    assert size(64, 32, 8, 1, 256, 128, 16, 0, 0) == 0                # whole sequences
    assert size(64, 32, 8, 1, 512, 128, 16, 512, 0) == 0
    assert size(64, 30, 8, 1, 4096, 128, 16, 0, 0) == 0               # heads do not divide
    assert size(0, 32, 8, 1, 512, 128, 16, 0, 0) == 0
    assert size(4, 32, 8, 1, 16384, 128, 16, 0, 0) > 0
    # a window needs no more than the entries it spans
    assert size(4, 32, 8, 1, 16384, 128, 16, 512, 100) <= size(4, 32, 8, 1, 160, 128, 16, 512, 0)
    acc = lib.pa_accumulate_workspace_size
    assert acc(2, 8, 2, 3, 100) >= 2 * 2 * 100 * 12 * 4
    assert acc(2, 7, 2, 3, 100) == 0 and acc(0, 8, 2, 1, 100) == 0
    assert lib.pa_evict_workspace_size(2, 4, 100, 60) >= 2 * 4 * 40 * 8
    assert lib.pa_evict_workspace_size(2, 4, 100, 0) == 0


@host_only
def test_accumulate_arguments(lib):
    def call(**kw):
        a = dict(w=P, wo=P, pos=P, entries=64, q=P, k=P, ks=None, fmt=0, tables=P, mbs=4, lens=P,
                 seen=None, mcl=64, B=1, T=1, NB=4, hq=4, hkv=4, D=64, BS=16, scale=0.125,
                 decay=1.0, ws=P, wsb=1 << 30)
        a.update(kw)
        return lib.pa_accumulate_weights(*a.values(), None)
    assert call(B=0) == OK
    for name in ("w", "wo", "q", "k", "tables", "lens"):
        assert call(**{name: None}) == INVALID
    assert call(fmt=3) == INVALID and call(fmt=-1) == INVALID
    assert call(fmt=1) == INVALID and call(fmt=2) == INVALID          # no scales
    assert call(entries=63) == INVALID                                # shorter than the context
    assert call(mcl=65, entries=80) == INVALID
    assert call(T=5, mcl=4) == INVALID
    assert call(hq=6, hkv=4) == INVALID
    assert call(D=96) == UNSUPPORTED and call(BS=32) == UNSUPPORTED
    assert call(hq=64, hkv=1, T=2) == UNSUPPORTED
    assert call(B=16384) == UNSUPPORTED                               # 65536 pairs
    assert call(ws=None) == WORKSPACE and call(wsb=16) == WORKSPACE
    assert call(ws=vp(272)) == INVALID
    assert call(q=vp(264)) == INVALID and call(k=vp(264)) == INVALID


@host_only
def test_evict_arguments(lib):
    def call(**kw):
        a = dict(new=P, k=P, v=P, fmt=0, tables=P, mbs=4, lens=Z, mcl=64, w=P, pos=P, entries=64,
                 budget=16, recent=4, B=1, NB=4, hkv=4, D=64, BS=16, ws=P, wsb=1 << 30)
        a.update(kw)
        return lib.pa_evict_tokens(*a.values(), None)
    assert call(B=0) == OK
    for name in ("new", "k", "v", "tables", "lens", "w", "pos"):
        assert call(**{name: None}) == INVALID
    assert call(new=Z) == INVALID                                     # over context_lens
    assert call(budget=0) == INVALID and call(recent=-1) == INVALID
    assert call(recent=17) == INVALID                                 # above the budget
    assert call(fmt=3) == INVALID
    assert call(entries=63) == INVALID and call(mcl=65, entries=80) == INVALID
    assert call(D=96) == UNSUPPORTED and call(BS=32) == UNSUPPORTED
    assert call(B=16384) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(wsb=16) == WORKSPACE
    assert call(k=vp(264)) == INVALID and call(v=vp(264)) == INVALID


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    import paged_kv_cache_221_gb300 as pa
    k = torch.zeros((4, 2, pa.int4_page_bytes(64)), dtype=torch.uint8)
    s = torch.ones(2)
    slots = torch.zeros(1, dtype=torch.int64)
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pa.reshape_and_cache_int4(x, x, k, k, slots, s, s)
    with pytest.raises(ValueError, match="CUDA"):
        pa.gather_cache_int4(k, k, slots, s, s)
    with pytest.raises(ValueError, match="CUDA"):
        pa.attention_int4(x, k, k, s, s, slots, slots)
    with pytest.raises(ValueError, match="CUDA"):
        pa.accumulate_weights(x, k, slots, slots, x)
    with pytest.raises(ValueError, match="CUDA"):
        pa.evict_tokens(k, k, slots, slots, x, x, 4, 1)


def test_block_manager_truncate():
    import paged_kv_cache_221_gb300 as pa
    bm = pa.BlockManager(8)
    bm.add_sequence(1, 50)                                            # blocks 0-3
    bm.fork(1, 2)
    bm.truncate(1, 33)                                                # 3 blocks
    assert bm.num_tokens(1) == 33 and bm.ref_count(3) == 1 and bm.num_free_blocks() == 4
    bm.truncate(1, 32)
    assert bm.ref_count(2) == 1 and bm.num_free_blocks() == 4
    bm.truncate(2, 0)
    assert bm.num_free_blocks() == 6 and bm.num_tokens(2) == 0
    slot, copy = bm.append_slot(1)                                    # 32 tokens: a new block
    assert slot == 2 * 16 and copy is None
    for bad in ((9, 1), (1, 34), (1, -1)):
        with pytest.raises(pa.PagedAttnError):
            bm.truncate(*bad)
    assert bm.num_tokens(1) == 33
