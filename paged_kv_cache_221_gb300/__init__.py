"""GB300-native paged decode attention.

A thin PyTorch binding over the C ABI of ``libpaged_attn.so`` (declared in
``include/paged_attn.h``).  This module only checks tensor shapes, dtypes and
devices and marshals pointers and the current CUDA stream; every step of the
computation runs in the library's sm_103a kernels.  PyTorch is used for device
memory and streams only.

Layouts (bf16 unless stated):
    q, out        [num_seqs, num_query_tokens, num_q_heads, head_dim]
    k_cache,
    v_cache       [num_blocks, num_kv_heads, block_size, head_dim]
    block_tables  [num_seqs, max_blocks_per_seq] int32
    context_lens  [num_seqs] int32 (counts the newest token / the drafts)
    key, value    [num_tokens, num_kv_heads, head_dim]
    slot_mapping  [num_tokens] int64

FP8 (E4M3) pages (``reshape_and_cache_fp8``, ``decode_fp8``, ``verify_fp8``):
    k_cache       [num_blocks, num_kv_heads, block_size, head_dim] uint8 codes
    v_cache       [num_blocks, num_kv_heads, head_dim, block_size] uint8 codes
    k_scale,
    v_scale       [num_kv_heads] float32 (value = code value * scale)

INT4 pages (``reshape_and_cache_int4``, ``gather_cache_int4``, ``attention_int4``):
    k_cache,
    v_cache       [num_blocks, num_kv_heads, int4_page_bytes(head_dim)] uint8: 16 rows of
                  head_dim/2 code bytes, then 16 rows of head_dim/32 E4M3 scales
    k_scale,
    v_scale       [num_kv_heads] float32 (value = (code - 8) * scale * head scale)

Bounded caches (``accumulate_weights``, ``evict_tokens``; bf16, FP8 and INT4 pages):
    weights       [num_seqs, num_kv_heads, max_entries] float32
    positions     [num_seqs, num_kv_heads, max_entries] int32
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional

import numpy as np
import torch

from . import _lib
from ._lib import PagedAttnError, STATUS_NAMES

__all__ = ["reshape_and_cache", "decode", "verify", "decode_shared_prefix", "workspace_size",
           "default_partition_size", "get_device_error", "selftest_wait_timeout", "library",
           "copy_blocks", "BlockManager", "reshape_and_cache_fp8", "decode_fp8", "verify_fp8",
           "attention", "spec_accept", "GraphRunner", "reshape_and_cache_int4",
           "gather_cache_int4", "attention_int4", "int4_workspace_size", "int4_page_bytes",
           "accumulate_weights", "accumulate_workspace_size", "evict_tokens",
           "evict_workspace_size", "prompt_attention", "prompt_workspace_size",
           "extend_sequences", "truncate_sequences", "token_logprobs",
           "PagedAttnError", "STATUS_NAMES"]


def library() -> ctypes.CDLL:
    """The loaded ``libpaged_attn.so`` (raises ImportError if it was not built)."""
    return _lib.load()


def _vp(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _stream(dev: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need(name, t, dtype, ndim, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def reshape_and_cache(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, slot_mapping: torch.Tensor) -> None:
    """Scatter new K/V rows into their cache slots (in place, bit-exact)."""
    _need("k_cache", k_cache, torch.bfloat16, 4)
    dev = k_cache.device
    _need("v_cache", v_cache, torch.bfloat16, 4, dev)
    _need("key", key, torch.bfloat16, 3, dev)
    _need("value", value, torch.bfloat16, 3, dev)
    _need("slot_mapping", slot_mapping, torch.int64, 1, dev)
    NB, Hkv, BS, D = k_cache.shape
    N = key.shape[0]
    if v_cache.shape != k_cache.shape or key.shape != (N, Hkv, D) or value.shape != key.shape \
            or slot_mapping.shape[0] != N:
        raise ValueError("inconsistent shapes")
    st = library().pa_reshape_and_cache(_vp(key), _vp(value), _vp(k_cache), _vp(v_cache),
                                        _vp(slot_mapping), N, NB, Hkv, D, BS, _stream(dev))
    _lib.check("pa_reshape_and_cache", st)


def _fp8_pools(k_cache, v_cache, k_scale, v_scale):
    _need("k_cache", k_cache, torch.uint8, 4)
    dev = k_cache.device
    _need("v_cache", v_cache, torch.uint8, 4, dev)
    NB, Hkv, BS, D = k_cache.shape
    if tuple(v_cache.shape) != (NB, Hkv, D, BS):
        raise ValueError("v_cache must be [num_blocks, num_kv_heads, head_dim, block_size]")
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        _need(name, t, torch.float32, 1, dev)
        if t.shape[0] != Hkv:
            raise ValueError(f"{name} must have num_kv_heads entries")
    return dev, NB, Hkv, BS, D


def reshape_and_cache_fp8(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                          v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                          k_scale: torch.Tensor, v_scale: torch.Tensor) -> None:
    """Quantise new bf16 K/V rows to E4M3 (value / scale) and store them in FP8 pages."""
    dev, NB, Hkv, BS, D = _fp8_pools(k_cache, v_cache, k_scale, v_scale)
    _need("key", key, torch.bfloat16, 3, dev)
    _need("value", value, torch.bfloat16, 3, dev)
    _need("slot_mapping", slot_mapping, torch.int64, 1, dev)
    N = key.shape[0]
    if key.shape != (N, Hkv, D) or value.shape != key.shape or slot_mapping.shape[0] != N:
        raise ValueError("inconsistent shapes")
    st = library().pa_reshape_and_cache_fp8(_vp(key), _vp(value), _vp(k_cache), _vp(v_cache),
                                            _vp(slot_mapping), _vp(k_scale), _vp(v_scale), N,
                                            NB, Hkv, D, BS, _stream(dev))
    _lib.check("pa_reshape_and_cache_fp8", st)


def verify_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
               k_scale: torch.Tensor, v_scale: torch.Tensor, block_tables: torch.Tensor,
               context_lens: torch.Tensor, max_context_len: Optional[int] = None,
               scale: Optional[float] = None, partition_size: int = 0,
               workspace: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, new_key: Optional[torch.Tensor] = None,
               new_value: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``verify`` (T >= 1 query tokens per sequence) over FP8 pages.

    With ``new_key`` / ``new_value`` (bf16, [B*T, Hkv, D] or [B, T, Hkv, D]) the query
    tokens' K/V are quantised and stored at positions L-T .. L-1 inside the same launch.
    """
    dev, NB, Hkv, BS, D = _fp8_pools(k_cache, v_cache, k_scale, v_scale)
    _need("q", q, torch.bfloat16, 4, dev)
    _need("block_tables", block_tables, torch.int32, 2, dev)
    _need("context_lens", context_lens, torch.int32, 1, dev)
    B, T, Hq, Dq = q.shape
    if Dq != D or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("inconsistent shapes")
    if max_context_len is None:
        max_context_len = int(context_lens.max().item()) if B else T   # host sync
    mcl = int(max_context_len)
    if out is None:
        out = torch.empty_like(q)
    else:
        _need("out", out, torch.bfloat16, 4, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    need = workspace_size(B, Hq, T, mcl, D, BS, partition_size, 0) if B else 0
    ws, wsb = _workspace(dev, workspace, need)
    if new_key is not None or new_value is not None:
        for name, t in (("new_key", new_key), ("new_value", new_value)):
            if t is None or t.numel() != B * T * Hkv * D:
                raise ValueError(f"{name} must hold [B, T, Hkv, D] values")
            _need(name, t, torch.bfloat16, t.dim(), dev)
        st = library().pa_decode_append_fp8(
            _vp(out), _vp(q), _vp(new_key), _vp(new_value), _vp(k_cache), _vp(v_cache),
            _vp(k_scale), _vp(v_scale), _vp(block_tables), block_tables.shape[1],
            _vp(context_lens), mcl, B, T, NB, Hq, Hkv, D, BS, scale, partition_size, _vp(ws),
            wsb, _stream(dev))
        _lib.check("pa_decode_append_fp8", st)
        return out
    st = library().pa_verify_fp8(_vp(out), _vp(q), _vp(k_cache), _vp(v_cache), _vp(k_scale),
                                 _vp(v_scale), _vp(block_tables), block_tables.shape[1],
                                 _vp(context_lens), mcl, B, T, NB, Hq, Hkv, D, BS, scale,
                                 partition_size, _vp(ws), wsb, _stream(dev))
    _lib.check("pa_verify_fp8", st)
    return out


def attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              block_tables: torch.Tensor, context_lens: torch.Tensor,
              max_context_len: Optional[int] = None, scale: Optional[float] = None,
              partition_size: int = 0, workspace: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, new_key: Optional[torch.Tensor] = None,
              new_value: Optional[torch.Tensor] = None, window_size: int = 0,
              k_scale: Optional[torch.Tensor] = None,
              v_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The general per-sequence call (``pa_attention``): q [B, T, Hq, D]; bf16 pools, or FP8
    pools when ``k_scale`` / ``v_scale`` are given; optional fused append of the query
    tokens' K/V; ``window_size`` > 0 for sliding-window attention (each query token sees
    its last ``window_size`` positions)."""
    fp8 = k_scale is not None
    if fp8:
        dev, NB, Hkv, BS, D = _fp8_pools(k_cache, v_cache, k_scale, v_scale)
        _need("q", q, torch.bfloat16, 4, dev)
        _need("block_tables", block_tables, torch.int32, 2, dev)
        _need("context_lens", context_lens, torch.int32, 1, dev)
        B, T, Hq, Dq = q.shape
        if Dq != D or block_tables.shape[0] != B or context_lens.shape[0] != B:
            raise ValueError("inconsistent shapes")
        if max_context_len is None:
            max_context_len = int(context_lens.max().item()) if B else T   # host sync
        mcl = int(max_context_len)
        if out is None:
            out = torch.empty_like(q)
        else:
            _need("out", out, torch.bfloat16, 4, dev)
    else:
        dev, B, T, Hq, D, NB, Hkv, BS, mcl, out = _attn_common(q, k_cache, v_cache, block_tables,
                                                              context_lens, max_context_len, out)
    if (new_key is None) != (new_value is None):
        raise ValueError("new_key and new_value go together")
    if new_key is not None:
        for name, t in (("new_key", new_key), ("new_value", new_value)):
            if t.numel() != B * T * Hkv * D:
                raise ValueError(f"{name} must hold [B, T, Hkv, D] values")
            _need(name, t, torch.bfloat16, t.dim(), dev)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    need = workspace_size(B, Hq, T, mcl, D, BS, partition_size, 0) if B else 0
    ws, wsb = _workspace(dev, workspace, need)
    st = library().pa_attention(_vp(out), _vp(q), _vp(new_key), _vp(new_value), _vp(k_cache),
                                _vp(v_cache), _vp(k_scale), _vp(v_scale), 1 if fp8 else 0,
                                int(window_size), _vp(block_tables), block_tables.shape[1],
                                _vp(context_lens), mcl, B, T, NB, Hq, Hkv, D, BS, scale,
                                partition_size, _vp(ws), wsb, _stream(dev))
    _lib.check("pa_attention", st)
    return out


def decode_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
               k_scale: torch.Tensor, v_scale: torch.Tensor, block_tables: torch.Tensor,
               context_lens: torch.Tensor, max_context_len: Optional[int] = None,
               scale: Optional[float] = None, partition_size: int = 0,
               workspace: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, new_key: Optional[torch.Tensor] = None,
               new_value: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Single-token decode over FP8 pages; q is [B, Hq, D] or [B, 1, Hq, D].

    With ``new_key`` / ``new_value`` ([B, Hkv, D] bf16) the new token is quantised and
    stored at position L-1 of every sequence inside the same launch."""
    squeeze = q.dim() == 3
    q4 = q.unsqueeze(1) if squeeze else q
    if q4.shape[1] != 1:
        raise ValueError("decode_fp8 takes one query token per sequence (use verify_fp8)")
    o4 = None if out is None else (out.unsqueeze(1) if squeeze else out)
    r = verify_fp8(q4, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                   max_context_len, scale, partition_size, workspace, o4, new_key, new_value)
    return r.squeeze(1) if squeeze else r


def workspace_size(num_seqs: int, num_q_heads: int, num_query_tokens: int, max_context_len: int,
                   head_dim: int, block_size: int = 16, partition_size: int = 0,
                   max_prefix_blocks: int = 0) -> int:
    """Scratch bytes an attention call with these sizes needs (0 if none)."""
    return int(library().pa_workspace_size(num_seqs, num_q_heads, num_query_tokens,
                                           max_context_len, head_dim, block_size, partition_size,
                                           max_prefix_blocks))


def default_partition_size(num_seqs: int, num_kv_heads: int, max_context_len: int,
                           block_size: int = 16) -> int:
    return int(library().pa_default_partition_size(num_seqs, num_kv_heads, max_context_len,
                                                   block_size))


def _attn_common(q, k_cache, v_cache, block_tables, context_lens, max_context_len, out):
    _need("k_cache", k_cache, torch.bfloat16, 4)
    dev = k_cache.device
    _need("v_cache", v_cache, torch.bfloat16, 4, dev)
    _need("q", q, torch.bfloat16, 4, dev)
    _need("block_tables", block_tables, torch.int32, 2, dev)
    _need("context_lens", context_lens, torch.int32, 1, dev)
    B, T, Hq, D = q.shape
    NB, Hkv, BS, Dk = k_cache.shape
    if v_cache.shape != k_cache.shape or Dk != D or block_tables.shape[0] != B or \
            context_lens.shape[0] != B:
        raise ValueError("inconsistent shapes")
    if max_context_len is None:
        max_context_len = int(context_lens.max().item()) if B else T   # host sync
    if out is None:
        out = torch.empty_like(q)
    else:
        _need("out", out, torch.bfloat16, 4, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    return dev, B, T, Hq, D, NB, Hkv, BS, int(max_context_len), out


def _workspace(dev, workspace, need):
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not (workspace.is_cuda and workspace.device == dev and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor on the cache's device")
    return workspace, workspace.numel() * workspace.element_size()


def verify(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
           block_tables: torch.Tensor, context_lens: torch.Tensor,
           max_context_len: Optional[int] = None, scale: Optional[float] = None,
           partition_size: int = 0, workspace: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, new_key: Optional[torch.Tensor] = None,
           new_value: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of T draft tokens per sequence ([B, T, Hq, D]) with a causal mask among drafts.

    With ``new_key`` / ``new_value`` ([B*T, Hkv, D] or [B, T, Hkv, D]) the query tokens' K/V
    are first stored at positions L-T .. L-1 of every sequence, inside the same launch
    (reshape_and_cache fused).
    """
    dev, B, T, Hq, D, NB, Hkv, BS, mcl, out = _attn_common(q, k_cache, v_cache, block_tables,
                                                          context_lens, max_context_len, out)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    need = workspace_size(B, Hq, T, mcl, D, BS, partition_size, 0) if B else 0
    ws, wsb = _workspace(dev, workspace, need)
    lib = library()
    if new_key is not None or new_value is not None:
        for name, t in (("new_key", new_key), ("new_value", new_value)):
            if t is None or t.numel() != B * T * Hkv * D:
                raise ValueError(f"{name} must hold [B, T, Hkv, D] values")
            _need(name, t, torch.bfloat16, t.dim(), dev)
        st = lib.pa_decode_append(_vp(out), _vp(q), _vp(new_key), _vp(new_value), _vp(k_cache),
                                  _vp(v_cache), _vp(block_tables), block_tables.shape[1],
                                  _vp(context_lens), mcl, B, T, NB, Hq, Hkv, D, BS, scale,
                                  partition_size, _vp(ws), wsb, _stream(dev))
        _lib.check("pa_decode_append", st)
        return out
    if T == 1:
        st = lib.pa_decode(_vp(out), _vp(q), _vp(k_cache), _vp(v_cache), _vp(block_tables),
                           block_tables.shape[1], _vp(context_lens), mcl, B, NB, Hq, Hkv, D, BS,
                           scale, partition_size, _vp(ws), wsb, _stream(dev))
        _lib.check("pa_decode", st)
    else:
        st = lib.pa_verify(_vp(out), _vp(q), _vp(k_cache), _vp(v_cache), _vp(block_tables),
                           block_tables.shape[1], _vp(context_lens), mcl, B, T, NB, Hq, Hkv, D,
                           BS, scale, partition_size, _vp(ws), wsb, _stream(dev))
        _lib.check("pa_verify", st)
    return out


def decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
           block_tables: torch.Tensor, context_lens: torch.Tensor,
           max_context_len: Optional[int] = None, scale: Optional[float] = None,
           partition_size: int = 0, workspace: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, new_key: Optional[torch.Tensor] = None,
           new_value: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Single-token decode attention; q is [B, Hq, D] or [B, 1, Hq, D] (out has q's shape).

    With ``new_key`` / ``new_value`` ([B, Hkv, D]) the new token's K/V is stored at position
    L-1 of every sequence inside the same launch before attention reads it.
    """
    squeeze = q.dim() == 3
    q4 = q.unsqueeze(1) if squeeze else q
    if q4.shape[1] != 1:
        raise ValueError("decode takes one query token per sequence (use verify for drafts)")
    o4 = None if out is None else (out.unsqueeze(1) if squeeze else out)
    r = verify(q4, k_cache, v_cache, block_tables, context_lens, max_context_len, scale,
               partition_size, workspace, o4, new_key, new_value)
    return r.squeeze(1) if squeeze else r


def decode_shared_prefix(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                         block_tables: torch.Tensor, context_lens: torch.Tensor,
                         seq_group: torch.Tensor, group_prefix_blocks: torch.Tensor,
                         max_group_size: int, max_prefix_blocks: int,
                         max_context_len: Optional[int] = None, scale: Optional[float] = None,
                         partition_size: int = 0, workspace: Optional[torch.Tensor] = None,
                         out: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                         v_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Decode where groups of sequences share copy-on-write prefix blocks, read once per group.

    With ``k_scale`` / ``v_scale`` the pools are FP8 (E4M3) pages as for ``decode_fp8``."""
    squeeze = q.dim() == 3
    q4 = q.unsqueeze(1) if squeeze else q
    o4 = None if out is None else (out.unsqueeze(1) if squeeze else out)
    fp8 = k_scale is not None
    if fp8:
        dev, NB, Hkv, BS, D = _fp8_pools(k_cache, v_cache, k_scale, v_scale)
        _need("q", q4, torch.bfloat16, 4, dev)
        _need("block_tables", block_tables, torch.int32, 2, dev)
        _need("context_lens", context_lens, torch.int32, 1, dev)
        B, T, Hq, Dq = q4.shape
        if Dq != D or block_tables.shape[0] != B or context_lens.shape[0] != B:
            raise ValueError("inconsistent shapes")
        if max_context_len is None:
            max_context_len = int(context_lens.max().item()) if B else T   # host sync
        mcl = int(max_context_len)
        if o4 is None:
            o4 = torch.empty_like(q4)
        else:
            _need("out", o4, torch.bfloat16, 4, dev)
    else:
        dev, B, T, Hq, D, NB, Hkv, BS, mcl, o4 = _attn_common(q4, k_cache, v_cache, block_tables,
                                                             context_lens, max_context_len, o4)
    if T != 1:
        raise ValueError("decode_shared_prefix takes one query token per sequence")
    _need("seq_group", seq_group, torch.int32, 1, dev)
    _need("group_prefix_blocks", group_prefix_blocks, torch.int32, 1, dev)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    need = workspace_size(B, Hq, 1, mcl, D, BS, partition_size, max_prefix_blocks) if B else 0
    ws, wsb = _workspace(dev, workspace, need)
    if fp8:
        st = library().pa_decode_shared_prefix_fp8(
            _vp(o4), _vp(q4), _vp(k_cache), _vp(v_cache), _vp(k_scale), _vp(v_scale),
            _vp(block_tables), block_tables.shape[1], _vp(context_lens), mcl, B, NB, Hq, Hkv, D,
            BS, scale, partition_size, _vp(seq_group), _vp(group_prefix_blocks),
            group_prefix_blocks.shape[0], max_group_size, max_prefix_blocks, _vp(ws), wsb,
            _stream(dev))
        _lib.check("pa_decode_shared_prefix_fp8", st)
        return o4.squeeze(1) if squeeze else o4
    st = library().pa_decode_shared_prefix(
        _vp(o4), _vp(q4), _vp(k_cache), _vp(v_cache), _vp(block_tables), block_tables.shape[1],
        _vp(context_lens), mcl, B, NB, Hq, Hkv, D, BS, scale, partition_size, _vp(seq_group),
        _vp(group_prefix_blocks), group_prefix_blocks.shape[0], max_group_size,
        max_prefix_blocks, _vp(ws), wsb, _stream(dev))
    _lib.check("pa_decode_shared_prefix", st)
    return o4.squeeze(1) if squeeze else o4


def int4_page_bytes(head_dim: int) -> int:
    """Bytes of one INT4 page (16 tokens of one kv head)."""
    return 16 * (head_dim // 2 + head_dim // 32)


_KV_BF16, _KV_FP8, _KV_INT4 = 0, 1, 2


# The calls below are made once per layer and token, so their host time counts: arguments are
# checked with a few attribute reads each (``_need`` words the error), sizes of workspaces are
# computed once per shape, and pointers go to ctypes as plain integers.
_Tensor, _u8, _bf16, _f32, _i32, _i64 = (torch.Tensor, torch.uint8, torch.bfloat16, torch.float32,
                                         torch.int32, torch.int64)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _is(t, dtype, ndim, index):
    return (t.__class__ is _Tensor and t.dtype is dtype and t.get_device() == index
            and t.dim() == ndim and t.is_contiguous())


def _want(name, t, dtype, ndim, dev):
    if not _is(t, dtype, ndim, dev.index):
        _need(name, t, dtype, ndim, dev)


@functools.lru_cache(maxsize=None)
def _entry(name):
    return getattr(_lib.load(), name)


def _call(name, dev, *args):
    """library().name(*args, stream) with dev current, on its current stream."""
    index = dev.index
    stream = _raw_stream(index) if _raw_stream is not None else \
        torch.cuda.current_stream(dev).cuda_stream
    if torch.cuda.current_device() == index:
        st = _entry(name)(*args, stream)
    else:
        with torch.cuda.device(index):
            st = _entry(name)(*args, stream)
    if st:
        _lib.check(name, st)


def _scratch(dev, workspace, need):
    """(pointer, bytes, tensor to keep until the call is made)."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not (workspace.is_cuda and workspace.device == dev and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor on the cache's device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


_INT4_DIMS = {int4_page_bytes(d): d for d in (64, 128)}


def _int4_pools(k_cache, v_cache, k_scale, v_scale):
    if not isinstance(k_cache, _Tensor) or not k_cache.is_cuda:
        _need("k_cache", k_cache, _u8, 3)
    dev = k_cache.device
    index = dev.index
    if not (_is(k_cache, _u8, 3, index) and _is(v_cache, _u8, 3, index) and
            _is(k_scale, _f32, 1, index) and _is(v_scale, _f32, 1, index)):
        for name, t, dtype, ndim in (("k_cache", k_cache, _u8, 3), ("v_cache", v_cache, _u8, 3),
                                     ("k_scale", k_scale, _f32, 1), ("v_scale", v_scale, _f32, 1)):
            _need(name, t, dtype, ndim, dev)
    shape = k_cache.shape
    NB, Hkv, page = shape
    D = _INT4_DIMS.get(page)
    if D is None:
        raise ValueError("INT4 pools are [num_blocks, num_kv_heads, int4_page_bytes(head_dim)] "
                         f"with head_dim 64 or 128, got pages of {page} bytes")
    if v_cache.shape != shape:
        raise ValueError("inconsistent shapes")
    if k_scale.numel() != Hkv or v_scale.numel() != Hkv:
        raise ValueError("k_scale and v_scale must have num_kv_heads entries")
    return dev, NB, Hkv, D


def reshape_and_cache_int4(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                           v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                           k_scale: torch.Tensor, v_scale: torch.Tensor) -> None:
    """Quantise new bf16 K/V rows [N, Hkv, D] into INT4 pages at their slots (negative slots
    are skipped)."""
    dev, NB, Hkv, D = _int4_pools(k_cache, v_cache, k_scale, v_scale)
    _want("key", key, _bf16, 3, dev)
    _want("value", value, _bf16, 3, dev)
    _want("slot_mapping", slot_mapping, _i64, 1, dev)
    shape = key.shape
    N = shape[0]
    if shape != (N, Hkv, D) or value.shape != shape or slot_mapping.numel() != N:
        raise ValueError("inconsistent shapes")
    _call("pa_reshape_and_cache_int4", dev, key.data_ptr(), value.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), slot_mapping.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), N,
          NB, Hkv, D, 16)


def gather_cache_int4(k_cache: torch.Tensor, v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                      k_scale: torch.Tensor, v_scale: torch.Tensor):
    """The values held in INT4 slots as bf16: (key, value), each [N, Hkv, D]; rows with a
    negative slot are zero."""
    dev, NB, Hkv, D = _int4_pools(k_cache, v_cache, k_scale, v_scale)
    _want("slot_mapping", slot_mapping, _i64, 1, dev)
    N = slot_mapping.numel()
    key = torch.empty((N, Hkv, D), dtype=_bf16, device=dev)
    value = torch.empty_like(key)
    _call("pa_gather_cache_int4", dev, key.data_ptr(), value.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), slot_mapping.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), N,
          NB, Hkv, D, 16)
    return key, value


@functools.lru_cache(maxsize=1024)
def int4_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                        num_query_tokens: int, max_context_len: int, head_dim: int,
                        partition_size: int = 0, window_size: int = 0) -> int:
    """Scratch bytes ``attention_int4`` needs with these sizes (0 if none)."""
    return int(library().pa_int4_workspace_size(num_seqs, num_q_heads, num_kv_heads,
                                                num_query_tokens, max_context_len, head_dim, 16,
                                                partition_size, window_size))


def _max_len(max_context_len, context_lens, least):
    if max_context_len is None:
        max_context_len = context_lens.max().item() if context_lens.numel() else least  # host sync
    return int(max_context_len)


def attention_int4(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   k_scale: torch.Tensor, v_scale: torch.Tensor, block_tables: torch.Tensor,
                   context_lens: torch.Tensor, max_context_len: Optional[int] = None,
                   scale: Optional[float] = None, partition_size: int = 0,
                   workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   new_key: Optional[torch.Tensor] = None,
                   new_value: Optional[torch.Tensor] = None,
                   window_size: int = 0) -> torch.Tensor:
    """Attention over INT4 pages: q [B, T, Hq, D] or, for one query token, [B, Hq, D] (out has
    q's shape).

    With ``new_key`` / ``new_value`` ([B*T, Hkv, D] or [B, T, Hkv, D] bf16) the query tokens'
    K/V are quantised and stored at positions L-T .. L-1 first; ``window_size`` > 0 limits each
    query token to its last ``window_size`` positions.
    """
    dev, NB, Hkv, D = _int4_pools(k_cache, v_cache, k_scale, v_scale)
    index = dev.index
    ndim = 3 if isinstance(q, _Tensor) and q.dim() == 3 else 4
    if not (_is(q, _bf16, ndim, index) and _is(block_tables, _i32, 2, index) and
            _is(context_lens, _i32, 1, index)):
        _need("q", q, _bf16, ndim, dev)
        _need("block_tables", block_tables, _i32, 2, dev)
        _need("context_lens", context_lens, _i32, 1, dev)
    shape = q.shape
    if ndim == 4:
        B, T, Hq, Dq = shape
    else:
        (B, Hq, Dq), T = shape, 1
    rows, mbs = block_tables.shape
    if Dq != D or rows != B or context_lens.numel() != B:
        raise ValueError("inconsistent shapes")
    mcl = _max_len(max_context_len, context_lens, T)
    if out is None:
        out = torch.empty_like(q)
    else:
        _want("out", out, _bf16, ndim, dev)
        if out.shape != shape:
            raise ValueError("out must have q's shape")
    nk = nv = None
    if new_key is not None or new_value is not None:
        if new_key is None or new_value is None:
            raise ValueError("new_key and new_value go together")
        for name, t in (("new_key", new_key), ("new_value", new_value)):
            _want(name, t, _bf16, t.dim() if isinstance(t, _Tensor) else 3, dev)
            if t.numel() != B * T * Hkv * D:
                raise ValueError(f"{name} must hold [B, T, Hkv, D] values")
        nk, nv = new_key.data_ptr(), new_value.data_ptr()
    need = int4_workspace_size(B, Hq, Hkv, T, mcl, D, partition_size, window_size)
    ws, wsb, keep = _scratch(dev, workspace, need)
    _call("pa_attention_int4", dev, out.data_ptr(), q.data_ptr(), nk, nv, k_cache.data_ptr(),
          v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), int(window_size),
          block_tables.data_ptr(), mbs, context_lens.data_ptr(), mcl, B, T, NB, Hq, Hkv, D, 16,
          D ** -0.5 if scale is None else float(scale), partition_size, ws, wsb)
    return out


def _stat(name, t, dtype, dev, B, Hkv, mcl):
    _want(name, t, dtype, 3, dev)
    shape = t.shape
    if shape[0] != B or shape[1] != Hkv or shape[2] < mcl:
        raise ValueError(f"{name} must be [num_seqs, num_kv_heads, max_entries >= "
                         f"max_context_len], got {tuple(shape)}")
    return shape


def _kv_format(k_cache):
    """(format, dtype, dims) of a K pool by its type and shape."""
    if not isinstance(k_cache, _Tensor):
        raise TypeError("k_cache must be a torch.Tensor")
    if k_cache.dtype is _bf16:
        fmt = _KV_BF16, _bf16, 4
    elif k_cache.dim() == 3:
        fmt = _KV_INT4, _u8, 3
    else:
        fmt = _KV_FP8, _u8, 4
    if not (k_cache.is_cuda and _is(k_cache, fmt[1], fmt[2], k_cache.get_device())):
        _need("k_cache", k_cache, fmt[1], fmt[2])
    return fmt


@functools.lru_cache(maxsize=1024)
def accumulate_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                              num_query_tokens: int, max_context_len: int) -> int:
    """Scratch bytes ``accumulate_weights`` needs with these sizes."""
    return int(library().pa_accumulate_workspace_size(num_seqs, num_q_heads, num_kv_heads,
                                                      num_query_tokens, max_context_len))


def accumulate_weights(q: torch.Tensor, k_cache: torch.Tensor, block_tables: torch.Tensor,
                       context_lens: torch.Tensor, weights: torch.Tensor,
                       positions: Optional[torch.Tensor] = None,
                       seq_lens: Optional[torch.Tensor] = None,
                       max_context_len: Optional[int] = None, scale: Optional[float] = None,
                       decay: float = 1.0, k_scale: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Add the softmax weights of q [B, T, Hq, D] (or [B, Hq, D]) to each cache entry's sum.

    ``weights`` [B, Hkv, max_entries] float32 becomes ``decay * weights`` plus the weights
    each entry receives, in place or in ``out``; the T newest entries start afresh, and their
    ``positions`` are set from ``seq_lens`` (tokens seen by each sequence; default
    ``context_lens``).  The K pool may hold bf16, FP8 (with ``k_scale``) or INT4 pages (3-dim,
    with ``k_scale``).  All T tokens of every sequence count: of verified drafts, pass those
    that were accepted (one call for the sequences that kept the same number)."""
    fmt = _kv_format(k_cache)[0]
    dev = k_cache.device
    pool = k_cache.shape
    NB, Hkv = pool[0], pool[1]
    index = dev.index
    ndim = 3 if isinstance(q, _Tensor) and q.dim() == 3 else 4
    if not (_is(q, _bf16, ndim, index) and _is(block_tables, _i32, 2, index) and
            _is(context_lens, _i32, 1, index)):
        _need("q", q, _bf16, ndim, dev)
        _need("block_tables", block_tables, _i32, 2, dev)
        _need("context_lens", context_lens, _i32, 1, dev)
    shape = q.shape
    if ndim == 4:
        B, T, Hq, D = shape
    else:
        (B, Hq, D), T = shape, 1
    rows, mbs = block_tables.shape
    page = (NB, Hkv, int4_page_bytes(D)) if fmt == _KV_INT4 else (NB, Hkv, 16, D)
    if pool != page or rows != B or context_lens.numel() != B:
        raise ValueError("inconsistent shapes")
    if fmt == _KV_BF16:
        if k_scale is not None:
            raise ValueError("bf16 pages take no k_scale")
    else:
        _want("k_scale", k_scale, _f32, 1, dev)
        if k_scale.numel() != Hkv:
            raise ValueError("k_scale must have num_kv_heads entries")
    mcl = _max_len(max_context_len, context_lens, T)
    entries = _stat("weights", weights, _f32, dev, B, Hkv, mcl)
    if out is None:
        out = weights
    elif _stat("out", out, _f32, dev, B, Hkv, mcl) != entries:
        raise ValueError("out must have the shape of weights")
    if positions is not None and \
            _stat("positions", positions, _i32, dev, B, Hkv, mcl) != entries:
        raise ValueError("positions must have the shape of weights")
    if seq_lens is not None:
        _want("seq_lens", seq_lens, _i32, 1, dev)
        if seq_lens.numel() != B:
            raise ValueError("inconsistent shapes")
    need = accumulate_workspace_size(B, Hq, Hkv, T, mcl)
    ws, wsb, keep = _scratch(dev, workspace, need)
    _call("pa_accumulate_weights", dev, weights.data_ptr(), out.data_ptr(),
          None if positions is None else positions.data_ptr(), entries[2], q.data_ptr(),
          k_cache.data_ptr(), None if k_scale is None else k_scale.data_ptr(), fmt,
          block_tables.data_ptr(), mbs, context_lens.data_ptr(),
          None if seq_lens is None else seq_lens.data_ptr(), mcl, B, T, NB, Hq, Hkv, D, 16,
          D ** -0.5 if scale is None else float(scale), float(decay), ws, wsb)
    return out


@functools.lru_cache(maxsize=1024)
def evict_workspace_size(num_seqs: int, num_kv_heads: int, max_context_len: int,
                         budget: int) -> int:
    """Scratch bytes ``evict_tokens`` needs with these sizes."""
    return int(library().pa_evict_workspace_size(num_seqs, num_kv_heads, max_context_len, budget))


def evict_tokens(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                 context_lens: torch.Tensor, weights: torch.Tensor, positions: torch.Tensor,
                 budget: int, num_recent: int, max_context_len: Optional[int] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Cut every sequence with more than ``budget`` entries down to it, in place.

    Of each (sequence, kv head) the ``num_recent`` newest entries stay, and of the others
    those with the largest ``weights`` (ties: the lowest index); kept entries from ``budget``
    on move into the gaps below it, with their ``weights`` and ``positions``.  Returns the new
    context lengths (int32 [B], min(L, budget)).  Pools: bf16, FP8 or INT4 pages, owned by
    these sequences alone (no shared copy-on-write blocks)."""
    fmt, dtype, ndim = _kv_format(k_cache)
    dev = k_cache.device
    _want("v_cache", v_cache, dtype, ndim, dev)
    pool = k_cache.shape
    NB, Hkv = pool[0], pool[1]
    if fmt == _KV_INT4:
        BS, D = 16, _INT4_DIMS.get(pool[2], 0)
        good = D > 0 and v_cache.shape == pool
    else:
        BS, D = pool[2], pool[3]
        good = v_cache.shape == ((NB, Hkv, D, BS) if fmt == _KV_FP8 else pool)
    _want("block_tables", block_tables, _i32, 2, dev)
    _want("context_lens", context_lens, _i32, 1, dev)
    B = context_lens.numel()
    rows, mbs = block_tables.shape
    if not good or rows != B:
        raise ValueError("inconsistent shapes")
    mcl = max(1, _max_len(max_context_len, context_lens, 1))
    entries = _stat("weights", weights, _f32, dev, B, Hkv, mcl)
    if _stat("positions", positions, _i32, dev, B, Hkv, mcl) != entries:
        raise ValueError("positions must have the shape of weights")
    new_lens = torch.empty_like(context_lens)
    need = evict_workspace_size(B, Hkv, mcl, budget)
    ws, wsb, keep = _scratch(dev, workspace, need)
    _call("pa_evict_tokens", dev, new_lens.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), fmt,
          block_tables.data_ptr(), mbs, context_lens.data_ptr(), mcl, weights.data_ptr(),
          positions.data_ptr(), entries[2], int(budget), int(num_recent), B, NB, Hkv, D, BS, ws,
          wsb)
    return new_lens


def _int(x):
    """x for a 32-bit argument: ctypes would take a larger one modulo 2^32."""
    return max(-2 ** 31, min(2 ** 31 - 1, int(x)))


@functools.lru_cache(maxsize=1024)
def prompt_workspace_size(num_tokens: int, num_seqs: int, num_q_heads: int, num_kv_heads: int,
                          max_context_len: int, head_dim: int, partition_size: int = 0,
                          window_size: int = 0) -> int:
    """Scratch bytes ``prompt_attention`` needs with these sizes (0 if none)."""
    return int(library().pa_prompt_workspace_size(
        _int(num_tokens), _int(num_seqs), _int(num_q_heads), _int(num_kv_heads),
        _int(max_context_len), _int(head_dim), 16, _int(partition_size), _int(window_size)))


def prompt_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     block_tables: torch.Tensor, context_lens: torch.Tensor,
                     query_starts: torch.Tensor, max_context_len: Optional[int] = None,
                     scale: Optional[float] = None, window_size: int = 0,
                     partition_size: int = 0, workspace: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                     v_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention of packed prompts over their pages: q [N, Hq, D], of which rows
    ``query_starts[b] .. query_starts[b + 1] - 1`` (int32 [B + 1]) are the newest positions of
    sequence b's context, already stored in the cache (with a cached prefix in front of them, or
    none).  Any number of query tokens per sequence, 0 among them; rows of ``out`` that belong
    to no sequence are left as they are.  bf16 pools, or FP8 pools with ``k_scale`` /
    ``v_scale``; ``window_size`` > 0 limits each query token to its last ``window_size``
    positions."""
    fp8 = k_scale is not None or v_scale is not None
    if fp8:
        dev, NB, Hkv, BS, D = _fp8_pools(k_cache, v_cache, k_scale, v_scale)
    else:
        _need("k_cache", k_cache, _bf16, 4)
        dev = k_cache.device
        _want("v_cache", v_cache, _bf16, 4, dev)
        NB, Hkv, BS, D = k_cache.shape
        if v_cache.shape != k_cache.shape:
            raise ValueError("inconsistent shapes")
    _want("q", q, _bf16, 3, dev)
    _want("block_tables", block_tables, _i32, 2, dev)
    _want("context_lens", context_lens, _i32, 1, dev)
    _want("query_starts", query_starts, _i32, 1, dev)
    N, Hq, Dq = q.shape
    B, mbs = block_tables.shape
    if Dq != D or context_lens.numel() != B or query_starts.numel() != B + 1:
        raise ValueError("inconsistent shapes")
    mcl = _int(max(1, _max_len(max_context_len, context_lens, 1)))
    window_size, partition_size = _int(window_size), _int(partition_size)
    if out is None:
        out = torch.empty_like(q)
    else:
        _want("out", out, _bf16, 3, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    need = prompt_workspace_size(N, B, Hq, Hkv, mcl, D, partition_size, window_size)
    ws, wsb, keep = _scratch(dev, workspace, need)
    _call("pa_prompt_attention", dev, out.data_ptr(), q.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), k_scale.data_ptr() if fp8 else None,
          v_scale.data_ptr() if fp8 else None, _KV_FP8 if fp8 else _KV_BF16, window_size,
          block_tables.data_ptr(), mbs, context_lens.data_ptr(), mcl, query_starts.data_ptr(), N, B,
          NB, Hq, Hkv, D, BS, D ** -0.5 if scale is None else float(scale), partition_size, ws, wsb)
    return out


def _batch_state(block_tables, context_lens, ref_counts):
    if not isinstance(block_tables, _Tensor) or not block_tables.is_cuda:
        _need("block_tables", block_tables, _i32, 2)
    dev = block_tables.device
    _want("block_tables", block_tables, _i32, 2, dev)
    _want("context_lens", context_lens, _i32, 1, dev)
    _want("ref_counts", ref_counts, _i32, 1, dev)
    B, mbs = block_tables.shape
    if context_lens.numel() != B:
        raise ValueError("inconsistent shapes")
    return dev, B, mbs, ref_counts.numel()


def extend_sequences(block_tables: torch.Tensor, context_lens: torch.Tensor,
                     ref_counts: torch.Tensor, new_lens: torch.Tensor, num_tokens: int):
    """Take ``new_lens`` new tokens (int32 [B]) into every sequence, on the device.

    ``block_tables`` [B, max_blocks], ``context_lens`` [B] and ``ref_counts`` [num_blocks] (all
    int32; a block of count 0 is free) are updated in place, in the block manager's order: the
    lowest free block each time, a shared and partly filled last block replaced by a copy.
    Returns ``(query_starts [B + 1] int32, slot_mapping [num_tokens] int64, positions
    [num_tokens] int32, block_copies [B, 2] int32)``: the inputs of ``prompt_attention``,
    ``reshape_and_cache`` (rows behind the last token have slot -1) and ``copy_blocks`` ((0, 0)
    where there is nothing to copy).  ``num_tokens`` is a bound on the sum of ``new_lens``.  A
    call that cannot be met changes nothing, returns an empty batch and sets the device error."""
    dev, B, mbs, NB = _batch_state(block_tables, context_lens, ref_counts)
    _want("new_lens", new_lens, _i32, 1, dev)
    if new_lens.numel() != B:
        raise ValueError("inconsistent shapes")
    num_tokens = int(num_tokens)
    if not 0 <= num_tokens <= 2 ** 30:
        raise ValueError("num_tokens must be between 0 and 2^30")
    starts = torch.empty(B + 1, dtype=_i32, device=dev)
    slots = torch.empty(num_tokens, dtype=_i64, device=dev)
    positions = torch.empty(num_tokens, dtype=_i32, device=dev)
    copies = torch.empty((B, 2), dtype=_i32, device=dev)
    _call("pa_extend_sequences", dev, block_tables.data_ptr(), mbs, context_lens.data_ptr(),
          ref_counts.data_ptr(), new_lens.data_ptr(), B, num_tokens, NB, 16, starts.data_ptr(),
          slots.data_ptr(), positions.data_ptr(), copies.data_ptr())
    return starts, slots, positions, copies


def truncate_sequences(block_tables: torch.Tensor, context_lens: torch.Tensor,
                       ref_counts: torch.Tensor, new_context_lens: torch.Tensor) -> None:
    """Cut every sequence back to ``new_context_lens`` tokens (int32 [B], at most its length; 0
    frees it) in the state of ``extend_sequences``: blocks behind them lose an owner, their table
    entries become -1."""
    dev, B, mbs, NB = _batch_state(block_tables, context_lens, ref_counts)
    _want("new_context_lens", new_context_lens, _i32, 1, dev)
    if new_context_lens.numel() != B:
        raise ValueError("inconsistent shapes")
    _call("pa_truncate_sequences", dev, block_tables.data_ptr(), mbs, context_lens.data_ptr(),
          ref_counts.data_ptr(), new_context_lens.data_ptr(), B, NB, 16)


_LOGITS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, num_top: int = 0):
    """``(logprobs [N], entropy [N], top_logprobs [N, num_top], top_tokens [N, num_top])`` of
    logits [N, V] (float32, bf16 or fp16; rows may be strided) for the given tokens (int32 [N];
    negative: none).  Results are float32 in nats, the tokens int32; of equally probable
    alternatives the lower index comes first; ``num_top`` is at most 32."""
    if not isinstance(logits, _Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    dtype = _LOGITS.get(logits.dtype)
    if dtype is None:
        raise TypeError(f"logits must be float32, bfloat16 or float16, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError(f"logits must have 2 dims, got shape {tuple(logits.shape)}")
    N, V = logits.shape
    stride = logits.stride(0) if N > 1 else V
    if V > 1 and logits.stride(1) != 1 or stride < V:
        raise ValueError("the logits of a row must be contiguous, and rows must not overlap")
    dev = logits.device
    _want("tokens", tokens, _i32, 1, dev)
    if tokens.numel() != N:
        raise ValueError("inconsistent shapes")
    num_top = int(num_top)
    if not 0 <= num_top <= min(32, V):
        raise ValueError("num_top must be between 0 and 32 and at most the vocabulary")
    logprobs = torch.empty(N, dtype=_f32, device=dev)
    entropy = torch.empty(N, dtype=_f32, device=dev)
    top_logprobs = torch.empty((N, num_top), dtype=_f32, device=dev)
    top_tokens = torch.empty((N, num_top), dtype=_i32, device=dev)
    _call("pa_token_logprobs", dev, logprobs.data_ptr(), entropy.data_ptr(),
          top_logprobs.data_ptr(), top_tokens.data_ptr(), logits.data_ptr(), stride, dtype,
          tokens.data_ptr(), _int(N), _int(V), num_top)
    return logprobs, entropy, top_logprobs, top_tokens


def get_device_error(device=None) -> int:
    """Synchronise the current stream and return (and clear) the device error status."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else \
        torch.device(device)
    return int(library().pa_get_device_error(_stream(dev)))


LAST_KERNEL_NAMES = {0: "none", 1: "per_unit", 2: "persistent", 3: "tcgen05"}


def last_attention_kernel() -> str:
    """The kernel of this thread's last per-sequence attention launch: "none",
    "per_unit", "persistent" or "tcgen05" (a diagnostic)."""
    return LAST_KERNEL_NAMES[int(library().pa_last_attention_kernel())]


def selftest_wait_timeout(timeout_ns: int, device=None) -> None:
    """Launch the bounded-wait self test (read the outcome with get_device_error)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else \
        torch.device(device)
    _lib.check("pa_selftest_wait_timeout",
               library().pa_selftest_wait_timeout(int(timeout_ns), _stream(dev)))


def copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, pairs) -> None:
    """Copy whole physical blocks src -> dst in both pools (copy-on-write), bit-exact: bf16, FP8
    or INT4 pools.

    ``pairs``: sequence of (src, dst) ids or an int32 tensor [n, 2] (host or device), such as
    ``extend_sequences`` returns; a pair with src == dst copies nothing.
    """
    if not isinstance(k_cache, torch.Tensor):
        raise TypeError("k_cache must be a torch.Tensor")
    codes = k_cache.dtype == torch.uint8
    kind = (torch.uint8, 3 if k_cache.dim() == 3 else 4) if codes else (torch.bfloat16, 4)
    _need("k_cache", k_cache, *kind)
    dev = k_cache.device
    _need("v_cache", v_cache, *kind, dev)
    shape = tuple(k_cache.shape)
    if codes and len(shape) == 4:
        shape = (shape[0], shape[1], shape[3], shape[2])     # V pages lie by head dim
    if tuple(v_cache.shape) != shape:
        raise ValueError("inconsistent shapes")
    t = pairs if isinstance(pairs, torch.Tensor) else torch.tensor(list(pairs), dtype=torch.int32)
    t = t.to(device=dev, dtype=torch.int32).reshape(-1, 2).contiguous()
    if t.shape[0] == 0:
        return
    NB = shape[0]
    if codes:
        _call("pa_copy_block_bytes", dev, k_cache.data_ptr(), v_cache.data_ptr(), t.data_ptr(),
              t.shape[0], NB, k_cache[0].numel() if NB else 0)
        return
    _, Hkv, BS, D = shape
    st = library().pa_copy_blocks(_vp(k_cache), _vp(v_cache), _vp(t), t.shape[0], NB, Hkv, D, BS,
                                  _stream(dev))
    _lib.check("pa_copy_blocks", st)


def spec_accept(target_probs: torch.Tensor, draft_tokens: torch.Tensor,
                draft_probs: Optional[torch.Tensor] = None,
                accept_uniforms: Optional[torch.Tensor] = None,
                sample_uniforms: Optional[torch.Tensor] = None, greedy: bool = False):
    """Speculative acceptance after verify: (out_tokens [B, K+1] int32, num_accepted [B]).

    target_probs float32 [B, K+1, V]; draft_tokens int32 [B, K]; for sampling also
    draft_probs float32 [B, K, V], accept_uniforms uint32-valued int32/int64 [B, K] (low 24
    bits used) and sample_uniforms [B] (32-bit values).  Uniform tensors are passed as
    int32 views of the 32-bit patterns.
    """
    _need("target_probs", target_probs, torch.float32, 3)
    dev = target_probs.device
    B, K1, V = target_probs.shape
    K = K1 - 1
    _need("draft_tokens", draft_tokens, torch.int32, 2, dev)
    if tuple(draft_tokens.shape) != (B, K):
        raise ValueError("draft_tokens must be [B, K]")
    if not greedy:
        _need("draft_probs", draft_probs, torch.float32, 3, dev)
        _need("accept_uniforms", accept_uniforms, torch.int32, 2, dev)
        _need("sample_uniforms", sample_uniforms, torch.int32, 1, dev)
        if tuple(draft_probs.shape) != (B, K, V) or tuple(accept_uniforms.shape) != (B, K) \
                or sample_uniforms.shape[0] != B:
            raise ValueError("inconsistent shapes")
    out = torch.empty((B, K + 1), dtype=torch.int32, device=dev)
    kept = torch.empty(B, dtype=torch.int32, device=dev)
    st = library().pa_spec_accept(_vp(target_probs), _vp(draft_probs if not greedy else None),
                                  _vp(draft_tokens), _vp(accept_uniforms if not greedy else None),
                                  _vp(sample_uniforms if not greedy else None), B, K, V,
                                  1 if greedy else 0, _vp(out), _vp(kept), _stream(dev))
    _lib.check("pa_spec_accept", st)
    return out, kept


class GraphRunner:
    """CUDA graphs of the attention step for fixed batch-size classes (``pa_runner_*``).

    The runner captures one ``pa_attention`` call per class over static buffers sized for
    the largest class, which this object allocates and exposes: write a step's inputs into
    rows 0 .. B-1 of ``q``, ``new_key``, ``new_value``, ``block_tables`` and
    ``context_lens``, call ``step(B)``, read rows 0 .. B-1 of ``out``.  Rows B .. c-1 of
    the class c are padded on the device with a one-block sequence in ``pad_block`` (a
    physical block no sequence uses).  ``partition_size`` 0 captures each class with the
    library default for its batch size.

    With ``host_staging`` the runner also allocates page-locked host mirrors ``h_q``,
    ``h_new_key``, ``h_new_value``, ``h_block_tables``, ``h_context_lens`` and ``h_out``,
    and every class graph copies the inputs in and the output back itself: write the
    step's inputs into the host rows, call ``step(B)``, synchronise, read ``h_out``.
    """

    def __init__(self, k_cache: torch.Tensor, v_cache: torch.Tensor, num_q_heads: int,
                 max_context_len: int, max_blocks_per_seq: int, pad_block: int,
                 partition_size: int, classes=(1, 2, 4, 8, 16), num_query_tokens: int = 1,
                 scale: Optional[float] = None, window_size: int = 0, fused_append: bool = True,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                 host_staging: bool = False):
        self._lib = library()
        fp8 = k_scale is not None
        if fp8:
            dev, NB, Hkv, BS, D = _fp8_pools(k_cache, v_cache, k_scale, v_scale)
        else:
            _need("k_cache", k_cache, torch.bfloat16, 4)
            dev = k_cache.device
            _need("v_cache", v_cache, torch.bfloat16, 4, dev)
            NB, Hkv, BS, D = k_cache.shape
        classes = sorted(int(c) for c in classes)
        Bmax, T = classes[-1], int(num_query_tokens)
        self.classes = classes
        # the inputs live in one block (q, new_key, new_value, block_tables, context_lens,
        # 256-byte aligned), mirrored on the host when staging, so one copy moves them all
        shapes = [("q", (Bmax, T, num_q_heads, D), torch.bfloat16),
                  ("new_key", (Bmax * T, Hkv, D), torch.bfloat16),
                  ("new_value", (Bmax * T, Hkv, D), torch.bfloat16),
                  ("block_tables", (Bmax, max_blocks_per_seq), torch.int32),
                  ("context_lens", (Bmax,), torch.int32)]
        offs, total = [], 0
        for _, shp, dt in shapes:
            offs.append(total)
            n = int(np.prod(shp)) * torch.tensor([], dtype=dt).element_size()
            total += (n + 255) // 256 * 256

        def carve(block):
            return {name: block[o:o + int(np.prod(shp)) * torch.tensor([], dtype=dt)
                                .element_size()].view(dt).view(shp)
                    for (name, shp, dt), o in zip(shapes, offs)}

        self._dblock = torch.zeros(total, dtype=torch.uint8, device=dev)
        d = carve(self._dblock)
        self.q, self.block_tables, self.context_lens = d["q"], d["block_tables"], d["context_lens"]
        self.new_key = d["new_key"] if fused_append else None
        self.new_value = d["new_value"] if fused_append else None
        self.block_tables.fill_(pad_block)
        self.context_lens.fill_(T)
        self.out = torch.zeros_like(self.q)
        need = max(workspace_size(c, num_q_heads, T, max_context_len, D, BS, partition_size, 0)
                   for c in classes)
        self.workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        self._keep = (k_cache, v_cache, k_scale, v_scale)
        host = None
        if host_staging:
            self._hblock = torch.zeros(total, dtype=torch.uint8).pin_memory()
            hb = carve(self._hblock)
            self.h_q, self.h_block_tables = hb["q"], hb["block_tables"]
            self.h_context_lens = hb["context_lens"]
            self.h_new_key = hb["new_key"] if fused_append else None
            self.h_new_value = hb["new_value"] if fused_append else None
            self.h_block_tables.fill_(pad_block)
            self.h_context_lens.fill_(T)
            self.h_out = torch.empty(self.out.shape, dtype=self.out.dtype).pin_memory()
            host = (self.h_q.data_ptr(),
                    self.h_new_key.data_ptr() if fused_append else None,
                    self.h_new_value.data_ptr() if fused_append else None,
                    self.h_block_tables.data_ptr(), self.h_context_lens.data_ptr(),
                    self.h_out.data_ptr())
        self._classes_c = (ctypes.c_int * len(classes))(*classes)
        cfg = _lib.RunnerConfig(num_q_heads, Hkv, D, BS, T, max_blocks_per_seq, max_context_len,
                                NB, 1 if fp8 else 0, int(window_size), int(partition_size),
                                1.0 / math.sqrt(D) if scale is None else float(scale),
                                int(pad_block), len(classes), self._classes_c)
        bufs = _lib.RunnerBuffers(self.out.data_ptr(), self.q.data_ptr(),
                                  self.new_key.data_ptr() if fused_append else None,
                                  self.new_value.data_ptr() if fused_append else None,
                                  self.block_tables.data_ptr(), self.context_lens.data_ptr(),
                                  k_cache.data_ptr(), v_cache.data_ptr(),
                                  k_scale.data_ptr() if fp8 else None,
                                  v_scale.data_ptr() if fp8 else None,
                                  self.workspace.data_ptr(),
                                  self.workspace.numel(), *(host or (None,) * 6))
        h = ctypes.c_void_p()
        torch.cuda.synchronize(dev)
        _lib.check("pa_runner_create", self._lib.pa_runner_create(ctypes.byref(cfg),
                                                                  ctypes.byref(bufs),
                                                                  ctypes.byref(h)))
        self._h = h
        self.device = dev

    def class_of(self, num_seqs: int) -> int:
        return int(self._lib.pa_runner_class_of(self._h, num_seqs))

    def step(self, num_seqs: int) -> None:
        _lib.check("pa_runner_step", self._lib.pa_runner_step(self._h, num_seqs,
                                                              _stream(self.device)))

    def close(self):
        if getattr(self, "_h", None):
            self._lib.pa_runner_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class BlockManager:
    """Host-side block manager of the paged KV cache (the library's native C++ manager).

    Sequences own ordered lists of physical blocks; ``fork`` shares them; the
    first append into a shared, partly filled block returns a copy to perform
    (copy-on-write).  New blocks are the lowest-numbered free ones.
    """

    def __init__(self, num_blocks: int, block_size: int = 16):
        self._lib = library()
        h = ctypes.c_void_p()
        _lib.check("pa_bm_create", self._lib.pa_bm_create(num_blocks, block_size, ctypes.byref(h)))
        self._h = h
        self.num_blocks = num_blocks
        self.block_size = block_size

    def close(self):
        if self._h:
            self._lib.pa_bm_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def add_sequence(self, seq_id: int, num_tokens: int) -> None:
        _lib.check("pa_bm_add_sequence", self._lib.pa_bm_add_sequence(self._h, seq_id, num_tokens))

    def fork(self, parent_id: int, child_id: int) -> None:
        _lib.check("pa_bm_fork", self._lib.pa_bm_fork(self._h, parent_id, child_id))

    def append_slot(self, seq_id: int):
        """Reserve the next token's slot: returns (slot, copy) with copy = (src, dst) or None."""
        slot = ctypes.c_int64()
        src, dst = ctypes.c_int32(), ctypes.c_int32()
        _lib.check("pa_bm_append_slot", self._lib.pa_bm_append_slot(
            self._h, seq_id, ctypes.byref(slot), ctypes.byref(src), ctypes.byref(dst)))
        return slot.value, (None if src.value < 0 else (src.value, dst.value))

    def truncate(self, seq_id: int, num_tokens: int) -> None:
        """Shorten a sequence to its first ``num_tokens`` tokens and drop the blocks behind them
        (after ``evict_tokens``, or to take back rejected drafts)."""
        _lib.check("pa_bm_truncate", self._lib.pa_bm_truncate(self._h, seq_id, num_tokens))

    def free_sequence(self, seq_id: int) -> None:
        _lib.check("pa_bm_free_sequence", self._lib.pa_bm_free_sequence(self._h, seq_id))

    def block_table(self, seq_ids, max_blocks_per_seq: int):
        """(block_tables int32 [n, max_blocks], context_lens int32 [n]) as host tensors."""
        ids = torch.tensor(list(seq_ids), dtype=torch.int32)
        n = ids.numel()
        tables = torch.empty((n, max_blocks_per_seq), dtype=torch.int32)
        lens = torch.empty(n, dtype=torch.int32)
        _lib.check("pa_bm_block_table", self._lib.pa_bm_block_table(
            self._h, _vp(ids) if n else None, n, max_blocks_per_seq,
            _vp(tables) if n else None, _vp(lens) if n else None))
        return tables, lens

    def num_free_blocks(self) -> int:
        return int(self._lib.pa_bm_num_free_blocks(self._h))

    def ref_count(self, block: int) -> int:
        return int(self._lib.pa_bm_ref_count(self._h, block))

    def num_tokens(self, seq_id: int) -> int:
        return int(self._lib.pa_bm_num_tokens(self._h, seq_id))
