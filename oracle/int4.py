"""fp64 CPU oracle for INT4 KV pages.

TEST INFRASTRUCTURE ONLY (same rules as ``oracle.py``; it shares no code with the CUDA
path).

A page is 16 tokens of one (block, kv head): 16 rows of D/2 bytes, dim d in byte d/2 (even d
in the low nibble), then 16 rows of D/32 E4M3 scale bytes, one for 32 dims.  A value is
``(code - 8) * e4m3(scale) * head_scale``.  Writing a token: the scale is the E4M3 value nearest
to ``max|x| / (7 head_scale)`` (float32 product and quotient; ties to even, saturating), the
code the integer nearest to ``x / (scale * head_scale)`` (the product in float32, the
comparison exact, ties to even), limited to -7 .. 7, plus 8; a zero or NaN scale gives code 8.
"""
from __future__ import annotations

import numpy as np

from . import fp8 as F
from . import oracle as O

GROUP = 32
BLOCK = 16


def page_bytes(D: int) -> int:
    return BLOCK * (D // 2 + D // GROUP)


def quantize(bits_bf16: np.ndarray, head_scale: float):
    """(codes uint8 [..., D], scale bytes uint8 [..., D/32]) of bf16 rows [..., D]."""
    x = O.bf16_bits_to_f64(bits_bf16)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    hs = np.float32(head_scale)
    with np.errstate(invalid="ignore", over="ignore"):
        amax = np.abs(g).max(-1)                      # NaN if the group holds one
        scales = F.encode((amax.astype(np.float32) / (np.float32(7) * hs)).astype(np.float64))
        step = (F.decode(scales).astype(np.float32) * hs).astype(np.float64)[..., None]
        good = step > 0
        q = np.where(good, g / np.where(good, step, 1.0), 0.0)
        codes = np.clip(np.rint(q), -7, 7) + 8
    return codes.astype(np.uint8).reshape(x.shape), scales


def dequantize(codes: np.ndarray, scales: np.ndarray, head_scale: float) -> np.ndarray:
    """fp64 values of codes [..., D] and scale bytes [..., D/32]."""
    step = F.decode(scales) * float(np.float32(head_scale))
    return (codes.astype(np.float64) - 8.0) * np.repeat(step, GROUP, axis=-1)


def pack(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Pages uint8 [..., page_bytes] of codes [..., 16, D] and scales [..., 16, D/32]."""
    rows = codes[..., 0::2] | (codes[..., 1::2] << 4)
    lead = codes.shape[:-2]
    return np.concatenate([rows.reshape(*lead, -1), scales.reshape(*lead, -1)], -1)


def unpack(pages: np.ndarray, D: int):
    """(codes [..., 16, D], scales [..., 16, D/32]) of pages."""
    rows = pages[..., :BLOCK * D // 2].reshape(*pages.shape[:-1], BLOCK, D // 2)
    codes = np.empty((*rows.shape[:-1], D), dtype=np.uint8)
    codes[..., 0::2] = rows & 15
    codes[..., 1::2] = rows >> 4
    return codes, pages[..., BLOCK * D // 2:].reshape(*pages.shape[:-1], BLOCK, D // GROUP)


def reshape_and_cache(key, value, k_pages, v_pages, slots, k_scale, v_scale):
    """New pools with each token's quantised K/V in its slot; negative slots are skipped."""
    out = []
    D = key.shape[-1]
    for new, pages, scale in ((key, k_pages, k_scale), (value, v_pages, v_scale)):
        codes, sc = unpack(np.array(pages, copy=True), D)
        sc = np.array(sc, copy=True)
        for i, slot in enumerate(np.asarray(slots).tolist()):
            if slot < 0:
                continue
            for h in range(pages.shape[1]):
                c, s = quantize(new[i, h], scale[h])
                codes[slot // BLOCK, h, slot % BLOCK] = c
                sc[slot // BLOCK, h, slot % BLOCK] = s
        out.append(pack(codes, sc))
    return out


def rows(pages, table, n, h, head_scale, D):
    """fp64 values of entries 0 .. n-1 of kv head h of one sequence."""
    j = np.arange(n)
    codes, sc = unpack(pages[np.asarray(table)[j // BLOCK], h], D)
    return dequantize(codes[j, j % BLOCK], sc[j, j % BLOCK], head_scale)


def attention(q_bits, k_pages, v_pages, k_scale, v_scale, tables, lens, scale, window=0):
    """(out, mag): fp64 attention [B, T, Hq, D], and sum_j p_j |v_j| for error bounds."""
    B, T, Hq, D = q_bits.shape
    Hkv = k_pages.shape[1]
    out, mag = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq, D))
    for b in range(B):
        L = int(lens[b])
        for g in range(Hkv):
            K = rows(k_pages, tables[b], L, g, k_scale[g], D)
            V = rows(v_pages, tables[b], L, g, v_scale[g], D)
            for h in range(g * Hq // Hkv, (g + 1) * Hq // Hkv):
                for t in range(T):
                    last = L - T + t
                    first = max(0, last - window + 1) if window else 0
                    q = O.bf16_bits_to_f64(q_bits[b, t, h])
                    p = O.softmax(O.scores(K[first:last + 1], q, scale))
                    out[b, t, h] = p @ V[first:last + 1]
                    mag[b, t, h] = p @ np.abs(V[first:last + 1])
    return out, mag
