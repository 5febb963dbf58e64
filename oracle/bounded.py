"""fp64 CPU oracle for accumulated attention weights and eviction.

TEST INFRASTRUCTURE ONLY (same rules as ``oracle.py``; it shares no code with the CUDA
path).  The cache is given as dense rows per (sequence, kv head); pages are gathered and
scattered by the caller.
"""
from __future__ import annotations

import math

import numpy as np

from . import oracle as O


def accumulate(weights, positions, q_bits, keys, lens, seq_lens, scale, decay):
    """(weights, positions, gained): the arrays after one call, and the sum each entry gained.

    weights float64 and positions int [B, Hkv, E]; keys[b][g] fp64 [L, D]."""
    B, T, Hq, _ = q_bits.shape
    Hkv = weights.shape[1]
    w, pos, gained = weights.copy(), positions.copy(), np.zeros_like(weights)
    for b in range(B):
        L = int(lens[b])
        for g in range(Hkv):
            new = np.zeros(L)
            for h in range(g * Hq // Hkv, (g + 1) * Hq // Hkv):
                for t in range(T):
                    n = L - T + t + 1
                    q = O.bf16_bits_to_f64(q_bits[b, t, h])
                    new[:n] += O.softmax(O.scores(keys[b][g][:n], q, scale))
            gained[b, g, :L] = new
            w[b, g, :L - T] = decay * weights[b, g, :L - T] + new[:L - T]
            w[b, g, L - T:L] = new[L - T:]
            pos[b, g, L - T:L] = int(seq_lens[b]) - T + np.arange(T)
    return w, pos, gained


def select(weights, positions, budget, num_recent):
    """The moves [(from, to), ...] that cut one (sequence, kv head) to `budget` entries."""
    n = len(weights)
    if n <= budget:
        return []
    newest = max(int(x) for x in positions)

    def order(j):
        w = float(weights[j])
        protected = int(positions[j]) > newest - num_recent
        # newest first, then larger weights (NaN last), then the lower index
        return (not protected, math.isnan(w), 0.0 if math.isnan(w) else -w, j)

    keep = set(sorted(range(n), key=order)[:budget])
    gaps = [j for j in range(budget) if j not in keep]
    movers = [j for j in range(budget, n) if j in keep]
    assert len(gaps) == len(movers)
    return list(zip(movers, gaps))
