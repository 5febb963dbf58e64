"""Random paged caches for the INT4-page and bounded-cache tests, in every page format."""
import numpy as np

import workloads as W
from oracle import fp8 as F
from oracle import int4 as Q4
from oracle import oracle as O

BLOCK = 16


class Case:
    """A paged cache with sequences of the given lengths, on the host.

    Pages are those of N(0, 1) values; slots that hold no token hold garbage, NaN among it.
    """

    def __init__(self, seed, lens, Hq, Hkv, D, T=1, fmt="int4", spare=3, extra_blocks=0,
                 power_of_two=False):
        rng = np.random.default_rng(seed)
        self.fmt, self.D, self.T, self.Hq, self.Hkv = fmt, D, T, Hq, Hkv
        self.lens = np.asarray(lens, dtype=np.int32)
        self.scale = 1.0 / np.sqrt(D)
        B = len(lens)
        need = [-(-n // BLOCK) for n in lens]
        self.mbs = max(max(need), 1) + extra_blocks
        self.NB = sum(need) + spare
        ids = rng.permutation(self.NB)
        self.tables = np.zeros((B, self.mbs), dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = ids[at:at + n]
            at += n
        self.q = W.f32_to_bf16_bits(rng.standard_normal((B, T, Hq, D)).astype(np.float32))
        used = np.zeros((self.NB, BLOCK), dtype=bool)
        for b, n in enumerate(lens):
            for j in range(n):
                used[self.tables[b, j // BLOCK], j % BLOCK] = True
        s = rng.uniform(0.02, 0.3, (2, Hkv)).astype(np.float32)
        if power_of_two:
            s = np.exp2(np.rint(np.log2(s))).astype(np.float32)
        self.k_scale, self.v_scale = s
        self.new_key, self.new_value = (
            W.f32_to_bf16_bits(rng.standard_normal((B * T, Hkv, D)).astype(np.float32))
            for _ in range(2))
        self.slots = np.array([int(self.tables[b, j // BLOCK]) * BLOCK + j % BLOCK
                               for b, n in enumerate(lens) for j in range(n - T, n)],
                              dtype=np.int64)
        for name in ("k", "v"):
            x = W.f32_to_bf16_bits(
                rng.standard_normal((self.NB, Hkv, BLOCK, D)).astype(np.float32))
            if fmt == "bf16":
                x = np.where(used[:, None, :, None], x, np.uint16(0x7FC0))
            elif fmt == "fp8":
                scale = self.k_scale if name == "k" else self.v_scale
                c = np.stack([F.quantize(x[:, h], scale[h]) for h in range(Hkv)], 1)
                x = np.where(used[:, None, :, None], c, np.uint8(0x7F))
                x = np.ascontiguousarray(x.swapaxes(-1, -2)) if name == "v" else x
            else:
                scale = self.k_scale if name == "k" else self.v_scale
                parts = [Q4.quantize(x[:, h], scale[h]) for h in range(Hkv)]
                codes = np.stack([p[0] for p in parts], 1)
                sc = np.stack([p[1] for p in parts], 1)
                sc = np.where(used[:, None, :, None], sc, np.uint8(0x7F))
                x = Q4.pack(codes, sc)
            setattr(self, name, x)

    def rows(self, pool, b, g, n, name):
        """fp64 rows 0 .. n-1 of kv head g of sequence b from `pool` (host array)."""
        if self.fmt == "bf16":
            return O.gather_context(pool, self.tables[b], n, g, BLOCK)
        if self.fmt == "fp8":
            fn = F.gather_k if name == "k" else F.gather_v
            scale = self.k_scale if name == "k" else self.v_scale
            return fn(pool, self.tables[b], n, g, scale, BLOCK)
        scale = self.k_scale if name == "k" else self.v_scale
        return Q4.rows(pool, self.tables[b], n, g, scale[g], self.D)

    def score_size(self, keys):
        """Largest sum_d |q_d k_d| * scale * log2(e): what score rounding is relative to."""
        q = np.abs(O.bf16_bits_to_f64(self.q))
        G = self.Hq // self.Hkv
        big = 0.0
        for b in range(len(self.lens)):
            for g in range(self.Hkv):
                if len(keys[b][g]):
                    x = q[b, :, g * G:(g + 1) * G].reshape(-1, self.D) @ np.abs(keys[b][g]).T
                    big = max(big, x.max())
        return big * self.scale * 1.4427
