"""Batches of sequences on the host, as the oracle block manager keeps them."""
import numpy as np
import torch

from oracle.block_manager import BlockManager, OutOfBlocks


class Batch:
    """A batch on the device beside the same batch in the oracle's manager."""

    def __init__(self, num_blocks, mbs, device="cuda"):
        self.m = BlockManager(num_blocks, 16)
        self.NB, self.mbs, self.device = num_blocks, mbs, device
        self.ids = []

    def add(self, n):
        self.m.add_sequence(len(self.ids), n)
        self.ids.append(len(self.ids))

    def fork(self, parent):
        self.m.fork(parent, len(self.ids))
        self.ids.append(len(self.ids))

    def arrays(self):
        tables = np.full((len(self.ids), self.mbs), -1, dtype=np.int32)
        for r, b in enumerate(self.ids):
            tables[r, :len(self.m.tables[b])] = self.m.tables[b]
        lens = np.array([self.m.tokens[b] for b in self.ids], dtype=np.int32)
        return tables, lens, np.array(self.m.refs, dtype=np.int32)

    def upload(self):
        return [torch.from_numpy(a).to(self.device) for a in self.arrays()]

    def extend(self, new, num_tokens):
        """The outputs of a call that is met (the manager moves on); None if it has no blocks."""
        starts, slots, positions, copies = [0], [], [], []
        before = (list(self.m.refs), {k: list(v) for k, v in self.m.tables.items()},
                  dict(self.m.tokens))
        try:
            for b, n in zip(self.ids, new):
                copy = (0, 0)
                for _ in range(n):
                    positions.append(self.m.tokens[b])
                    slot, made = self.m.append_slot(b)
                    slots.append(slot)
                    copy = made or copy
                copies.append(copy)
                starts.append(len(slots))
        except OutOfBlocks:
            self.m.refs, self.m.tables, self.m.tokens = before
            return None
        behind = [-1] * (num_tokens - len(slots))
        return (np.array(starts, dtype=np.int32), np.array(slots + behind, dtype=np.int64),
                np.array(positions + behind, dtype=np.int32),
                np.array(copies, dtype=np.int32).reshape(len(self.ids), 2))

    def truncate(self, keep):
        for b, n in zip(self.ids, keep):
            table = self.m.tables[b]
            while len(table) > -(-n // 16):
                self.m.refs[table.pop()] -= 1
            self.m.tokens[b] = n
