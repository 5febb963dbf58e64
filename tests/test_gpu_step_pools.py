"""Block tables on the device over large pools, and reference counts at any address, against the
oracle's block manager."""
import random

import pytest
import torch

import paged_kv_cache_221_gb300 as pa
from test_gpu_step import dev, extend, same
from step_cases import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at", [0, 1, 2, 3])
@pytest.mark.parametrize("NB", [262143, 262144, 262145, 600001, 2 ** 22 + 5])
def test_pools_of_many_blocks(NB, at):
    """A thread looks after more than 32 blocks: free ones at both ends of the pool, at the ends of
    a thread's groups of 32, and anywhere, with counts that start `at` elements behind a 16-byte
    boundary."""
    r = random.Random(NB + at)
    run = -(-NB // (4 * 8192)) * 4                       # blocks of a thread
    run = -(-run // 32) * 32 if run > 32 else run
    free = {0, 1, NB - 1, NB - 2, NB - 33}
    for first in (0, run, 100 * run, NB // run * run):
        free |= {first + k for k in (0, 31, 32, 33, 63, run - 1) if first + k < NB}
    free = sorted(free | set(r.sample(range(NB), 60)))
    refs = torch.ones(NB + 4, dtype=torch.int32, device="cuda")[at:at + NB]
    assert refs.data_ptr() % 16 == 4 * at
    refs[torch.tensor(free, device="cuda")] = 0
    lens = [0] * 4
    tables = torch.full((4, 80), -1, dtype=torch.int32, device="cuda")
    state = [tables, dev(lens), refs]
    new = [16 * 20 + 1, 0, 3, 16 * (len(free) - 22) - 7]
    # a call that takes one block too many changes nothing
    pa.extend_sequences(*state, dev([n + 16 * (b == 3) for b, n in enumerate(new)]), sum(new) + 16)
    assert pa.get_device_error() == 7 and int((refs == 0).sum()) == len(free)
    starts, slots, pos, copies = pa.extend_sequences(*state, dev(new), sum(new) + 3)
    assert pa.get_device_error() == 0
    blocks = [free[:21], [], free[21:22], free[22:]]
    want, where = [], []
    for n, ids in zip(new, blocks):
        want += [ids[i // 16] * 16 + i % 16 for i in range(n)]
        where += range(n)
    assert slots.tolist() == want + [-1] * 3 and pos.tolist() == where + [-1] * 3
    assert starts.tolist() == [0, new[0], new[0], new[0] + 3, sum(new)] and not copies.any()
    for b, ids in enumerate(blocks):
        assert tables[b].tolist() == ids + [-1] * (80 - len(ids))
    assert bool((refs == 1).all())
    pa.truncate_sequences(*state, dev([0] * 4))
    assert pa.get_device_error() == 0
    assert (refs == 0).nonzero()[:, 0].tolist() == free and bool((tables == -1).all())


@pytest.mark.parametrize("at", [1, 3])
def test_batches_with_counts_at_any_address(at):
    """Forks, copies and blocks given back."""
    r = random.Random(at)
    b = Batch(4000, 40)
    for i in range(200):
        if i and r.random() < 0.4:
            b.fork(r.randrange(len(b.ids)))
        else:
            b.add(r.randrange(0, 90))
    state = b.upload()
    refs = torch.zeros(4004, dtype=torch.int32, device="cuda")[at:at + 4000]
    refs.copy_(state[2])
    state[2] = refs
    for _ in range(3):
        extend(b, state, [r.choice([0, 1, 5, 30]) for _ in b.ids], r.choice([0, 9]))
        keep = [r.randint(0, b.m.tokens[i]) if r.random() < 0.5 else b.m.tokens[i] for i in b.ids]
        pa.truncate_sequences(*state, dev(keep))
        assert pa.get_device_error() == 0
        b.truncate(keep)
        same(state, b.arrays())
