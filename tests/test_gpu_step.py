"""Block tables and slots of a batch on the device, against the oracle's block manager."""
import random

import numpy as np
import pytest
import torch

import paged_kv_cache_221_gb300 as pa
from step_cases import Batch

pytestmark = pytest.mark.gpu


def same(got, want):
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w), (g.cpu().numpy(), w)


def dev(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def extend(batch, state, new, spare=0):
    total = sum(new) + spare
    got = pa.extend_sequences(*state, dev(new), total)
    assert pa.get_device_error() == 0
    same(got, batch.extend(new, total))
    same(state, batch.arrays())
    return got


@pytest.mark.parametrize("spare", [0, 5])
@pytest.mark.parametrize("new", [[1], [0], [16], [17], [1, 0, 15, 16, 33], [0, 0, 0], [100, 1]])
def test_fresh_sequences(new, spare):
    b = Batch(40, 12)
    for _ in new:
        b.add(0)
    extend(b, b.upload(), new, spare)


def test_lengths_around_blocks():
    for n in (1, 2, 15, 16, 17):
        b = Batch(200, 9)
        for L in (0, 1, 14, 15, 16, 17, 31, 32, 33, 100):
            b.add(L)
        state = b.upload()
        extend(b, state, [n] * 10)
        extend(b, state, [n - 1] * 10, 3)


def test_shared_last_blocks():
    """Three owners of one partly filled block: the batch's order decides who copies."""
    for order in range(6):
        b = Batch(60, 8)
        b.add(37)
        b.add(32)
        b.fork(0)
        b.fork(0)
        b.fork(1)
        state = b.upload()
        r = random.Random(order)
        new = [r.choice([0, 1, 1, 20]) for _ in b.ids]
        got = extend(b, state, new)
        writers = sum(n > 0 for n in (new[0], new[2], new[3]))
        assert int((got[3][:, 0] != got[3][:, 1]).sum()) == min(writers, 2)
        extend(b, state, [1] * 5)
        extend(b, state, [1] * 5)


def test_forks_of_many_and_blocks_between():
    """Free blocks lie between used ones; forks of forks at every distance in the batch."""
    r = random.Random(3)
    b = Batch(3000, 40)
    for i in range(300):
        if i and r.random() < 0.4:
            b.fork(r.randrange(len(b.ids)))
        else:
            b.add(r.randrange(0, 90))
    state = b.upload()
    for step in range(4):
        extend(b, state, [r.choice([0, 1, 5, 30]) for _ in b.ids], r.choice([0, 9]))
        keep = [r.randint(0, b.m.tokens[i]) if r.random() < 0.5 else b.m.tokens[i] for i in b.ids]
        pa.truncate_sequences(*state, dev(keep))
        assert pa.get_device_error() == 0
        b.truncate(keep)
        same(state, b.arrays())


@pytest.mark.parametrize("B", [1, 31, 32, 1023, 1024, 1025, 2500])
def test_batch_sizes(B):
    r = random.Random(B)
    b = Batch(2 * B + 7, 4)
    for _ in range(B):
        b.add(r.choice([0, 3, 16]))
    extend(b, b.upload(), [r.choice([0, 1, 4]) for _ in range(B)], 2)


@pytest.mark.parametrize("NB", [1, 2, 3, 4, 5, 31, 33, 4095, 4097, 40001])
def test_pool_sizes(NB):
    """The last free blocks of pools of every size, those at the end too."""
    tables = torch.full((1, NB + 1), -1, dtype=torch.int32, device="cuda")
    lens, refs = dev([0]), torch.ones(NB, dtype=torch.int32, device="cuda")
    free = sorted(random.Random(NB).sample(range(NB), min(NB, 40)))
    refs[torch.tensor(free, device="cuda")] = 0
    starts, slots, pos, copies = pa.extend_sequences(tables, lens, refs, dev([16 * len(free)]),
                                                     16 * len(free))
    assert pa.get_device_error() == 0
    assert tables[0, :len(free)].tolist() == free and int(refs.min()) == 1
    assert slots.tolist() == [16 * f + i for f in free for i in range(16)]
    assert pos.tolist() == list(range(16 * len(free)))


def test_many_tokens():
    """The slots of a large burst have a launch of their own."""
    r = random.Random(9)
    b = Batch(9000, 900)
    for i in range(40):
        b.add(r.randrange(0, 200))
    b.fork(3)
    new = [r.choice([0, 1, 700]) for _ in b.ids]
    new[5] = 12000
    extend(b, b.upload(), new, 1000)


def test_calls_that_cannot_be_met():
    def state():
        b = Batch(10, 6)
        b.add(20)
        b.add(50)
        b.fork(0)
        return b, b.upload()
    BOUNDS, BLOCKS = 5, 7
    cases = [([60, 40, 1], 110, BLOCKS), ([1, 1, 1], 2, BOUNDS), ([77, 0, 0], 90, BOUNDS),
             ([-1, 1, 1], 9, BOUNDS), ([2 ** 31 - 1, 1, 1], 9, BOUNDS),
             ([2 ** 30, 2 ** 30, 2 ** 30], 9, BOUNDS)]
    for new, total, error in cases:
        b, st = state()
        got = pa.extend_sequences(*st, dev(new), total)
        assert pa.get_device_error() == error, new
        same(st, b.arrays())
        assert got[0].tolist() == [0] * 4 and got[1].tolist() == [-1] * total
        assert got[2].tolist() == [-1] * total and got[3].tolist() == [[0, 0]] * 3
        assert pa.get_device_error() == 0
    b, st = state()
    st[0][1, 3] = 10                                     # the last block is outside the pool
    pa.extend_sequences(*st, dev([0, 1, 0]), 1)
    assert pa.get_device_error() == BOUNDS
    b, st = state()
    got = pa.extend_sequences(*st, dev([16384, 0, 0]), 20000)    # past the table, many tokens
    assert pa.get_device_error() == BOUNDS
    assert int(got[1].max()) == -1 and int(got[2].max()) == -1
    b, st = state()                                      # to the last free block: 4, one a copy
    extend(b, st, [12 + 32, 14 + 16, 0])
    assert int(st[2].min()) == 1


def test_truncation_refused():
    b = Batch(12, 4)
    b.add(20)
    b.add(33)
    st = b.upload()
    pa.truncate_sequences(*st, dev([21, 10]))
    assert pa.get_device_error() == 5
    b.truncate([20, 10])
    same(st, b.arrays())
    pa.truncate_sequences(*st, dev([-1, 10]))
    assert pa.get_device_error() == 5
    st[2][st[0][0, 1].long()] = 0                        # an entry that nobody owns
    pa.truncate_sequences(*st, dev([1, 0]))
    assert pa.get_device_error() == 5
    assert int(st[2].min()) == 0 and st[1].tolist() == [1, 0]


def test_stream_graph_and_empty():
    b = Batch(100, 8)
    for L in (5, 16, 40):
        b.add(L)
    st = b.upload()
    kept = [x.clone() for x in st]
    new = dev([3, 20, 1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = pa.extend_sequences(*st, new, 30)
    s.synchronize()
    want = b.extend([3, 20, 1], 30)
    same(got, want)
    for x, y in zip(st, kept):
        x.copy_(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = pa.extend_sequences(*st, new, 30)
    g.replay()
    torch.cuda.synchronize()
    same(got, want)
    same(st, b.arrays())
    new.fill_(1)
    g.replay()
    torch.cuda.synchronize()
    same(got, b.extend([1, 1, 1], 30))
    none = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    got = pa.extend_sequences(none, none[:, 0], st[2], none[:, 0], 3)
    assert got[0].tolist() == [0] and got[1].tolist() == [-1] * 3 and got[2].tolist() == [-1] * 3
    pa.truncate_sequences(none, none[:, 0], st[2], none[:, 0])
    assert pa.get_device_error() == 0


def test_refusals():
    b = Batch(10, 4)
    b.add(3)
    t, n, r = b.upload()
    new = dev([1])
    with pytest.raises(TypeError):
        pa.extend_sequences(t, n, r, new.long(), 1)
    with pytest.raises(ValueError):
        pa.extend_sequences(t, n, r, dev([1, 1]), 2)
    with pytest.raises(ValueError):
        pa.extend_sequences(t, n, r, new, -1)
    with pytest.raises(ValueError):
        pa.extend_sequences(t.repeat(1, 2)[:, ::2], n, r, new, 1)
    with pytest.raises(ValueError):
        pa.truncate_sequences(t, dev([1, 1]), r, new)
    with pytest.raises(pa.PagedAttnError):
        pa.truncate_sequences(t, n, r, n)
    big = torch.zeros((12289, 1), dtype=torch.int32, device="cuda")
    with pytest.raises(pa.PagedAttnError):
        pa.extend_sequences(big, big[:, 0].contiguous(), r, big[:, 0].contiguous(), 1)


def test_new_lengths_past_32_bits():
    """Four sequences of 2^30 new tokens: their sum is 0 in 32 bits, the call is not met."""
    tables = torch.empty(4, 2 ** 26, dtype=torch.int32, device="cuda")
    lens, refs = dev([0] * 4), dev([0] * 64)
    starts, slots, pos, copies = pa.extend_sequences(tables, lens, refs, dev([2 ** 30] * 4), 16)
    assert pa.get_device_error() == 5
    assert starts.tolist() == [0] * 5 and slots.tolist() == [-1] * 16 and pos.tolist() == [-1] * 16
    assert not copies.any() and not lens.any() and not refs.any()


def test_last_block_without_an_owner():
    """It counts as free and would be handed out to two sequences."""
    b = Batch(8, 4)
    b.add(20)
    b.add(5)
    st = b.upload()
    st[2][st[0][0, 1].long()] = 0
    before = [x.clone() for x in st]
    got = pa.extend_sequences(*st, dev([1, 20]), 21)
    assert pa.get_device_error() == 5 and int(got[1].max()) == -1
    assert all(torch.equal(x, y) for x, y in zip(before, st))
    with pytest.raises(pa.PagedAttnError):
        pa.extend_sequences(*st, st[1], 25)


def test_largest_batch():
    b = Batch(20000, 3)
    for i in range(12288):
        b.add((0, 3, 16)[i % 3])
    state = b.upload()
    extend(b, state, [i % 2 for i in range(12288)])
    with pytest.raises(pa.PagedAttnError):
        pa.extend_sequences(torch.zeros((12289, 1), dtype=torch.int32, device="cuda"),
                            dev([0] * 12289), state[2], dev([0] * 12289), 1)
