"""Copy-on-write of pools of every page format, with the pairs that extend_sequences reports."""
import pytest
import torch

import paged_kv_cache_221_gb300 as pa
from step_cases import Batch

pytestmark = pytest.mark.gpu


def pools(kind, NB, Hkv, D, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "bf16":
        shapes, dtype = [(NB, Hkv, 16, D)] * 2, torch.bfloat16
    elif kind == "fp8":
        shapes, dtype = [(NB, Hkv, 16, D), (NB, Hkv, D, 16)], torch.uint8
    else:
        shapes, dtype = [(NB, Hkv, pa.int4_page_bytes(D))] * 2, torch.uint8
    out = []
    for s in shapes:
        n = (2 if dtype == torch.bfloat16 else 1) * torch.Size(s).numel()
        out.append(torch.randint(0, 256, (n,), dtype=torch.uint8, generator=g,
                                 device="cuda").view(dtype).view(s))
    return out


def raw(pool):
    return pool.view(torch.uint8).view(pool.shape[0], -1)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (3, 64), (8, 128)])
def test_pairs(kind, Hkv, D):
    k, v = pools(kind, 40, Hkv, D)
    before = [raw(x).clone() for x in (k, v)]
    pairs = [(3, 0), (0 + 7, 39), (7, 7), (5, 12), (2, 2)]
    pa.copy_blocks(k, v, pairs)
    assert pa.get_device_error() == 0
    for x, was in zip((k, v), before):
        for s, d in pairs:
            was[d] = was[s]
        assert torch.equal(raw(x), was)
    pa.copy_blocks(k, v, [(1, 40), (4, 6), (-1, 3)])
    assert pa.get_device_error() == 5
    for x, was in zip((k, v), before):
        was[6] = was[4]
        assert torch.equal(raw(x), was)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_pairs_of_a_batch(kind):
    """Block 0 is the lowest free one, so that a copy goes there while the sequences without a
    copy report (0, 0)."""
    m = Batch(24, 6)
    for n in (16, 5, 21, 32, 9):
        m.add(n)
    for parent in (1, 2, 2):
        m.fork(parent)
    m.truncate([0] + [m.m.tokens[b] for b in m.ids[1:]])     # block 0 has become free
    state = m.upload()
    k, v = pools(kind, 24, 2, 128, 1)
    before = [raw(x).clone() for x in (k, v)]
    new = [0, 3, 1, 2, 0, 4, 2, 5]
    copies = pa.extend_sequences(*state, torch.tensor(new, dtype=torch.int32, device="cuda"),
                                 sum(new))[3]
    pairs = m.extend(new, sum(new))[3].tolist()
    assert copies.tolist() == pairs
    assert sum(s != d for s, d in pairs) == 3 and any(d == 0 and s for s, d in pairs)
    pa.copy_blocks(k, v, copies)
    assert pa.get_device_error() == 0
    for x, was in zip((k, v), before):
        old = was.clone()
        for s, d in pairs:
            if s != d:
                was[d] = old[s]
        assert torch.equal(raw(x), was)


def test_graph():
    k, v = pools("int4", 10, 2, 64)
    pairs = torch.tensor([[0, 0], [1, 4]], dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        pa.copy_blocks(k, v, pairs[:1])
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.copy_blocks(k, v, pairs)
    pairs.copy_(torch.tensor([[2, 0], [3, 9]]))
    want = [raw(x).clone() for x in (k, v)]
    graph.replay()
    torch.cuda.synchronize()
    for x, was in zip((k, v), want):
        was[0], was[9] = was[2].clone(), was[3].clone()
        assert torch.equal(raw(x), was)


def test_refusals():
    k, v = pools("fp8", 4, 2, 64)
    k4, v4 = pools("int4", 4, 2, 64)
    b, _ = pools("bf16", 4, 2, 64)
    with pytest.raises(TypeError):
        pa.copy_blocks(k, b, [(0, 1)])
    with pytest.raises(TypeError):
        pa.copy_blocks(b.half(), b.half(), [(0, 1)])
    with pytest.raises(ValueError):
        pa.copy_blocks(k, k, [(0, 1)])                       # V pages lie by head dim
    with pytest.raises(ValueError):
        pa.copy_blocks(k4, v, [(0, 1)])
    with pytest.raises(ValueError):
        pa.copy_blocks(k4, v4[:3], [(0, 1)])
    with pytest.raises(ValueError):
        pa.copy_blocks(k4.cpu(), v4, [(0, 1)])
    pa.copy_blocks(k4, v4, [])
