"""Ways of use that the documentation names for bounded caches and INT4 pages: the sums of a whole
prompt, the sums of accepted drafts alone, and copy-on-write of INT4 blocks."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():          # collected on CPU-only hosts, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import __graft_entry__  # noqa: E402

__graft_entry__.build()

import paged_kv_cache_221_gb300 as pa  # noqa: E402
from bounded_cases import Case  # noqa: E402
from gpu_util import to_dev  # noqa: E402
from oracle import bounded as BD  # noqa: E402


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert pa.get_device_error() == 0, "device error word was set"


def close(got, ref, gained, c, keys, calls):
    """Scores err by 2^-20 of sum |q k|, ex2 and a call's sums by 2^-19, each call's result is
    rounded to fp32."""
    rel = 2.0 ** -20 * c.score_size(keys) + 2.0 ** -19
    tol = rel * gained + calls * 2.0 ** -23 * np.abs(ref) + 1e-37
    assert (np.abs(got.cpu().double().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("n", [5, 64, 131])
def test_sums_of_a_prompt_in_chunks(fmt, n):
    """Successive calls with up to 64 query rows per kv head, context_lens at each chunk's end."""
    Hq, Hkv, D, T = 6, 2, 64, 21
    c = Case(61, [n], Hq, Hkv, D, T=n, fmt=fmt)
    k, tables = to_dev(c.k), to_dev(c.tables)
    scale = None if fmt == "bf16" else to_dev(c.k_scale)
    q = to_dev(c.q)
    w = torch.full((1, Hkv, n + 4), 7.0, device="cuda")
    pos = torch.full((1, Hkv, n + 4), -1, dtype=torch.int32, device="cuda")
    ends = list(range(T, n, T)) + [n]
    at = 0
    for e in ends:
        end = torch.tensor([e], dtype=torch.int32, device="cuda")
        pa.accumulate_weights(q[:, at:e].contiguous(), k, tables, end, w, pos, max_context_len=e,
                              scale=c.scale, k_scale=scale)
        at = e
    keys = [[c.rows(c.k, 0, g, n, "k") for g in range(Hkv)]]
    ref, _, gained = BD.accumulate(np.zeros((1, Hkv, n)), np.zeros((1, Hkv, n), int), c.q, keys,
                                   c.lens, c.lens, c.scale, 1.0)
    close(w[:, :, :n], ref, gained, c, keys, len(ends))
    assert (w[:, :, n:] == 7).all() and (pos[:, :, n:] == -1).all()
    assert (pos[:, :, :n].cpu() == torch.arange(n)).all()


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_sums_of_accepted_drafts(fmt):
    """Sequences that kept the same number of tokens go together, with their lengths after it."""
    T, Hq, Hkv, D = 4, 4, 2, 64
    kept = np.array([1, 3, 4, 1, 3, 2], dtype=np.int32)
    c = Case(62, [40, 90, 4, 300, 33, 17], Hq, Hkv, D, T=T, fmt=fmt)
    rng = np.random.default_rng(0)
    w0 = rng.exponential(1.0, (6, Hkv, 304)).astype(np.float32)
    p0 = np.tile(np.arange(304, dtype=np.int32), (6, Hkv, 1))
    seen = c.lens + np.int32(11)                      # tokens seen, the drafts among them
    w, pos = to_dev(w0), to_dev(p0)
    k, q, tables = to_dev(c.k), to_dev(c.q), to_dev(c.tables)
    lens, seen_d = to_dev(c.lens), to_dev(seen)
    for n in range(1, T + 1):
        rows = torch.tensor(np.flatnonzero(kept == n), device="cuda")
        if len(rows) == 0:
            continue
        wn, pn = w[rows], pos[rows]
        pa.accumulate_weights(q[rows, :n].contiguous(), k, tables[rows], lens[rows] - (T - n), wn,
                              pn, seen_d[rows] - (T - n), max_context_len=300, scale=c.scale,
                              decay=0.5, k_scale=None if fmt == "bf16" else to_dev(c.k_scale))
        w[rows], pos[rows] = wn, pn
    keys = [[c.rows(c.k, b, g, int(n), "k") for g in range(Hkv)] for b, n in enumerate(c.lens)]
    for b in range(6):
        n, L = int(kept[b]), int(c.lens[b] - T + kept[b])
        ref, rp, gained = BD.accumulate(w0[b:b + 1].astype(float), p0[b:b + 1], c.q[b:b + 1, :n],
                                        [[x[:L] for x in keys[b]]], [L], [seen[b] - T + n],
                                        c.scale, 0.5)
        close(w[b:b + 1], ref, gained, c, keys, 1)
        np.testing.assert_array_equal(pos[b:b + 1].cpu().numpy(), rp)


def test_copy_on_write_of_int4_blocks():
    """A forked sequence's partly filled block is copied by indexing the pools."""
    Hkv, D = 2, 64
    bm = pa.BlockManager(8)
    bm.add_sequence(0, 20)
    bm.fork(0, 1)
    gen = torch.Generator("cuda").manual_seed(0)
    k, v = (torch.randint(0, 120, (8, Hkv, pa.int4_page_bytes(D)), generator=gen, device="cuda",
                          dtype=torch.uint8) for _ in range(2))
    slot, (src, dst) = bm.append_slot(1)
    before = k.clone()
    for pool in (k, v):
        pool[dst] = pool[src]
    new = torch.randn((2, 1, Hkv, D), generator=gen, device="cuda").bfloat16()
    one = torch.ones(Hkv, device="cuda")
    pa.reshape_and_cache_int4(new[0], new[1], k, v, torch.tensor([slot], device="cuda"), one, one)
    tables, lens = bm.block_table([0, 1], 2)
    assert lens.tolist() == [20, 21] and tables[0, 0] == tables[1, 0] and tables[1, 1] == dst
    assert torch.equal(k[src], before[src])
    at = [torch.arange(20) for _ in range(2)]
    slots = [(tables[b][at[b] // 16] * 16 + at[b] % 16).long().cuda() for b in range(2)]
    a, b = (pa.gather_cache_int4(k, v, s, one, one) for s in slots)
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16))
    assert torch.equal(a[1].view(torch.int16), b[1].view(torch.int16))
