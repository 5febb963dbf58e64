"""Accumulated attention weights and eviction on the GPU against the fp64 oracle, over bf16,
FP8 and INT4 pages."""
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
from gpu_util import bits, to_dev  # noqa: E402
from oracle import bounded as BD  # noqa: E402
from oracle import int4 as Q4  # noqa: E402

FORMATS = ["bf16", "fp8", "int4"]


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert pa.get_device_error() == 0, "device error word was set"


class Dev:
    def __init__(self, c):
        for name in ("q", "k", "v", "k_scale", "v_scale", "tables", "lens", "new_key",
                     "new_value", "slots"):
            setattr(self, name, to_dev(getattr(c, name)))
        self.scale = None if c.fmt == "bf16" else self.k_scale


def host(t):
    return bits(t) if t.dtype == torch.bfloat16 else t.cpu().numpy()


def keys_of(c, pool=None):
    return [[c.rows(c.k if pool is None else pool, b, g, int(n), "k") for g in range(c.Hkv)]
            for b, n in enumerate(c.lens)]


def observe(c, d, w0, p0, seen, decay=1.0, **kw):
    """One call, checked against the oracle; returns the device arrays."""
    w, pos = torch.tensor(w0, dtype=torch.float32, device="cuda"), torch.tensor(
        p0, dtype=torch.int32, device="cuda")
    kw.setdefault("max_context_len", max(c.T, int(c.lens.max())))
    got = pa.accumulate_weights(d.q, d.k, d.tables, d.lens, w, pos, to_dev(seen), scale=c.scale,
                                decay=decay, k_scale=d.scale, **kw)
    assert got.data_ptr() == w.data_ptr()
    keys = keys_of(c)
    ref_w, ref_p, gained = BD.accumulate(np.asarray(w0, dtype=np.float32).astype(float), p0,
                                         c.q, keys, c.lens, seen, c.scale,
                                         float(np.float32(decay)))
    x = w.cpu().double().numpy()
    # a weight errs with its scores (fp32 accumulation, 2^-20 of sum |q k|), ex2 and the sums
    # over entries and rows (2^-19 together); decay * old + gained is rounded once more
    rel = 2.0 ** -20 * c.score_size(keys) + 2.0 ** -19
    inside = np.arange(w0.shape[-1]) < c.lens[:, None, None]
    tol = np.where(inside, rel * gained + 2.0 ** -23 * np.abs(ref_w) + 1e-37, 0.0)
    over = np.abs(x - ref_w) - tol
    assert np.isfinite(x).all() and over.max() <= 0, f"exceeds the bound by {over.max():.3e}"
    np.testing.assert_array_equal(pos.cpu().numpy(), ref_p)
    return w, pos


def start(c, E, seed=0):
    rng = np.random.default_rng(seed)
    w0 = rng.exponential(1.0, (len(c.lens), c.Hkv, E)).astype(np.float32)
    return w0, rng.integers(0, 1000, w0.shape).astype(np.int32)


# ------------------------------------------------------------------------------- weights
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,T", [(4, 4, 1), (8, 2, 1), (5, 1, 3), (12, 2, 2), (8, 2, 5),
                                      (4, 1, 16), (1, 1, 33)])
def test_weights_match(fmt, D, Hq, Hkv, T):
    c = Case(D + Hq + T, [T, T + 1, T + 15, T + 16, 100, 257], Hq, Hkv, D, T=T, fmt=fmt)
    w0, p0 = start(c, 260)
    observe(c, Dev(c), w0, p0, c.lens + np.int32(7))


@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
def test_decay_and_long_context(decay):
    """Several chunks per sequence; entries behind a context and after it stay."""
    c = Case(3, [3000, 1, 1024, 1025], 4, 2, 64, fmt="bf16")
    w0, p0 = start(c, 3001)
    observe(c, Dev(c), w0, p0, c.lens, decay=decay)


def test_old_contents_of_new_entries_do_not_matter():
    c = Case(4, [20, 40], 4, 2, 64, T=3, fmt="int4")
    w0, p0 = start(c, 48)
    for b, n in enumerate(c.lens):
        w0[b, :, n - 3:n] = np.nan
    observe(c, Dev(c), w0, p0, c.lens)


def test_out_and_defaults():
    c = Case(5, [20, 40], 4, 2, 64, fmt="fp8")
    d = Dev(c)
    w0, p0 = start(c, 40)
    w, pos = observe(c, d, w0, p0, c.lens)
    src, out = to_dev(w0), torch.full((2, 2, 40), 9.0, device="cuda")
    got = pa.accumulate_weights(d.q.squeeze(1), d.k, d.tables, d.lens, src, scale=c.scale,
                                k_scale=d.k_scale, out=out)
    assert got is out and torch.equal(src.cpu(), torch.tensor(w0))
    assert torch.equal(out[1], w[1]) and torch.equal(out[0, :, :20], w[0, :, :20])
    assert (out[0, :, 20:] == 9).all()
    # seq_lens defaults to context_lens
    p1 = torch.zeros_like(pos)
    pa.accumulate_weights(d.q, d.k, d.tables, d.lens, src, p1, scale=c.scale, k_scale=d.k_scale)
    assert p1[0, 0, 19] == 19 and p1[1, 1, 39] == 39 and p1.count_nonzero() == 4


def test_weights_are_the_same_every_time_and_in_a_graph():
    c = Case(6, [2500, 700, 90], 8, 2, 128, T=2, fmt="int4")
    d = Dev(c)
    w0 = torch.zeros((3, 2, 2500), device="cuda")
    need = pa.accumulate_workspace_size(3, 8, 2, 2, 2500)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")

    def call(out):
        return pa.accumulate_weights(d.q, d.k, d.tables, d.lens, w0, max_context_len=2500,
                                     scale=c.scale, k_scale=d.k_scale, workspace=ws, out=out)
    want = call(torch.zeros_like(w0)).clone()
    assert np.allclose(want.sum(-1).cpu().numpy(), 8, rtol=1e-5)
    out = torch.zeros_like(w0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            again = call(torch.zeros_like(w0))
        side.synchronize()
        assert torch.equal(again, want)


def test_bad_blocks_and_lengths_are_reported():
    c = Case(7, [100, 60, 33], 4, 2, 64, fmt="bf16")
    d = Dev(c)
    w = torch.ones((3, 2, 112), device="cuda")
    d.tables[0, 2] = c.NB
    d.lens[1], d.lens[2] = 200, 0
    pa.accumulate_weights(d.q, d.k, d.tables, d.lens, w, max_context_len=100, scale=c.scale)
    assert pa.get_device_error() == 5
    assert (w[1:] == 1).all() and (w[0, :, 32:48] == 1).all()      # the bad block's entries
    gain = w[0, :, :100].sum(-1) - 99
    assert torch.allclose(gain, torch.full_like(gain, 2.0), atol=1e-3)


@pytest.mark.parametrize("B,hi,T", [(1, 9000, 1), (257, 60, 1), (300, 40, 3), (1030, 33, 1)])
def test_weights_of_many_sequences(B, hi, T):
    """Batches around the chunks of lengths a warp holds and past the size up to which runs are
    balanced, and one sequence over all workers: rows sum to their number."""
    gen = torch.Generator("cuda").manual_seed(B)
    lens = torch.randint(T, hi + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    lens[0], lens[-1] = T, hi
    M = -(-hi // 16)
    tables = torch.randperm(B * M, generator=gen, device="cuda").int().view(B, M)
    k = torch.randn((B * M, 2, 16, 64), generator=gen, device="cuda").bfloat16()
    q = torch.randn((B, T, 6, 64), generator=gen, device="cuda").bfloat16()
    w = torch.full((B, 2, hi), 3.0, device="cuda")
    pa.accumulate_weights(q, k, tables, lens, w, max_context_len=hi, decay=0.0)
    live = torch.arange(hi, device="cuda") < lens[:, None, None]
    assert (w[~live.expand_as(w)] == 3).all()
    gained = torch.where(live, w, torch.zeros_like(w)).double()
    keys = k[tables.long()].transpose(1, 2).flatten(2, 3)[:, :, :hi].double()
    s = torch.einsum("bthgd,bhjd->bhtgj", q.double().view(B, T, 2, 3, 64), keys) / 8
    last = lens[:, None] - T + torch.arange(T, device="cuda")
    see = torch.arange(hi, device="cuda") <= last[..., None]
    ref = torch.softmax(s.masked_fill(~see[:, None, :, None], -float("inf")), -1).sum((2, 3))
    # scores err by 2^-20 of sum |q k| (at most 40 here, in units of log2), sums by 2^-19
    assert ((gained - ref).abs() <= (40 * 2.0 ** -20 + 2.0 ** -19) * ref + 1e-37).all()


# ------------------------------------------------------------------------------- eviction
def evict(c, d, w0, p0, budget, recent, mcl=None):
    """One call, checked entry by entry and page by page against the oracle."""
    w, pos = to_dev(w0), to_dev(p0)
    new = pa.evict_tokens(d.k, d.v, d.tables, d.lens, w, pos, budget, recent,
                          max(1, int(c.lens.max())) if mcl is None else mcl)
    assert new.cpu().tolist() == [min(int(n), budget) for n in c.lens]
    ref_w, ref_p = w0.copy(), p0.copy()
    rk, rv = c.k.copy(), c.v.copy()
    D = c.D
    if c.fmt == "int4":
        parts = [[np.array(x, copy=True) for x in Q4.unpack(p, D)] for p in (rk, rv)]
    for b, n in enumerate(c.lens):
        for g in range(c.Hkv):
            for a, z in BD.select(w0[b, g, :n], p0[b, g, :n], budget, recent):
                ref_w[b, g, z], ref_p[b, g, z] = w0[b, g, a], p0[b, g, a]
                src, dst = (c.tables[b, a // 16], a % 16), (c.tables[b, z // 16], z % 16)
                if c.fmt == "int4":
                    for pair in parts:
                        for x in pair:
                            x[dst[0], g, dst[1]] = x[src[0], g, src[1]]
                else:
                    rk[dst[0], g, dst[1]] = rk[src[0], g, src[1]]
                    if c.fmt == "fp8":
                        rv[dst[0], g, :, dst[1]] = rv[src[0], g, :, src[1]]
                    else:
                        rv[dst[0], g, dst[1]] = rv[src[0], g, src[1]]
    if c.fmt == "int4":
        rk, rv = (Q4.pack(*pair) for pair in parts)
    np.testing.assert_array_equal(host(pos), ref_p)
    np.testing.assert_array_equal(w.cpu().numpy(), ref_w)
    np.testing.assert_array_equal(host(d.k), rk)
    np.testing.assert_array_equal(host(d.v), rv)
    return new, w, pos


def stats(rng, lens, Hkv, E, kind):
    B = len(lens)
    if kind == "ties":
        w = rng.integers(0, 3, (B, Hkv, E)).astype(np.float32)
        w[rng.random(w.shape) < 0.2] = -0.0
    elif kind == "special":
        w = rng.standard_normal((B, Hkv, E)).astype(np.float32)
        for x in (np.nan, -np.nan, np.inf, -np.inf, 1e-42, -1e-42):
            w[rng.random(w.shape) < 0.06] = x
    elif kind == "equal":
        w = np.full((B, Hkv, E), 0.25, dtype=np.float32)
    else:
        w = np.exp(2 * rng.standard_normal((B, Hkv, E))).astype(np.float32)
    pos = np.stack([np.stack([rng.permutation(E + 50)[:E] for _ in range(Hkv)])
                    for _ in range(B)]).astype(np.int32)
    return w, pos


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (17, 5), (64, 64), (100, 30), (256, 0)])
def test_evict_matches(fmt, D, budget, recent):
    c = Case(budget + D, [0, 1, 16, 63, 100, 101, 257], 6, 3, D, T=0, fmt=fmt)
    rng = np.random.default_rng(budget + recent)
    for kind in ("spread", "ties"):
        w0, p0 = stats(rng, c.lens, 3, 260, kind)
        evict(c, Dev(c), w0, p0, budget, recent)


@pytest.mark.parametrize("kind", ["spread", "ties", "special", "equal"])
@pytest.mark.parametrize("budget,recent", [(700, 100), (1500, 0), (2999, 2999)])
def test_evict_long(kind, budget, recent):
    """Several scans per row; ties that straddle them; one entry too many."""
    c = Case(8, [3000, 701, 1501], 2, 2, 64, T=0, fmt="int4")
    w0, p0 = stats(np.random.default_rng(budget), c.lens, 2, 3008, kind)
    evict(c, Dev(c), w0, p0, budget, recent)


@pytest.mark.parametrize("kind", ["ties", "special"])
@pytest.mark.parametrize("top", [4096, 4097, 8192, 8193, 16384, 16385, 20000])
def test_evict_around_the_sizes_of_the_kernels(kind, top):
    """Rows up to and past what 8, 16 and 32 warps hold in registers, and from shared memory, with
    shorter rows beside them; a row one entry too long."""
    budget = top - 600
    c = Case(top, [top, budget + 1, budget + 300, 33], 1, 1, 64, T=0, fmt="int4")
    w0, p0 = stats(np.random.default_rng(top), c.lens, 1, top + 16, kind)
    evict(c, Dev(c), w0, p0, budget, 250)
    c = Case(top + 1, [top, 700], 1, 1, 64, T=0, fmt="int4")
    evict(c, Dev(c), w0[:2], p0[:2], 512, 100)


def test_evict_context_past_shared_memory():
    """A row whose keys do not fit in shared memory: read again at every pass."""
    n, budget = 60000, 20000
    gen = torch.Generator("cuda").manual_seed(0)
    k = torch.randn((n // 16, 1, 16, 64), generator=gen, device="cuda").bfloat16()
    v = torch.randn((n // 16, 1, 16, 64), generator=gen, device="cuda").bfloat16()
    tables = torch.randperm(n // 16, generator=gen, device="cuda").int()[None]
    w = torch.randint(0, 5000, (1, 1, n), generator=gen, device="cuda").float()
    pos = torch.randperm(n, generator=gen, device="cuda").int().view(1, 1, n)
    w0, p0 = w.clone(), pos.clone()
    old = k[tables[0].long()][:, 0].flatten(0, 1).clone()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    new = pa.evict_tokens(k, v, tables, lens, w, pos, budget, 1000, n)
    assert new.item() == budget
    ref = BD.select(w0[0, 0].cpu().numpy(), p0[0, 0].cpu().numpy(), budget, 1000)
    at = torch.arange(n, device="cuda")
    src, dst = (torch.tensor(x, device="cuda") for x in zip(*ref))
    at[dst] = src
    assert torch.equal(pos[0, 0, :budget], p0[0, 0][at[:budget]])
    assert torch.equal(w[0, 0, :budget], w0[0, 0][at[:budget]])
    got = k[tables[0].long()][:, 0].flatten(0, 1)
    assert torch.equal(got[:budget], old[at[:budget]])
    assert torch.equal(got[budget:], old[budget:])


@pytest.mark.parametrize("kind", ["spread", "ties", "special", "equal"])
@pytest.mark.parametrize("budget,recent", [(1, 1), (5, 0), (500, 100), (500, 497), (500, 500),
                                           (5000, 37)])
def test_evict_few(kind, budget, recent):
    """A few entries too many, around the number up to which they are found one by one; protected
    entries that leave fewer others than must go."""
    c = Case(11, [budget + d for d in (1, 2, 3, 7, 8, 9, 20)], 2, 2, 64, T=0, fmt="int4")
    w0, p0 = stats(np.random.default_rng(budget + recent), c.lens, 2, budget + 32, kind)
    evict(c, Dev(c), w0, p0, budget, recent)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("budget,recent,over", [(1, 0, 8), (3, 3, 8), (90, 20, 8), (90, 20, 9),
                                                (4090, 500, 6), (4090, 500, 7)])
def test_evict_with_a_close_bound(fmt, D, budget, recent, over):
    """max_context_len leaves at most 8 entries to drop (one launch), or just more."""
    c = Case(12 + over, [budget + over, budget + over - 1, budget + 1, budget, 0], 4, 2, D, T=0,
             fmt=fmt)
    w0, p0 = stats(np.random.default_rng(over), c.lens, 2, budget + 16, "ties")
    evict(c, Dev(c), w0, p0, budget, recent)


def test_evict_few_past_shared_memory():
    n, budget = 60000, 59995
    gen = torch.Generator("cuda").manual_seed(1)
    k = torch.randn((n // 16, 1, 16, 64), generator=gen, device="cuda").bfloat16()
    tables = torch.randperm(n // 16, generator=gen, device="cuda").int()[None]
    w = torch.randint(0, 2000, (1, 1, n), generator=gen, device="cuda").float()
    pos = torch.randperm(n, generator=gen, device="cuda").int().view(1, 1, n)
    ref = BD.select(w[0, 0].cpu().numpy(), pos[0, 0].cpu().numpy(), budget, 1000)
    at = torch.arange(n, device="cuda")
    for a, z in ref:
        at[z] = a
    w0, p0, old = w.clone(), pos.clone(), k[tables[0].long()][:, 0].flatten(0, 1).clone()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    assert pa.evict_tokens(k, k.clone(), tables, lens, w, pos, budget, 1000, n).item() == budget
    assert torch.equal(pos[0, 0, :budget], p0[0, 0][at[:budget]])
    assert torch.equal(w[0, 0, :budget], w0[0, 0][at[:budget]])
    assert torch.equal(k[tables[0].long()][:, 0].flatten(0, 1)[:budget], old[at[:budget]])


def test_evict_in_order_keeps_the_tail():
    """Equal weights and positions in order: the newest and the lowest indices stay."""
    c = Case(9, [50], 1, 1, 64, T=0, fmt="bf16")
    w0 = np.ones((1, 1, 64), dtype=np.float32)
    p0 = np.arange(64, dtype=np.int32)[None, None]
    _, _, pos = evict(c, Dev(c), w0, p0, 20, 8)
    assert sorted(pos[0, 0, :20].tolist()) == list(range(12)) + list(range(42, 50))


def test_nothing_to_evict_and_empty_batch():
    c = Case(10, [5, 20], 2, 2, 64, T=0, fmt="fp8")
    w0, p0 = stats(np.random.default_rng(0), c.lens, 2, 32, "spread")
    d = Dev(c)
    evict(c, d, w0, p0, 20, 3)
    evict(c, d, w0, p0, 1000, 3)                  # a budget above every length and the pool
    z = pa.evict_tokens(d.k, d.v, d.tables[:0], d.lens[:0], to_dev(w0[:0]), to_dev(p0[:0]), 4, 1, 20)
    assert z.shape == (0,)


def test_evict_reports_bad_tables_and_lengths():
    c = Case(11, [100, 60, 80], 2, 2, 64, T=0, fmt="bf16")
    w0, p0 = stats(np.random.default_rng(1), c.lens, 2, 112, "spread")
    d = Dev(c)
    d.tables[0, 5] = -1
    d.lens[1] = 101
    w, pos = to_dev(w0), to_dev(p0)
    new = pa.evict_tokens(d.k, d.v, d.tables, d.lens, w, pos, 30, 4, 100)
    assert pa.get_device_error() == 5
    assert new.tolist() == [100, 101, 30]
    np.testing.assert_array_equal(w[:2].cpu().numpy(), w0[:2])
    changed = (host(d.k) != c.k).any((1, 2, 3)).nonzero()[0]
    assert len(changed) and set(changed) <= set(c.tables[2].tolist())


def test_evict_in_a_graph_and_on_a_stream():
    c = Case(12, [300, 40], 2, 2, 128, T=0, fmt="int4")
    w0, p0 = stats(np.random.default_rng(2), c.lens, 2, 304, "spread")
    a, z = Dev(c), Dev(c)
    want, w1, pos1 = evict(c, a, w0, p0, 64, 16)
    w, pos = to_dev(w0), to_dev(p0)
    ws = torch.empty(pa.evict_workspace_size(2, 2, 300, 64), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        new = pa.evict_tokens(z.k, z.v, z.tables, z.lens, w, pos, 64, 16, 300, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(new, want) and torch.equal(w, w1) and torch.equal(pos, pos1)
    assert torch.equal(z.k, a.k) and torch.equal(z.v, a.v)
    y, side = Dev(c), torch.cuda.Stream()
    w, pos = to_dev(w0), to_dev(p0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        pa.evict_tokens(y.k, y.v, y.tables, y.lens, w, pos, 64, 16, 300)
    side.synchronize()
    assert torch.equal(y.k, a.k) and torch.equal(pos, pos1)


# ------------------------------------------------------------------------------- together
@pytest.mark.parametrize("fmt", FORMATS)
def test_bounded_decoding_loop(fmt):
    """The loop of a bounded cache: append, attend, add the weights up, evict; the block manager
    gives the dropped blocks back.  Each step is checked against the oracle on the cache that
    the step met."""
    budget, recent, D, Hq, Hkv = 40, 10, 64, 4, 2
    c = Case(13, [30, 55], Hq, Hkv, D, fmt=fmt, extra_blocks=4)
    bm = pa.BlockManager(c.NB)
    for b, n in enumerate(c.lens):
        bm.add_sequence(b, int(n))
    tables, lens = bm.block_table([0, 1], c.mbs)
    # the manager's blocks: move the case's pages there
    k, v = np.zeros_like(c.k), np.zeros_like(c.v)
    for b, n in enumerate(c.lens):
        for i in range(-(-int(n) // 16)):
            k[tables[b, i]], v[tables[b, i]] = c.k[c.tables[b, i]], c.v[c.tables[b, i]]
    c.k, c.v, c.tables = k, v, tables.numpy()
    d = Dev(c)
    E = c.mbs * 16
    w = np.zeros((2, Hkv, E), dtype=np.float32)
    pos = np.broadcast_to(np.arange(E, dtype=np.int32), w.shape).copy()
    seen = c.lens.copy()
    gen = torch.Generator("cuda").manual_seed(0)
    for step in range(6):
        if step:
            for b in range(2):
                bm.append_slot(b)
            tables, lens = bm.block_table([0, 1], c.mbs)
            seen = seen + 1
            d.tables, d.lens = tables.clamp(min=0).cuda(), lens.cuda()
            new = torch.randn((2, 2, Hkv, D), generator=gen, device="cuda").bfloat16()
            d.q = torch.randn((2, 1, Hq, D), generator=gen, device="cuda").bfloat16()
            kw = dict(max_context_len=int(lens.max()), new_key=new[0], new_value=new[1])
            if fmt == "int4":
                out = pa.attention_int4(d.q, d.k, d.v, d.k_scale, d.v_scale, d.tables, d.lens, **kw)
            else:
                sc = {} if fmt == "bf16" else {"k_scale": d.k_scale, "v_scale": d.v_scale}
                out = pa.attention(d.q, d.k, d.v, d.tables, d.lens, **kw, **sc)
            c.q, c.k, c.v = bits(d.q), host(d.k), host(d.v)
            c.tables, c.lens = tables.numpy().clip(0), lens.numpy()
            for b in range(2):
                for h in range(Hq):
                    n, g = int(c.lens[b]), h * Hkv // Hq
                    s = c.rows(c.k, b, g, n, "k") @ (
                        d.q[b, 0, h].double().cpu().numpy()) * c.scale
                    p = np.exp(s - s.max())
                    ref = p / p.sum() @ c.rows(c.v, b, g, n, "v")
                    err = np.abs(out[b, 0, h].double().cpu().numpy() - ref)
                    assert (err <= 1e-2 + 2.0 ** -8 * np.abs(ref)).all()
        wd, pd = observe(c, d, w, pos, seen, decay=0.9)
        w, pos = wd.cpu().numpy(), pd.cpu().numpy()
        new, wd, pd = evict(c, d, w, pos, budget, recent)
        w, pos = wd.cpu().numpy(), pd.cpu().numpy()
        for b in range(2):
            bm.truncate(b, min(int(c.lens[b]), budget))
        assert new.tolist() == [bm.num_tokens(0), bm.num_tokens(1)]
        c.k, c.v = host(d.k), host(d.v)
    assert bm.num_free_blocks() == c.NB - 2 * 3
