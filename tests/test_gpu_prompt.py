"""Attention of packed prompts over the paged cache, against 64 bits."""
import pytest
import torch

import paged_kv_cache_221_gb300 as pa
from prompt_cases import Prompts, check

pytestmark = pytest.mark.gpu


def attend(c, **kw):
    return pa.prompt_attention(c.q, c.k, c.v, c.tables, c.ctx, c.starts, kw.pop("most", c.most),
                               k_scale=c.k_scale, v_scale=c.v_scale, **kw)


def run(c, scale=None, window=0, **kw):
    got = attend(c, scale=scale, window_size=window, **kw)
    assert pa.get_device_error() == 0
    check(got, *c.exact(scale, window), rows=slice(0, sum(c.new)))
    return got


@pytest.mark.parametrize("D", [64, 128])
def test_one_short_prompt(D):
    run(Prompts(1, [16], [0], 4, 4, D))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (32, 8), (8, 1), (6, 2), (5, 1), (21, 3), (64, 1),
                                   (71, 1), (128, 1)])
def test_head_layouts(heads, D):
    run(Prompts(2, [77, 1, 200], [0, 33, 140], *heads, D))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256,
                               257, 511, 513, 1000])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2)])
def test_lengths(n, heads):
    run(Prompts(n, [n], [0], *heads, 128))


@pytest.mark.parametrize("cached", [1, 15, 16, 17, 96, 127, 128, 129, 1000])
@pytest.mark.parametrize("n", [1, 5, 64, 130])
def test_behind_a_cached_prefix(n, cached):
    run(Prompts(n + cached, [n], [cached], 8, 2, 128))


def test_many_sequences_and_empty_ones():
    new = [(37 * i) % 90 if i % 7 else 0 for i in range(150)]
    cached = [(61 * i) % 300 if i % 5 else 0 for i in range(150)]
    run(Prompts(3, new, cached, 4, 2, 64, behind=11))
    run(Prompts(4, [0, 0, 0, 9], [0, 5, 0, 0], 4, 2, 64))


@pytest.mark.parametrize("B", [1, 31, 32, 33, 34, 1023, 1025, 1100])
def test_sequence_counts(B):
    run(Prompts(B, [1 + i % 3 for i in range(B)], [i % 40 for i in range(B)], 2, 1, 64))


@pytest.mark.parametrize("window", [1, 2, 16, 100, 127, 128, 129, 300, 5000, 2 ** 31 - 1])
@pytest.mark.parametrize("heads", [(4, 4), (16, 2)])
def test_windows(window, heads):
    c = Prompts(5, [300, 1, 130], [0, 400, 77], *heads, 128)
    run(c, window=window)
    run(c, window=window, partition_size=128)


@pytest.mark.parametrize("size", [128, 256, 384, 1024, 0])
@pytest.mark.parametrize("D", [64, 128])
def test_partitions(size, D):
    run(Prompts(6, [33, 1, 300], [1500, 700, 0], 8, 2, D), partition_size=size)


def test_partitions_of_many_heads_and_rows():
    run(Prompts(7, [70, 3], [900, 5000], 64, 2, 128), partition_size=512)
    run(Prompts(8, [2], [20000], 32, 8, 128))


def test_long_prompt():
    run(Prompts(9, [3001, 2500], [0, 1111], 8, 2, 128))


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 3.0])
def test_scales(scale):
    run(Prompts(10, [150, 40], [0, 300], 4, 2, 128), scale=scale)


# ------------------------------------------------------------------------------- FP8 pages
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(4, 4), (32, 8), (5, 1), (128, 1)])
def test_fp8_head_layouts(heads, D):
    run(Prompts(20, [77, 1, 200], [0, 33, 140], *heads, D, fp8=True))


@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 65, 127, 128, 129, 257, 1000])
@pytest.mark.parametrize("D", [64, 128])
def test_fp8_lengths(n, D):
    run(Prompts(n, [n, 3], [0, n], 8, 2, D, fp8=True))


@pytest.mark.parametrize("window", [1, 16, 100, 128, 300])
def test_fp8_windows_and_partitions(window):
    c = Prompts(21, [300, 1, 130], [0, 400, 77], 8, 2, 128, fp8=True)
    run(c, window=window)
    run(c, window=window, partition_size=128)
    run(c, partition_size=256)


def test_fp8_many_sequences_and_long_ones():
    new = [(37 * i) % 90 if i % 7 else 0 for i in range(150)]
    cached = [(61 * i) % 300 if i % 5 else 0 for i in range(150)]
    run(Prompts(22, new, cached, 4, 2, 64, fp8=True, behind=11))
    run(Prompts(23, [3001, 40], [0, 5000], 8, 2, 128, fp8=True))


def test_fp8_query_rows_of_any_size():
    """Rows whose elements lie far outside f16 keep their directions: a factor on q is one on the
    scale."""
    c = Prompts(24, [150, 20], [0, 200], 8, 2, 128, fp8=True)
    for e in (-110, -60, -20, 20, 60, 110):
        d = Prompts(24, [150, 20], [0, 200], 8, 2, 128, fp8=True)
        d.q = c.q * 2.0 ** e
        assert torch.equal(attend(d, scale=128 ** -0.5 * 2.0 ** -e), attend(c))
    d.q = c.q.clone()
    d.q[::3] *= 2.0 ** 40                                 # of one tile, rows far apart
    d.q[1::3] = 0
    run(d, scale=128 ** -0.5 * 2.0 ** -40)


# ------------------------------------------------------------------------------- special values
def put(c, b, j, head, d, value, pool="v"):
    """One element of entry j of sequence b."""
    x = getattr(c, pool)
    blk = int(c.tables[b, j // 16])
    if c.fp8:
        value = {float("inf"): 0x7F, float("-inf"): 0x7F}.get(value, 0x7F)
        if pool == "v":
            x[blk, head, d, j % 16] = value
        else:
            x[blk, head, j % 16, d] = value
    else:
        x[blk, head, j % 16, d] = value


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_reach_the_rows_that_see_them(fp8, heads, value):
    """A NaN or infinity in V reaches every query token at or behind its position, in its head
    dim, and no other; the same with windows and cut keys."""
    for window, part in ((0, 0), (0, 128), (40, 0), (40, 128), (200, 0)):
        c = Prompts(30, [300, 90], [20, 500], *heads, 128, fp8=fp8)
        for j in (0, 19, 20, 100, 255, 256, 319):
            put(c, 0, j, j % heads[1], (j * 7) % 128, value)
        for j in (3, 499, 500, 589):
            put(c, 1, j, 1, j % 128, value)
        run(c, window=window, partition_size=part)


def test_opposite_infinities():
    c = Prompts(31, [200], [0], 4, 4, 128)
    put(c, 0, 50, 1, 5, float("inf"))
    put(c, 0, 120, 1, 5, float("-inf"))
    run(c)


@pytest.mark.parametrize("fp8", [False, True])
def test_keys_of_nan_and_infinite_scores(fp8):
    """A NaN score, or one of +inf, makes the rows that see it NaN and no others; a key of -inf
    scores has no weight."""
    nan = float("nan")
    c = Prompts(32, [200, 40], [10, 0], 4, 4, 128, fp8=fp8)
    for j in (60, 130):
        put(c, 0, j, 2, 9, nan, "k")
    got = attend(c)
    assert pa.get_device_error() == 0
    pos = torch.arange(10, 210, device="cuda")
    want = torch.zeros((240, 4), dtype=torch.bool, device="cuda")
    want[:200, 2] = pos >= 60
    assert torch.equal(torch.isnan(got).any(-1), want) and torch.equal(torch.isnan(got).all(-1), want)
    if fp8:
        return
    c = Prompts(33, [200], [0], 4, 4, 128)
    c.q = c.q.abs() + 0.01
    put(c, 0, 70, 1, 9, float("-inf"), "k")
    run(c)
    put(c, 0, 0, 1, 9, float("-inf"), "k")
    got = attend(c)                                       # token 0 of that head sees nothing else
    assert torch.isnan(got[0, 1]).all() and torch.isfinite(got[1:]).all()
    put(c, 0, 70, 1, 9, float("inf"), "k")
    got = attend(c)
    assert torch.isfinite(got[1:70]).all() and torch.isnan(got[70:, 1]).all()
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("power", [10, 20, 30, 60, 100])
def test_large_scores(fp8, power):
    """Past 2^26 a score has no bits behind the point; the row is its largest score's value."""
    c = Prompts(34, [300], [100], 4, 2, 128, fp8=fp8)
    got = attend(c, scale=2.0 ** power)
    assert pa.get_device_error() == 0
    k, v = (x.repeat_interleave(2, 0) for x in c.kv(0))
    s = c.q.double().transpose(0, 1) @ k.transpose(1, 2)
    s = s.masked_fill(torch.arange(400, device="cuda") > torch.arange(100, 400, device="cuda")[:, None],
                      -float("inf"))
    two = s.topk(2, -1)
    # rows whose two best scores differ by what fp32's products can tell apart, and by 20 or more
    # when scaled: all other weights then come to less than 400 e^-20
    clear = (two.values[..., 0] - two.values[..., 1] > max(1e-3, 20 * 2.0 ** -power)).transpose(0, 1)
    want = torch.gather(v, 1, two.indices[..., :1].expand(-1, -1, 128)).transpose(0, 1)
    assert torch.isfinite(got).all()
    # the one weight and the output are rounded, 2^-8 each (that weight is 1 only where the
    # reference is that row's maximum, and it may lie up to 8 below)
    assert ((got.double() - want).abs()[clear] <= 2.0 ** -7 * want.abs()[clear] + 1e-5).all()
    assert clear.double().mean() > 0.9


# ------------------------------------------------------------------------------- calls
def test_rows_of_no_sequence_are_left():
    c = Prompts(40, [40, 0, 70], [0, 10, 5], 4, 2, 64, behind=30)
    out = torch.full_like(c.q, 7.0)
    got = attend(c, out=out)
    assert got is out and (out[110:] == 7.0).all() and not (out[:110] == 7.0).all()
    d = Prompts(40, [40, 70], [0, 5], 4, 2, 64, behind=9)
    d.q = torch.cat([d.q[110:], d.q[:110]])               # the first rows belong to nobody
    d.starts += 9
    out = torch.full_like(d.q, 7.0)
    attend(d, out=out)
    assert (out[:9] == 7.0).all()
    e = Prompts(40, [40, 70], [0, 5], 4, 2, 64)
    assert torch.equal(out[9:], attend(e))
    assert pa.get_device_error() == 0


def test_sequences_out_of_bounds_are_skipped():
    BOUNDS = 5
    c = Prompts(41, [40, 50, 60], [10, 20, 30], 4, 2, 64)
    want = attend(c)
    for bad in (49, -3, 91, 2 ** 31 - 1):                 # sequence 1 holds 70
        ctx = c.ctx.clone()
        ctx[1] = bad
        out = torch.full_like(c.q, 7.0)
        pa.prompt_attention(c.q, c.k, c.v, c.tables, ctx, c.starts, 90, out=out)
        assert pa.get_device_error() == BOUNDS, bad
        assert torch.equal(out[:40], want[:40]) and torch.equal(out[90:], want[90:])
        assert (out[40:90] == 7.0).all()
    for starts in ([0, 40, 151, 150], [0, 40, 30, 150], [-1, 40, 90, 150], [0, 40, 90, 2 ** 31 - 1]):
        s = torch.tensor(starts, dtype=torch.int32, device="cuda")
        pa.prompt_attention(c.q, c.k, c.v, c.tables, c.ctx, s, 90)
        assert pa.get_device_error() == BOUNDS, starts
    c = Prompts(41, [1000, 20, 30], [0, 0, 2000], 4, 2, 64)
    s = torch.tensor([0, 1000, 50, 1050], dtype=torch.int32, device="cuda")
    pa.prompt_attention(c.q, c.k, c.v, c.tables, c.ctx, s, c.most)
    assert pa.get_device_error() == BOUNDS
    for fp8 in (False, True):
        c = Prompts(42, [40, 50, 60], [10, 20, 30], 4, 2, 64, fp8=fp8)
        want = attend(c)
        for bad in (c.NB, -1, 2 ** 31 - 1, -2 ** 31):
            t = c.tables.clone()
            t[1, 2] = bad
            got = pa.prompt_attention(c.q, c.k, c.v, t, c.ctx, c.starts, c.most,
                                      k_scale=c.k_scale, v_scale=c.v_scale)
            assert pa.get_device_error() == BOUNDS, bad
            assert torch.equal(got[:40], want[:40]) and torch.equal(got[90:], want[90:])


def test_bound_workspace_and_streams():
    c = Prompts(43, [33, 9], [2000, 100], 8, 2, 128)
    want = run(c)
    check(attend(c, most=c.mbs * 16), *c.exact())
    assert torch.equal(attend(c), want)
    size = pa.prompt_workspace_size(c.N, 2, 8, 2, c.most, 128, 256)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    a = attend(c, partition_size=256, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = attend(c, partition_size=256)
    s.synchronize()
    assert torch.equal(a, b)
    with pytest.raises(pa.PagedAttnError):
        attend(c, partition_size=256, workspace=ws[:size - 256])
    with pytest.raises(pa.PagedAttnError):
        attend(c, partition_size=100)


def test_graphs_that_share_a_workspace():
    """Two captured calls on one workspace, replayed in turn with new inputs and lengths."""
    c = Prompts(44, [70, 20], [900, 400], 8, 2, 128)
    d = Prompts(45, [30, 50], [100, 1500], 8, 2, 128)
    ws = torch.empty(max(pa.prompt_workspace_size(x.N, 2, 8, 2, x.most, 128, 256) for x in (c, d)),
                     dtype=torch.uint8, device="cuda")
    want = [attend(x, partition_size=256) for x in (c, d)]
    graphs = []
    for x in (c, d):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = attend(x, partition_size=256, workspace=ws)
        graphs.append((g, out))
    for _ in range(3):
        for g, _out in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (_g, out), w in zip(graphs, want):
        assert torch.equal(out, w)
    c.ctx -= 300                                          # the same graph, shorter contexts
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], attend(c, partition_size=256))
    assert pa.get_device_error() == 0


def test_the_same_call_twice_and_two_at_once():
    c = Prompts(46, [600, 300, 40], [0, 77, 900], 8, 2, 128)
    want = attend(c)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams * 3:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(attend(c))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert pa.get_device_error() == 0


def test_empty_calls():
    c = Prompts(47, [5], [0], 4, 2, 64)
    out = pa.prompt_attention(c.q[:0], c.k, c.v, c.tables, c.ctx, c.starts, c.most)
    assert out.shape == (0, 4, 64)
    out = pa.prompt_attention(c.q, c.k, c.v, c.tables[:0], c.ctx[:0], c.starts[:1], c.most,
                              out=torch.full_like(c.q, 3.0))
    assert (out == 3.0).all()
    zero = torch.zeros_like(c.starts)
    out = pa.prompt_attention(c.q, c.k, c.v, c.tables, torch.zeros_like(c.ctx), zero, c.most,
                              out=torch.full_like(c.q, 3.0))
    assert (out == 3.0).all() and pa.get_device_error() == 0


def test_equals_single_token_attention():
    """One query token per sequence is a decode step."""
    c = Prompts(48, [1] * 20, [17 * i for i in range(20)], 8, 2, 128)
    got = attend(c)
    dec = pa.attention(c.q[:, None], c.k, c.v, c.tables, c.ctx, c.most)[:, 0]
    out, size = c.exact()
    check(got, out, size)
    check(dec, out, size)


def test_refusals():
    c = Prompts(49, [20, 10], [0, 5], 4, 2, 64)

    def call(**kw):
        a = dict(q=c.q, k=c.k, v=c.v, t=c.tables, n=c.ctx, s=c.starts, most=c.most)
        rest = {k: kw.pop(k) for k in list(kw) if k not in a}
        a.update(kw)
        return pa.prompt_attention(*a.values(), **rest)

    for kw in (dict(q=c.q.float()), dict(s=c.starts.long()), dict(n=c.ctx.long()),
               dict(k=c.k.half()), dict(out=c.q.float())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(q=c.q[None]), dict(q=c.q[:, :, :32]), dict(s=c.starts[:2]), dict(n=c.ctx[:1]),
               dict(v=c.v[:1]), dict(q=c.q.cpu()), dict(out=c.q[:3]), dict(q=c.q.transpose(0, 1))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises((TypeError, ValueError)):
        call(k_scale=torch.ones(2, device="cuda"))
    for kw in (dict(most=c.mbs * 16 + 1), dict(window_size=-1), dict(partition_size=-128),
               dict(q=c.q[:, :3].contiguous())):
        with pytest.raises(pa.PagedAttnError):
            call(**kw)


@pytest.mark.parametrize("fp8", [False, True])
def test_units_taken_as_ctas_come_free(fp8):
    """More query tiles than SMs: a counter in the workspace, whatever it held, on two streams at
    once with workspaces of their own, and by two graphs in turn on one."""
    c = Prompts(50, [1400, 0, 1300], [0, 3, 200], 16, 16, 64, fp8=fp8, behind=5)
    d = Prompts(51, [900, 2000], [600, 0], 16, 16, 64, fp8=fp8)
    want = [run(x)[:sum(x.new)] for x in (c, d)]
    sizes = [pa.prompt_workspace_size(x.N, len(x.new), 16, 16, x.most, 64) for x in (c, d)]
    assert sizes == [256, 256]
    outs = []
    for x in (c, d):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(attend(x))
    torch.cuda.synchronize()
    for x, w, o in zip((c, d), want, outs):
        assert torch.equal(o[:sum(x.new)], w)
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    graphs = []
    for x in (c, d):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = attend(x, workspace=ws, out=torch.zeros_like(x.q))
        graphs.append((g, out))
    for _ in range(3):
        for g, _out in graphs:
            g.replay()
    torch.cuda.synchronize()
    for x, w, (_, o) in zip((c, d), want, graphs):
        assert torch.equal(o[:sum(x.new)], w)
    assert pa.get_device_error() == 0


def test_rows_past_32_bits():
    """2^31 elements of q and out, and pages past 4 GB, at their ends."""
    B, Hq, Hkv, D = 66000, 128, 8, 128
    g = torch.Generator(device="cuda").manual_seed(52)
    NB = 140000                                           # 4.6 GB each for K and V
    k = torch.zeros((NB, Hkv, 16, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    for x in (k, v):
        x[:4] = torch.randn((4, Hkv, 16, D), generator=g, device="cuda").bfloat16()
        x[-4:] = torch.randn((4, Hkv, 16, D), generator=g, device="cuda").bfloat16()
    q = torch.empty((2 * B, Hq, D), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    assert q.numel() > 2 ** 31
    tables = torch.arange(B, device="cuda").int()[:, None] % 4
    tables[1::2] += NB - 4
    lens = torch.full((B,), 5, dtype=torch.int32, device="cuda")
    starts = torch.arange(B + 1, device="cuda").int() * 2
    out = pa.prompt_attention(q, k, v, tables, lens, starts, 16)
    assert pa.get_device_error() == 0
    for b in (0, 1, 65535, 65998, 65999):
        kk, vv = (x[tables[b, 0], :, :5].double().repeat_interleave(Hq // Hkv, 0) for x in (k, v))
        s = torch.einsum("nhd,hld->hnl", q[2 * b:2 * b + 2].double(), kk) * D ** -0.5
        s[:, 0, 4] = -float("inf")
        w = s.softmax(-1)
        check(out[2 * b:2 * b + 2], torch.einsum("hnl,hld->nhd", w, vv),
              torch.einsum("hnl,hld->nhd", w, vv.abs()))
