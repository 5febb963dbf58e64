"""Prompt attention where its arithmetic has its borders, against values worked out by hand."""
import math

import pytest
import torch

import paged_kv_cache_221_gb300 as pa
from gpu_util import MAX_REL_L2
from prompt_cases import Prompts, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("step", [8, 16, 64])
@pytest.mark.parametrize("start", [2 ** 26 - 64, 2 ** 26, 2 ** 26 + 64])
def test_scores_that_a_few_bits_tell_apart(start, step, fp8):
    """Scores past 2^26 are multiples of 8 in fp32: each tile's best one is `step` above the last
    tile's, in powers of two, and the weights 2^0, 2^step, .. 2^(3 step) hold to the end."""
    c = Prompts(1, [600], [0], 2, 2, 128, fp8=fp8)
    kind = torch.uint8 if fp8 else torch.bfloat16
    # k = (2^13, n, 0 ..) and q = (2^13, 8, 0 ..): 2^26 + 8 n; FP8 codes of 2^8 and n / 32 with
    # scales of 2^5, where n / 32 is an E4M3 value for the n below
    first, top, scale = (2.0 ** 8, 2.0 ** 5, 2.0 ** 5) if fp8 else (2.0 ** 13, 1.0, 1.0)
    k = torch.zeros((c.NB, 2, 16, 128), device="cuda")
    want_n = {0: (start - 2 ** 26) // 8}
    for t in range(1, 4):
        want_n[128 * t + 5] = want_n[0] + t * step // 8
    for j, n in want_n.items():
        blk, at = int(c.tables[0, j // 16]), j % 16
        k[blk, :, at, 0] = first
        k[blk, :, at, 1] = n / top
    if fp8:
        code = k.to(torch.float8_e4m3fn)
        assert torch.equal(code.float(), k)
        c.k, c.k_scale = code.view(torch.uint8), torch.full_like(c.k_scale, scale)
        assert c.k.dtype == kind
    else:
        c.k = k.to(kind)
        assert torch.equal(c.k.float(), k)
    c.q = torch.zeros_like(c.q)
    c.q[:, :, 0], c.q[:, :, 1] = 2.0 ** 13, 8.0
    got = pa.prompt_attention(c.q, c.k, c.v, c.tables, c.ctx, c.starts, c.most,
                              scale=math.log(2.0), k_scale=c.k_scale, v_scale=c.v_scale)
    assert pa.get_device_error() == 0
    _, v = c.kv(0)
    s = torch.full((600, 600), -math.inf, dtype=torch.float64, device="cuda")
    for j, n in want_n.items():
        s[j:, j] = 8.0 * (n - want_n[0])
    w = torch.softmax(s * math.log(2.0), -1)
    want = torch.einsum("nj,hjd->nhd", w, v)
    size = torch.einsum("nj,hjd->nhd", w, v.abs())
    assert torch.isfinite(got).all()
    assert ((got.double() - want).abs() <= 2.0 ** -8 * (want.abs() + size) * (1 + 2.0 ** -4)).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("mark", [-1, 2 ** 31 - 1])
@pytest.mark.parametrize("window", [1, 16, 17, 100, 128, 300])
def test_blocks_in_front_of_the_window_may_be_gone(window, mark, fp8):
    """Table entries of blocks wholly before the first query token's window are not looked at, and
    neither is what the blocks hold, as for single-token attention."""
    kind = dict(fp8=fp8, extra_blocks=2)
    for new, cached in (([300, 1, 130], [0, 400, 777]), ([1] * 9, [61 * i for i in range(9)])):
        c = Prompts(2, new, cached, 8, 2, 128, **kind)
        most = dict(window_size=window, k_scale=c.k_scale, v_scale=c.v_scale)

        def attend(tables, **kw):
            return pa.prompt_attention(c.q, c.k, c.v, tables, c.ctx, c.starts, c.most, **most, **kw)
        want = attend(c.tables), attend(c.tables, partition_size=128)
        assert pa.get_device_error() == 0
        gone, held = c.tables.clone(), c.tables
        for b, n in enumerate(cached):
            first = max(0, n - window + 1) // 16
            for blk in held[b, :first].tolist():
                c.k[blk] = c.v[blk] = 0x7F if fp8 else float("nan")
            gone[b, :first] = mark
        got = attend(gone), attend(gone, partition_size=128)
        assert pa.get_device_error() == 0
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        if len(set(new)) == 1:                            # the same call of single-token attention
            pa.attention(c.q[:, None], c.k, c.v, gone, c.ctx, c.most, **most)
            assert pa.get_device_error() == 0
        # the first block that the window reaches is looked at
        b = max(range(len(cached)), key=cached.__getitem__)
        gone[b, max(0, cached[b] - window + 1) // 16] = mark
        attend(gone)
        assert pa.get_device_error() == 5


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B", [2, 4, 8])
def test_cut_keys_shared_out_by_a_counter(B, fp8):
    """Several short questions behind long contexts: their keys are cut and the partitions taken as
    CTAs come free, whatever the workspace held, twice, and from a graph with other lengths."""
    Hq, Hkv, D = 32, 8, 128
    cached = [31999 - 3001 * b % 9000 for b in range(B)]
    c = Prompts(3 + B, [64] * B, cached, Hq, Hkv, D, fp8=fp8)
    size = pa.prompt_workspace_size(c.N, B, Hq, Hkv, c.most, D)
    # partial results of every row, their statistics, and the counter
    parts = (size - 256) // (c.N * Hq * (4 * D + 8))
    assert parts > 1 and size == c.N * Hq * parts * (4 * D + 8) + 256
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")

    def attend(**kw):
        return pa.prompt_attention(c.q, c.k, c.v, c.tables, c.ctx, c.starts, c.most,
                                   k_scale=c.k_scale, v_scale=c.v_scale, **kw)
    got = attend(workspace=ws)
    assert pa.get_device_error() == 0
    want, size = c.exact()
    check(got, want, size)
    off = (got.double() - want).norm(dim=(0, 2)) / want.norm(dim=(0, 2))
    assert off.max() <= MAX_REL_L2
    assert torch.equal(attend(workspace=ws), got) and torch.equal(attend(), got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = attend(workspace=ws)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got)
    c.ctx -= torch.arange(B, device="cuda").int() * 2000
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, attend()) and pa.get_device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("order", ["codes", "mixed"])
def test_every_value_by_itself(order, D):
    """Rows that see one key return its values, bit for bit: every bf16 from 2^-126 to below 2^100
    and 0, page by page alike and page by page of all sizes."""
    codes = torch.arange(128, (127 + 100) << 7, device="cuda").int()
    codes = torch.cat([codes, codes + 0x8000, torch.zeros(64, device="cuda").int()])
    N = -(-codes.numel() // D)
    codes = torch.cat([codes, codes[:N * D - codes.numel()]])
    if order == "mixed":
        g = torch.Generator(device="cuda").manual_seed(D)
        codes = codes[torch.randperm(N * D, generator=g, device="cuda")]
    rows = codes.to(torch.int16).view(torch.bfloat16).view(N, D)
    c = Prompts(4, [N], [0], 4, 2, D)
    j = torch.arange(N, device="cuda")
    for head in range(2):
        c.v[c.tables[0, j // 16].long(), head, j % 16] = rows
    for kw in (dict(), dict(partition_size=128)):
        got = pa.prompt_attention(c.q, c.k, c.v, c.tables, c.ctx, c.starts, c.most, window_size=1,
                                  **kw)
        assert pa.get_device_error() == 0
        assert torch.equal(got, rows[:, None].expand(-1, 4, -1))


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("gap", [5, 25, 40, 80, 200])
def test_infinities_of_small_weights(gap, value):
    """An infinite or NaN value reaches the rows that see it however small its weight is, in pages
    that all rows see as at the mask's border; other head dims stay as they are."""
    c = Prompts(5, [200, 3], [400, 40], 4, 2, 128)
    c.q[:, :, 0] = 16.0
    c.k[:, :, :, 0] = 0
    for b, keys in enumerate(((7, 100, 395, 420), (5, 41))):
        for j in keys:
            blk = int(c.tables[b, j // 16])
            c.k[blk, :, j % 16] = 0
            c.k[blk, :, j % 16, 0] = -gap / 16.0 * 128 ** 0.5
            c.v[blk, :, j % 16, j % 128] = value
    for kw in (dict(), dict(partition_size=128), dict(window_size=330)):
        got = pa.prompt_attention(c.q, c.k, c.v, c.tables, c.ctx, c.starts, c.most, **kw)
        assert pa.get_device_error() == 0
        check(got, *c.exact(window=kw.get("window_size", 0)))


@pytest.mark.parametrize("fp8", [False, True])
def test_values_that_are_not_finite_anywhere(fp8):
    """Scattered over a long context, of both signs, and nothing else in some head dims."""
    c = Prompts(6, [300, 64], [3000, 9000], 8, 2, 128, fp8=fp8)
    g = torch.Generator(device="cuda").manual_seed(1)
    at = torch.rand(c.v.shape, generator=g, device="cuda")
    if fp8:
        c.v[at < 2e-6] = 0x7F
        c.v[:, :, 17] = 0x7F
    else:
        c.v[at < 1e-6] = math.inf
        c.v[at > 1 - 1e-6] = -math.inf
        c.v[..., 17] = math.nan
        c.v[..., 18] = math.inf
    for kw in (dict(), dict(partition_size=1024), dict(window_size=500)):
        got = pa.prompt_attention(c.q, c.k, c.v, c.tables, c.ctx, c.starts, c.most,
                                  k_scale=c.k_scale, v_scale=c.v_scale, **kw)
        assert pa.get_device_error() == 0
        out, size = exact_of_parts(c, kw.get("window_size", 0))
        check(got, out, size)


def exact_of_parts(c, window):
    """As Prompts.exact, the values that are not finite apart: a row that sees some in a head dim
    has their sum there."""
    kind = 0x7F if c.fp8 else None
    odd = c.v == kind if c.fp8 else ~torch.isfinite(c.v)
    used = c.v.clone()
    c.v = torch.where(odd, torch.zeros_like(used), used)
    out, size = c.exact(window=window)
    c.v = used
    row, G = 0, c.Hq // c.Hkv
    for b, (n, L) in enumerate(zip(c.new, c.lens)):
        _, v = c.kv(b)
        pos = torch.arange(L - n, L, device="cuda")
        first = (pos - window + 1).clamp(min=0) if window else torch.zeros_like(pos)
        v = v.repeat_interleave(G, 0)
        seen = {}
        for name, mark in (("nan", torch.isnan(v)), ("inf", v == math.inf), ("-inf", v == -math.inf)):
            count = torch.cat([torch.zeros_like(v[:, :1]), mark.double().cumsum(1)], 1)
            seen[name] = (count[:, pos + 1] - count[:, first] > 0).transpose(0, 1)
        rows = slice(row, row + n)
        out[rows] = torch.where(seen["inf"], math.inf, out[rows])
        out[rows] = torch.where(seen["-inf"], torch.where(seen["inf"], math.nan, -math.inf), out[rows])
        out[rows] = torch.where(seen["nan"], math.nan, out[rows])
        row += n
    return out, size


@pytest.mark.parametrize("value", [math.inf, -math.inf])
@pytest.mark.parametrize("gap", [60, 100, 300])
def test_infinities_behind_far_larger_scores(gap, value):
    """What was summed before a far larger score keeps its infinities, in one pass over the keys and
    where partitions are joined."""
    c = Prompts(7, [100], [600], 4, 2, 128)
    c.q[:, :, 0] = 16.0
    c.k[:, :, :, 0] = 0
    for j in range(300):
        c.k[int(c.tables[0, j // 16]), :, j % 16, 0] = -gap / 16.0 * 128 ** 0.5
    c.v[int(c.tables[0, 1]), :, 4, 9] = value             # of key 20
    for kw in (dict(), dict(partition_size=128), dict(partition_size=256)):
        got = pa.prompt_attention(c.q, c.k, c.v, c.tables, c.ctx, c.starts, c.most, **kw)
        assert pa.get_device_error() == 0
        out, size = c.exact()
        assert (out[:, :, 9] == value).all()
        check(got, out, size)
