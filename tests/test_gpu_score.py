"""Log probabilities, entropy and alternatives of rows of logits, against 64 bits."""
import math

import pytest
import torch

import paged_kv_cache_221_gb300 as pa

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def exact(x, tokens):
    x = x.double()
    lp = x - x.amax(-1, keepdim=True)             # 64 bits do not hold ln V beside fp32's lowest
    lp = lp - lp.exp().sum(-1, keepdim=True).log()
    p = lp.exp()
    h = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    given = torch.where(tokens < 0, 0.0, lp.gather(-1, tokens.clamp(min=0).long()[:, None])[:, 0])
    return lp, given, h


def bounds(x, lp):
    """fp32: a sum of V terms over 512 threads in pairs, 64 steps to join them, 2^-24 each; a
    term's argument and exponential, 2^-22 each; differences of logits, 2^-24 of the larger."""
    x = x.double()
    V = x.shape[-1]
    steps = (V / 1024 + 64) * 2.0 ** -24 + 2.0 ** -21
    top = x.amax(-1)
    far = torch.where(lp > -math.inf, lp.exp() * (x - top[:, None]).abs(), 0.0).sum(-1)
    rel = steps + 2.0 ** -22 * (far + 8)
    given = lambda v: rel + 2.0 ** -22 * (v.nan_to_num(0, 0, 0).abs() + top.abs())  # noqa: E731
    return given, rel * (2 + 2 * (far + 8))


def run(x, tokens, k):
    got = pa.token_logprobs(x, tokens, k)
    assert pa.get_device_error() == 0
    lp, given, h = exact(x, tokens)
    near, eh = bounds(x, lp)
    finite = given > -math.inf
    assert torch.equal(got[0].double()[~finite], given[~finite])
    assert ((got[0].double() - given).abs()[finite] <= near(given)[finite]).all()
    assert ((got[1].double() - h).abs() <= eh).all()
    order = torch.sort(x.float(), dim=-1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(got[3].long(), order)
    for c in range(k):
        v = lp.gather(-1, order[:, c:c + 1])[:, 0]
        f = v > -math.inf
        assert torch.equal(got[2][:, c].double()[~f], v[~f])
        assert ((got[2][:, c].double() - v).abs()[f] <= near(v)[f]).all()
    return got


def logits(seed, N, V, dtype, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((N, V), generator=g, device="cuda") * spread).to(dtype)
    return x, torch.randint(0, V, (N,), generator=g, device="cuda").int()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 16, 31, 127, 500, 1000, 2047, 4095, 4101, 8191, 32003])
@pytest.mark.parametrize("N", [1, 3, 160])
def test_sizes(N, V, dtype):
    x, t = logits(V + N, N, V, dtype)
    run(x, t, min(V, 20))


@pytest.mark.parametrize("k", [0, 1, 15, 16, 17, 31, 32])
@pytest.mark.parametrize("N", [2, 200])
def test_numbers_of_alternatives(N, k):
    x, t = logits(k, N, 50257, torch.bfloat16)
    run(x, t, k)


def test_full_vocabulary():
    for dtype in TYPES:
        x, t = logits(1, 3, 128256, dtype)
        run(x, t, 20)
    x, t = logits(2, 300, 128256, torch.bfloat16, spread=8.0)
    run(x, t, 5)
    x, t = logits(3, 2, 2 ** 19, torch.float16)
    run(x, t, 32)


@pytest.mark.parametrize("N", [4, 170])
@pytest.mark.parametrize("dtype", TYPES)
def test_ties(N, dtype):
    """Equal values: the lower index first, also where they are the whole row."""
    V = 40000
    x, t = logits(7, N, V, dtype)
    run((x * 2).round() / 2, t, 20)
    run(torch.zeros_like(x), t, 20)
    run(torch.full_like(x, -3.5), t, 32)
    y = torch.zeros_like(x)
    y[:, ::2] = -0.0                                    # the zeros are equal
    y[:, 39990] = 1.0
    run(y, t, 7)


@pytest.mark.parametrize("N", [4, 170])
def test_masked_rows(N):
    """-inf almost everywhere, as under a grammar; alternatives reach into the masked tokens."""
    V = 50000
    x, t = logits(8, N, V, torch.float32)
    y = torch.full_like(x, -math.inf)
    for i, keep in enumerate((1, 2, 5, 40)):
        y[i::4, 100 * i + 7:100 * i + 7 + keep] = x[i::4, :keep]
    run(y, t, 20)
    low = torch.finfo(torch.float32).min
    z = torch.full_like(x, low)
    z[:, 17] = 0.5
    run(z, t, 20)
    for dtype in TYPES:                                  # nothing but the lowest value
        run(torch.full((N, V), torch.finfo(dtype).min, dtype=dtype, device="cuda"), t, 3)


def test_values_in_order():
    """Ascending and descending rows, and large values in one thread's elements alone."""
    V = 60000
    x = torch.arange(V, device="cuda").float()[None].repeat(160, 1) / 1000
    x[1::2] = x[1::2].flip(-1)
    t = torch.zeros(160, dtype=torch.int32, device="cuda")
    run(x, t, 32)
    y, t = logits(9, 160, V, torch.float32)
    y[:, (torch.arange(V, device="cuda") // 4) % 512 == 37] += 100.0
    run(y, t, 32)
    run(y[:3], t[:3], 32)


def test_more_large_values_than_a_list_holds():
    """Above every bound from thread maxima: one warp's threads hold all the large values."""
    V = 400000
    y, t = logits(10, 2, V, torch.float32)
    y[:, (torch.arange(V, device="cuda") // 4) % 512 < 31] += 100.0
    run(y, t, 32)
    y, t = logits(11, 160, V, torch.float32)
    y[:, (torch.arange(V, device="cuda") // 4) % 512 < 31] += 100.0
    run(y, t, 32)


def test_rows_without_results():
    for N in (3, 160):
        for bad in (math.nan, math.inf):
            x, t = logits(12, N, 3000, torch.float32)
            x[1, 700] = bad
            lp, h, top, tok = pa.token_logprobs(x, t, 4)
            assert torch.isnan(lp[1]) and torch.isnan(h[1]) and torch.isnan(top[1]).all()
            assert ((tok >= 0) & (tok < 3000)).all()
            rest = torch.arange(N, device="cuda") != 1
            assert torch.isfinite(lp[rest]).all() and torch.isfinite(top[rest]).all()
        x, t = logits(13, N, 3000, torch.float32)
        x[2] = -math.inf
        lp, h, top, tok = pa.token_logprobs(x, t, 4)
        assert torch.isnan(lp[2]) and torch.isnan(h[2]) and torch.isnan(top[2]).all()
        x[2] = math.nan
        assert torch.isnan(pa.token_logprobs(x, t, 4)[0][2])
    assert pa.get_device_error() == 0


def test_strided_rows_and_given_tokens():
    x, t = logits(14, 9, 1003, torch.bfloat16)
    t[3], t[4] = -1, -7
    got = run(x[:, :1001], t.clamp(max=1000), 5)
    assert got[0][3] == 0 and got[0][4] == 0
    run(x[1::2, 1:1000], t[1::2].clamp(max=998).contiguous(), 5)
    t[0] = 1003
    lp = pa.token_logprobs(x, t)[0]
    assert torch.isnan(lp[0]) and torch.isfinite(lp[1:]).all()
    assert pa.get_device_error() == 5                    # PA_ERR_BOUNDS


def test_stream_graph_and_empty():
    x, t = logits(15, 40, 32000, torch.bfloat16)
    want = pa.token_logprobs(x, t, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = pa.token_logprobs(x, t, 8)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = pa.token_logprobs(x, t, 8)
    y, _ = logits(16, 40, 32000, torch.bfloat16)
    x.copy_(y)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(pa.token_logprobs(y, t, 8), got))
    out = pa.token_logprobs(x[:0], t[:0], 3)
    assert [tuple(o.shape) for o in out] == [(0,), (0,), (0, 3), (0, 3)]


def test_refusals():
    x, t = logits(17, 4, 100, torch.float32)
    with pytest.raises(TypeError):
        pa.token_logprobs(x.double(), t)
    with pytest.raises(TypeError):
        pa.token_logprobs(x, t.long())
    with pytest.raises(ValueError):
        pa.token_logprobs(x, t[:3])
    with pytest.raises(ValueError):
        pa.token_logprobs(x.T, t)
    with pytest.raises(ValueError):
        pa.token_logprobs(x, t, 33)
    with pytest.raises(ValueError):
        pa.token_logprobs(x[:, :5], t, 6)
    with pytest.raises(ValueError):
        pa.token_logprobs(x[:1].expand(4, 100), t)
    with pytest.raises(ValueError):
        pa.token_logprobs(x.cpu(), t)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_that_a_cluster_shares(dtype):
    """Few and long rows: ties over all parts, masks, odd places, rows without results."""
    V, N = 50001, 3
    x, t = logits(20, N, V, dtype)
    run((x * 2).round() / 2, t, 20)
    for v in (0.0, torch.finfo(dtype).min):
        run(torch.full_like(x, v), t, 32)
    y = torch.full_like(x, -math.inf)
    y[:, [0, 6250, 6251, 25000, 49999, 50000]] = x[:, :6]
    run(y, t, 20)
    run(x[:, 1:], t.clamp(max=V - 2), 20)
    run(x[::2, 3:], t[::2].clamp(max=V - 4).contiguous(), 0)
    for bad in (math.nan, math.inf):
        z = x.clone()
        z[1, 31000] = bad
        lp, h, top, tok = pa.token_logprobs(z, t, 4)
        assert torch.isnan(lp[1]) and torch.isnan(h[1]) and torch.isnan(top[1]).all()
        assert ((tok >= 0) & (tok < V)).all()
        assert torch.isfinite(lp[::2]).all() and torch.isfinite(top[::2]).all()
    z[2] = -math.inf
    lp, h, top, tok = pa.token_logprobs(z, t, 4)
    assert torch.isnan(lp[2]) and torch.isnan(h[2]) and torch.isnan(top[2]).all()
    t[0] = V
    lp = pa.token_logprobs(x, t)[0]
    assert torch.isnan(lp[0]) and torch.isfinite(lp[1:]).all()
    assert pa.get_device_error() == 5


def test_rows_past_32_bits():
    x = torch.empty((17000, 128256), dtype=torch.bfloat16, device="cuda").normal_()
    assert x.numel() > 2 ** 31
    t = torch.full((17000,), 128255, dtype=torch.int32, device="cuda")
    got = pa.token_logprobs(x, t, 3)
    for a, b in zip(got, run(x[-200:], t[-200:], 3)):
        assert torch.equal(a[-200:], b)
