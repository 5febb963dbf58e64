"""Log probabilities and entropy within what fp32 sums of this many terms can be off, against 64
bits, for rows of one CTA and of eight."""
import math

import pytest
import torch

import paged_kv_cache_221_gb300 as pa
from test_gpu_score import TYPES, exact, logits

pytestmark = pytest.mark.gpu


def bounds(x, lp):
    """A thread of 256 (of 8 x 256 where a cluster shares the row) adds its elements in steps of n,
    8 for float32 and 16 for the 16-bit types: n / 2 additions to its running sum and one to join
    the pair; then 5 joins of lanes, 8 of warps, 8 of CTAs.  2^-24 each, and in a join three
    operations more; a term's argument and exponential, 2^-22 each; differences of logits, 2^-24 of
    the larger."""
    n = 8 if x.dtype == torch.float32 else 16
    N, V = x.shape
    threads = 256 * (8 if N <= 64 and V >= max(48000, 1300 * N) else 1)
    x = x.double()
    steps = (V / threads * (n / 2 + 1) / n + 4 * (5 + 8 + 8)) * 2.0 ** -24 + 2.0 ** -21
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
    assert ((got[0].double() - given).abs() <= near(given)).all()
    assert ((got[1].double() - h).abs() <= eh).all()
    order = torch.sort(x.float(), dim=-1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(got[3].long(), order)
    for c in range(k):
        v = lp.gather(-1, order[:, c:c + 1])[:, 0]
        assert ((got[2][:, c].double() - v).abs() <= near(v)).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V", [(1, 48000), (3, 128256), (36, 47999), (64, 128256), (65, 128256),
                                 (38, 50257), (200, 32003), (5, 2 ** 19), (70, 2 ** 19)])
def test_sums(N, V, dtype):
    for spread in (0.0, 0.5, 4.0):
        x, t = logits(N + V, N, V, dtype, spread)
        run(x, t, 3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [3, 160])
def test_large_values_of_few_threads(N, dtype):
    """A thread's vectors are every 256th: all large values in one thread, or in one warp, whose
    maxima alone reach them."""
    V, n = 60000, 4 if dtype == torch.float32 else 8
    x, t = logits(N, N, V, dtype)
    at = torch.arange(V, device="cuda") // n % 256
    for few in (at == 37, at < 31, (at >= 64) & (at < 96)):
        y = x.clone()
        y[:, few] += 50.0
        run(y, t, 32)


@pytest.mark.parametrize("N,V", [(200, 4096), (4, 60000)])
def test_signs(N, V):
    """A log probability is never above 0 and an entropy never below, also where one token has
    nearly all of the probability and rounding is all that is left."""
    g = torch.Generator(device="cuda").manual_seed(V)
    for low in (-20.0, -40.0, -80.0):
        x = torch.randn((N, V), generator=g, device="cuda") + low
        rows = torch.arange(N, device="cuda")
        near = 5.4 * torch.rand(N, generator=g, device="cuda")
        shift = 10 * torch.randn(N, generator=g, device="cuda")
        x[rows, torch.randint(0, V // 2, (N,), generator=g, device="cuda")] = -near - 20.0
        at = torch.randint(V // 2, V, (N,), generator=g, device="cuda")
        x[rows, at] = 0.0
        x += shift[:, None]
        lp, h, top, _ = pa.token_logprobs(x, at.int(), 5)
        run(x, at.int(), 5)
        assert (lp <= 0).all() and (top <= 0).all() and (h >= 0).all()
        x[rows, torch.randint(0, V // 2, (N,), generator=g, device="cuda")] = shift - near
        lp, h, top, _ = pa.token_logprobs(x, at.int(), 5)
        run(x, at.int(), 5)
        assert (lp <= 0).all() and (top <= 0).all() and (h >= 0).all()
    x = torch.full((N, V), -math.inf, device="cuda")
    x[:, 5] = shift
    x[:, 5] += 0.1
    lp, h, top, _ = pa.token_logprobs(x, torch.full((N,), 5, dtype=torch.int32, device="cuda"), 1)
    assert (lp == 0).all() and (h == 0).all() and (top == 0).all()
