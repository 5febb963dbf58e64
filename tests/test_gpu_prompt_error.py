"""How far attention of packed prompts is from 64 bits: the relative L2 error that every bf16
output of the library keeps to, where the bound per element says little.

Rounding the exact outputs to bf16 alone is 1.6e-3 to 1.7e-3 with normal inputs; weights held in 8
significant bits would add 1.6e-3 in squares, weights in 11 bits 1e-4.  A page of 16 keys left out
of a context of n is sqrt(16 / n), 2.8e-2 of 20000 and 1.6e-2 of 65552.
"""
import pytest
import torch

import paged_kv_cache_221_gb300 as pa
from gpu_util import MAX_REL_L2
from prompt_cases import Prompts, check

pytestmark = pytest.mark.gpu


def run(c, window=0, factor=None, **kw):
    """The error of every head's outputs, and the bound per element; ``factor`` is one on the
    values of each head dim, divided out again so that every dim counts."""
    got = pa.prompt_attention(c.q, c.k, c.v, c.tables, c.ctx, c.starts, c.most, window_size=window,
                              k_scale=c.k_scale, v_scale=c.v_scale, **kw)
    assert pa.get_device_error() == 0
    rows = slice(0, sum(c.new))
    out, size = c.exact(window=window)
    check(got, out, size, rows=rows)
    got, out = got[rows].double(), out[rows]
    if factor is not None:
        got, out = got / factor, out / factor
    off = (got - out).norm(dim=(0, 2)) / out.norm(dim=(0, 2))
    assert off.max() <= MAX_REL_L2, f"relative L2 {off.max().item():.2e}"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_prompts(D, fp8):
    run(Prompts(1, [700, 128, 33, 1000], [0, 0, 0, 0], 16, 4, D, fp8=fp8))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_windows(D, fp8):
    run(Prompts(2, [1500, 40], [0, 900], 8, 2, D, fp8=fp8), window=300)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [(8, 2), (32, 4)])
def test_chunks_behind_long_contexts(heads, fp8):
    run(Prompts(3, [130, 64], [20000, 9001], *heads, 128, fp8=fp8))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cached", [19987, 65519])
def test_questions(cached, fp8):
    run(Prompts(4, [33], [cached], 16, 4, 128, fp8=fp8))


@pytest.mark.parametrize("power", [-100, -40, -24, -16, -9, -4, 4, 8, 9, 12, 40, 90])
@pytest.mark.parametrize("D", [64, 128])
def test_sizes_of_values(D, power):
    """A power of two on V is one on the outputs, bit for bit, or the error stays where it is:
    values far outside f16, and on both sides of what it holds."""
    c = Prompts(5, [300, 60], [0, 1000], 8, 2, D)
    c.v = c.v * 2.0 ** power
    run(c, factor=2.0 ** power)
    run(c, factor=2.0 ** power, partition_size=256)


@pytest.mark.parametrize("window", [0, 200])
def test_pages_and_dims_of_different_sizes(window):
    """Every page, and every head dim, with a size of its own."""
    for what in range(3):
        c = Prompts(6 + what, [500, 1, 90], [0, 300, 700], 8, 2, 128)
        g = torch.Generator(device="cuda").manual_seed(what)
        page = 2.0 ** torch.randint(-14, 14, (c.NB, 1, 1, 1), generator=g, device="cuda")
        dim = 2.0 ** torch.randint(-60, 60, (128,), generator=g, device="cuda")
        if what != 1:
            c.v = (c.v * page).bfloat16()
        if what != 0:
            c.v = (c.v * dim).bfloat16()
        run(c, window=window, factor=dim.double() if what else None)


def test_single_pages_that_f16_does_not_hold():
    """One large or tiny value makes its page a different one for the matrix product."""
    for value in (600.0, 3e4, 1e6, 2.0 ** -25, 2.0 ** -60, 1e-38):
        c = Prompts(9, [400, 20], [0, 800], 8, 2, 128)
        for j in range(0, 400, 37):
            blk = int(c.tables[0, j // 16])
            c.v[blk, j % 2, j % 16, (5 * j) % 128] = value
        run(c)
        run(c, partition_size=128)


def test_weights_of_every_size():
    """A first key that takes nearly all of the weight, with values of zero: what remains is the
    rest's, whose weights are 2^-8 to 2^-20 of the largest."""
    for gap in (6, 10, 14):
        c = Prompts(10, [400, 90], [0, 500], 4, 4, 128)
        c.q[:, :, 0] = 16.0
        c.k[:, :, :, 0] = 0
        for b in range(2):
            blk = int(c.tables[b, 0])
            c.k[blk, :, 0] = 0
            c.k[blk, :, 0, 0] = gap / 16.0 * 128 ** 0.5
            c.v[blk, :, 0] = 0
        run(c)


@pytest.mark.parametrize("D", [64, 128])
def test_values_with_zeros(D):
    """Head dims, keys and pages of zeros, of both signs."""
    c = Prompts(11, [300, 60], [0, 1000], 8, 2, D)
    c.v[..., D // 2:] = 0
    c.v[:, :, 3] = -0.0
    c.v[int(c.tables[0, 2])] = 0
    run(c)
    run(c, partition_size=256)
    run(c, window=150)
