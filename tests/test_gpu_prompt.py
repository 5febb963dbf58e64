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
