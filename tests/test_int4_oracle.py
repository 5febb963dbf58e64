"""Pins of the INT4-page and bounded-cache oracles (no GPU)."""
import itertools

import numpy as np
import pytest

import workloads as W
from bounded_cases import Case
from oracle import bounded as BD
from oracle import fp8 as F
from oracle import int4 as Q4
from oracle import oracle as O


def test_quantisation_error_is_half_a_step():
    rng = np.random.default_rng(0)
    x = W.f32_to_bf16_bits(rng.standard_normal((50, 128)).astype(np.float32))
    hs = 0.07
    codes, scales = Q4.quantize(x, hs)
    assert codes.min() >= 1 and codes.max() <= 15
    v, y = O.bf16_bits_to_f64(x), Q4.dequantize(codes, scales, hs)
    step = np.repeat(F.decode(scales), 32, -1) * float(np.float32(hs))
    inside = np.abs(v) <= 7.5 * step
    assert (np.abs(v - y)[inside] <= 0.5 * step[inside] * (1 + 1e-6)).all()
    # the scale rounds down by at most 1/16 of itself: 7 steps reach all but 1/16 of the largest
    assert (np.abs(v - y) <= np.maximum(0.5, 7 / 16) * step * (1 + 1e-6)).all()


def test_nearest_code_by_search():
    """Every code is the nearest of the 15, the even one at a tie."""
    rng = np.random.default_rng(1)
    x = W.f32_to_bf16_bits((rng.integers(-64, 65, (40, 32)) / 8).astype(np.float32))
    hs = 0.25
    codes, scales = Q4.quantize(x, hs)
    v = O.bf16_bits_to_f64(x)
    ties = 0
    for i in range(40):
        step = F.decode(scales[i])[0] * hs
        for d in range(32):
            err = [abs(v[i, d] - k * step) for k in range(-7, 8)]
            best = [k for k in range(-7, 8) if err[k + 7] == min(err)]
            ties += len(best) == 2
            k = best[0] if len(best) == 1 else [z for z in best if z % 2 == 0][0]
            assert codes[i, d] == k + 8
    assert ties > 5


def test_special_groups():
    x = np.zeros((4, 32), dtype=np.float32)
    x[1, 3], x[2, 5], x[3, 7] = np.nan, np.inf, -1e30
    x[2:, 0] = 1.0
    codes, scales = Q4.quantize(W.f32_to_bf16_bits(x), 0.5)
    assert scales[0, 0] == 0 and (codes[0] == 8).all()
    assert scales[1, 0] == 0x7F and np.isnan(Q4.dequantize(codes, scales, 0.5)[1]).all()
    assert scales[2, 0] == 0x7E and codes[2, 5] == 15
    assert scales[3, 0] == 0x7E and codes[3, 7] == 1


def test_pack_round_trip_and_layout():
    rng = np.random.default_rng(2)
    codes = rng.integers(0, 16, (3, 2, 16, 64), dtype=np.uint8)
    scales = rng.integers(0, 256, (3, 2, 16, 2), dtype=np.uint8)
    pages = Q4.pack(codes, scales)
    assert pages.shape == (3, 2, Q4.page_bytes(64)) and Q4.page_bytes(128) == 1088
    c, s = Q4.unpack(pages, 64)
    assert (c == codes).all() and (s == scales).all()
    t, d = 5, 37
    assert (pages[1, 1, t * 32 + d // 2] >> (4 * (d % 2))) & 15 == codes[1, 1, t, d]
    assert pages[2, 0, 16 * 32 + t * 2 + 1] == scales[2, 0, t, 1]


def test_attention_equals_dense_bf16_oracle():
    """On values that bf16 holds exactly, INT4 attention is the bf16 oracle's."""
    c = Case(3, [1, 15, 16, 40], 4, 2, 64, power_of_two=True)
    out, _ = Q4.attention(c.q, c.k, c.v, c.k_scale, c.v_scale, c.tables, c.lens, c.scale)
    pools = []
    for pages, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
        codes, sc = Q4.unpack(pages, 64)
        x = np.stack([Q4.dequantize(codes[:, h], sc[:, h], scale[h]) for h in range(2)], 1)
        pools.append(W.f32_to_bf16_bits(np.nan_to_num(x).astype(np.float32)))
    ref = O.paged_attention(c.q, *pools, c.tables, c.lens, c.scale, 2, 16)
    assert np.abs(out - ref).max() < 1e-12


def test_weights_sum_to_the_number_of_rows():
    c = Case(4, [7, 33], 6, 2, 64, T=3)
    keys = [[c.rows(c.k, b, g, c.lens[b], "k") for g in range(2)] for b in range(2)]
    w0, p0 = np.full((2, 2, 48), 5.0), np.zeros((2, 2, 48), dtype=np.int32)
    w, pos, gained = BD.accumulate(w0, p0, c.q, keys, c.lens, c.lens + 10, c.scale, 0.5)
    assert np.allclose(gained.sum(-1), 9)                       # 3 heads of 3 tokens
    assert (w[0, :, 7:] == 5).all() and (pos[1, :, 30:33] == [40, 41, 42]).all()
    assert np.allclose(w[1, 0, :30], 2.5 + gained[1, 0, :30])


def test_select_keeps_the_best_set():
    """Against every subset of the right size, on small cases with ties."""
    rng = np.random.default_rng(5)
    for _ in range(200):
        n = int(rng.integers(1, 9))
        budget = int(rng.integers(1, 9))
        recent = int(rng.integers(0, budget + 1))
        w = rng.integers(0, 4, n).astype(float)
        pos = rng.permutation(n)
        moves = BD.select(w, pos, budget, recent)
        if n <= budget:
            assert moves == []
            continue
        entry = list(range(n))
        for a, z in moves:
            assert a >= budget > z
            entry[z] = a
        kept = entry[:budget]
        assert len(set(kept)) == budget
        newest = [j for j in range(n) if pos[j] > n - 1 - recent]
        assert set(newest) <= set(kept)
        rest = [j for j in range(n) if j not in newest]
        best = max(sum(w[list(s)]) for s in itertools.combinations(rest, budget - len(newest)))
        assert sum(w[j] for j in kept if j not in newest) == pytest.approx(best)
        for j in kept:                                    # ties: no dropped equal below a kept one
            if j not in newest:
                assert all(i in kept or w[i] < w[j] or i > j for i in rest)
