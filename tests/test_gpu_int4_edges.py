"""Attention over INT4 pages where roundings, masks and integer ranges meet their ends."""
import ctypes

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():          # collected on CPU-only hosts, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import __graft_entry__  # noqa: E402

__graft_entry__.build()

import paged_kv_cache_221_gb300 as pa  # noqa: E402
import workloads as W  # noqa: E402
from bounded_cases import Case  # noqa: E402
from gpu_util import to_dev  # noqa: E402
from oracle import fp8 as F  # noqa: E402
from oracle import int4 as Q4  # noqa: E402
from oracle import oracle as O  # noqa: E402


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert pa.get_device_error() == 0, "device error word was set"


def attend(c, **kw):
    return pa.attention_int4(to_dev(c.q), to_dev(c.k), to_dev(c.v), to_dev(c.k_scale),
                             to_dev(c.v_scale), to_dev(c.tables), to_dev(c.lens),
                             int(c.lens.max()), c.scale, **kw)


def check(out, c, window=0):
    """Against the oracle; NaN exactly where it has NaN.  The bound: the output is rounded to
    bf16 (2^-8 of it); a weight is rounded to f16, which moves it against its row's sum (2^-11 of
    it times |v| + |out|), and times its scale rounded again (2^-11), each of them at least
    by 2^-25 where the row's largest weight is 2^3 or more (so 2^-28 of the sum), times codes of
    at most 7; scores err by 2^-20 of sum |q k|."""
    with np.errstate(invalid="ignore"):
        ref, mag = Q4.attention(c.q, c.k, c.v, c.k_scale, c.v_scale, c.tables, c.lens, c.scale,
                                window)
    got = out.float().cpu().double().numpy()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))
    keys = [[c.rows(c.k, b, g, int(n), "k") for g in range(c.Hkv)] for b, n in enumerate(c.lens)]
    score = 2.0 ** -20 * c.score_size(keys)
    s_max = np.nanmax(F.decode(Q4.unpack(c.v, c.D)[1]))
    small = int(c.lens.max()) * 2.0 ** -28 * 7 * (2 * s_max + 1) * float(c.v_scale.max())
    tol = (2.0 ** -8 + 2.0 ** -11) * np.abs(ref) + (2.0 ** -10 + 2.0 ** -16 + score) * mag + small
    ok = ~np.isnan(ref)
    assert (np.abs(got - ref)[ok] <= tol[ok]).all(), f"by {(np.abs(got - ref) - tol)[ok].max():.3e}"
    return ref


# ------------------------------------------------------------------------------- windows
@pytest.mark.parametrize("T", [1, 2, 5, 16])
@pytest.mark.parametrize("psize", [0, 32])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 40, 1 << 30])
def test_window_up_to_the_largest(window, psize, T):
    """A window past every context is no window, up to the largest integer."""
    c = Case(T, [T, 17 + T, 96 + T, 97, 300], 4, 2, 64, T=T)
    plain = attend(c, partition_size=psize)
    assert torch.isfinite(plain.float()).all()
    assert torch.equal(attend(c, window_size=window, partition_size=psize), plain)


# ------------------------------------------------------------------------------- NaN in V
def spoil_value(c, b, j, g, group):
    codes, sc = Q4.unpack(c.v, c.D)
    sc = np.array(sc, copy=True)
    sc[c.tables[b, j // 16], g, j % 16, group] = 0x7F
    c.v = Q4.pack(codes, sc)


@pytest.mark.parametrize("Hq,Hkv,D,T", [(4, 2, 64, 2), (6, 2, 128, 3), (8, 2, 128, 5),
                                        (4, 1, 64, 7), (8, 1, 128, 5), (2, 1, 128, 20)])
@pytest.mark.parametrize("psize", [0, 32])
def test_nan_value_of_the_newest_draft(Hq, Hkv, D, T, psize):
    """A draft's NaN reaches the rows that see it, in the dims of its scale, and no others."""
    c = Case(41, [300, 33, T], Hq, Hkv, D, T=T)
    for b in range(3):
        spoil_value(c, b, int(c.lens[b]) - 1, 0, b % 2)
    ref = check(attend(c, partition_size=psize), c)
    G = Hq // Hkv
    assert np.isnan(ref[0, T - 1, :G, :32]).all() and np.isfinite(ref[0, :T - 1]).all()
    assert np.isfinite(ref[0, T - 1, :, 32:]).all()


@pytest.mark.parametrize("psize", [0, 16])
@pytest.mark.parametrize("T", [2, 5])
def test_nan_value_behind_a_window(T, psize):
    """Seen by the first query token alone, and by all of them in a page that is an edge."""
    c = Case(42, [300, 70], 4, 2, 64, T=T)
    spoil_value(c, 0, 300 - T - 20 + 1, 1, 0)
    spoil_value(c, 1, 70 - 20, 0, 1)
    ref = check(attend(c, window_size=20, partition_size=psize), c, window=20)
    assert np.isnan(ref[0, 0, 2:, :32]).all() and np.isfinite(ref[0, 1:]).all()
    assert np.isnan(ref[1, :, :2, 32:]).all()


@pytest.mark.parametrize("j", [0, 100, 299])
def test_nan_key(j):
    """A row that sees a NaN score is NaN in every dim."""
    c = Case(43, [300, 50], 4, 2, 64, T=3)
    codes, sc = Q4.unpack(c.k, 64)
    sc = np.array(sc, copy=True)
    sc[c.tables[0, j // 16], 1, j % 16, 0] = 0x7F
    c.k = Q4.pack(codes, sc)
    ref = check(attend(c), c)
    assert np.isnan(ref[0, 2, 2:]).all() and np.isfinite(ref[0, :, :2]).all()


# ------------------------------------------------------------------------------- faint weights
@pytest.mark.parametrize("octaves", [12.0, 17.3, 20.0, 21.6])
@pytest.mark.parametrize("scale_code", [0x08, 0x10, 0x38, 0x7E])     # 2^-6, 2^-5, 1, 448
@pytest.mark.parametrize("codes", ["zero", "mixed"])
@pytest.mark.parametrize("D,T", [(64, 1), (128, 5)])
def test_one_dominant_entry_and_a_faint_tail(octaves, scale_code, codes, D, T):
    """A sequence taken whole: one entry holds nearly all the weight, 16384 others 2^-octaves of
    it each.  What little they add must not be lost one-sidedly."""
    L = 16384 + T
    rng = np.random.default_rng(7)
    c = Case(44, [L], 1, 1, D, T=T, power_of_two=True)
    q = np.zeros((1, T, 1, D))
    q[..., 0] = 1.0
    c.q = (np.float32(q).view(np.uint32) >> 16).astype(np.uint16)
    kc = np.full((c.NB, 1, 16, D), 8, dtype=np.uint8)
    ks = np.full((c.NB, 1, 16, D // 32), 0x38, dtype=np.uint8)
    c.k_scale[:] = octaves * np.log(2.0) * np.sqrt(D) / 7          # score octaves ln 2
    kc[c.tables[0, 0], 0, 3, 0] = 15
    c.k = Q4.pack(kc, ks)
    vc = np.full((c.NB, 1, 16, D), 8, dtype=np.uint8) if codes == "zero" else \
        rng.integers(1, 16, (c.NB, 1, 16, D), dtype=np.uint8)
    vc[c.tables[0, 0], 0, 3] = rng.choice([1, 15], D)
    c.v = Q4.pack(vc, np.full((c.NB, 1, 16, D // 32), scale_code, dtype=np.uint8))
    t = {n: to_dev(getattr(c, n)) for n in ("q", "k", "v", "k_scale", "v_scale", "tables",
                                            "lens")}
    out = torch.empty_like(t["q"])
    p = {n: ctypes.c_void_p(x.data_ptr()) for n, x in t.items()}
    st = pa.library().pa_attention_int4(
        ctypes.c_void_p(out.data_ptr()), p["q"], None, None, p["k"], p["v"], p["k_scale"],
        p["v_scale"], 0, p["tables"], c.mbs, p["lens"], L, 1, T, c.NB, 1, 1, D, 16,
        float(c.scale), 0, None, 0, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    ref, mag = Q4.attention(c.q, c.k, c.v, c.k_scale, c.v_scale, c.tables, c.lens, c.scale)
    got = out.float().cpu().double().numpy()
    hs, s = float(c.v_scale[0]), float(F.decode(np.array([scale_code], dtype=np.uint8))[0])
    # as check(): scores of at most `octaves` octaves; weights and products below
    # 2^-14 lose at most 2^-25 each, of a sum that is at least 2^3, times 7
    tail = L * 2.0 ** -octaves * 7 * s * hs
    small = L * 2.0 ** -28 * 7 * hs * (2 * s + 1)
    tol = ((2.0 ** -8 + 2.0 ** -11) * np.abs(ref) + (2.0 ** -10 + 2.0 ** -16) * mag +
           2.0 ** -20 * octaves * (mag + tail) + small)
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"{(err / tol).max():.2f} of the bound"


# ------------------------------------------------------------------------------- large scores
@pytest.mark.parametrize("octaves", [24, 26, 30, 60, 90])
@pytest.mark.parametrize("psize,D,T", [(0, 64, 2), (32, 128, 1), (0, 128, 6)])
def test_scores_past_what_fp32_resolves(octaves, psize, D, T):
    """Scores so large that their rounding is octaves: the largest one takes all the weight."""
    c = Case(51, [T, 17 + T, 40, 300, 2000], 4, 2, D, T=T)
    c.q = W.f32_to_bf16_bits((O.bf16_bits_to_f64(c.q) * 2.0 ** octaves).astype(np.float32))
    got = attend(c, partition_size=psize).float().cpu().double().numpy()
    assert np.isfinite(got).all()
    checked = 0
    for b, n in enumerate(c.lens):
        for h in range(4):
            K, V = (c.rows(p, b, h // 2, int(n), name) for p, name in ((c.k, "k"), (c.v, "v")))
            for t in range(T):
                x = O.bf16_bits_to_f64(c.q[b, t, h])
                s = K[:n - T + t + 1] @ x
                size = (np.abs(K[:n - T + t + 1]) @ np.abs(x)).max()
                top = np.sort(s)[-2:]
                # A score errs by 2^-20 of sum |q k|: rows whose two largest are within four times
                # that do not count.  Of the others the second one is more than 100 octaves down
                # (2^-18 * 2^24 * 20 / 8, less the error), so that its weight is nothing.
                if len(s) > 1 and top[1] - top[0] < 2.0 ** -18 * size:
                    continue
                assert size > 20 * 2.0 ** octaves
                checked += 1
                ref = V[int(np.argmax(s))]
                # rounded to bf16, and times its scale to f16
                assert (np.abs(got[b, t, h] - ref) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(ref)).all()
    assert checked > 8 * T


@pytest.mark.parametrize("octaves", [98, 105, 118])
@pytest.mark.parametrize("T,D", [(1, 128), (5, 64)])
def test_queries_near_the_largest_bf16(octaves, T, D):
    """Query rows up to 2^120 against keys as small: ordinary scores."""
    c = Case(52, [T, 40, 300], 4, 2, D, T=T, power_of_two=True)
    c.q = W.f32_to_bf16_bits((O.bf16_bits_to_f64(c.q) * 2.0 ** octaves).astype(np.float32))
    c.k_scale = (c.k_scale * 2.0 ** -95).astype(np.float32)
    c.scale *= 2.0 ** (95 - octaves)
    check(attend(c), c)
