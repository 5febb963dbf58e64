"""NaN and infinity among live keys and queries: a query row whose softmax is NaN gives NaN to
every entry that it sees and nothing to the others."""
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
from oracle import bounded as BD  # noqa: E402
from oracle import int4 as Q4  # noqa: E402
from oracle import oracle as O  # noqa: E402


def spoil_key(c, b, j, g, value):
    """Key j of (sequence b, kv head g) becomes NaN, or holds `value` in dim 0 (bf16 pages)."""
    at = (c.tables[b, j // 16], g, j % 16)
    if c.fmt == "bf16":
        c.k[at][0] = W.f32_to_bf16_bits(np.array([value], dtype=np.float32))[0]
    elif c.fmt == "fp8":
        c.k[at] = 0x7F
    else:
        codes, sc = Q4.unpack(c.k, c.D)
        sc = np.array(sc, copy=True)
        sc[at] = 0x7F
        c.k = Q4.pack(codes, sc)


def check(c, decay=0.5):
    rng = np.random.default_rng(0)
    w0 = rng.exponential(1.0, (len(c.lens), c.Hkv, int(c.lens.max()) + 3)).astype(np.float32)
    w = to_dev(w0)
    pa.accumulate_weights(to_dev(c.q), to_dev(c.k), to_dev(c.tables), to_dev(c.lens), w,
                          max_context_len=int(c.lens.max()), scale=c.scale, decay=decay,
                          k_scale=None if c.fmt == "bf16" else to_dev(c.k_scale))
    keys = [[c.rows(c.k, b, g, int(n), "k") for g in range(c.Hkv)]
            for b, n in enumerate(c.lens)]
    with np.errstate(invalid="ignore"):
        ref, _, gained = BD.accumulate(w0.astype(float), np.zeros(w0.shape, int), c.q, keys,
                                       c.lens, c.lens, c.scale, decay)
    got = w.cpu().double().numpy()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    # finite rows: scores of N(0, 1) values err by 2^-20 of sum |q k| (below 2^7 in log2 units for
    # 64 dims), ex2 and the sums by 2^-19
    tol = (2.0 ** -13 + 2.0 ** -19) * np.abs(gained) + 2.0 ** -23 * np.abs(ref) + 1e-37
    assert (np.abs(got - ref)[ok] <= tol[ok]).all()
    assert pa.get_device_error() == 0
    return ref


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("T,j", [(1, 0), (1, 299), (1, 1200), (4, 1000), (4, 1299)])
def test_nan_key(fmt, T, j):
    """In an early, a middle and the newest page; the last draft's own key."""
    c = Case(31, [1300, 40, 700], 6, 2, 64, T=T, fmt=fmt)
    spoil_key(c, 0, j, 1, np.nan)
    ref = check(c)
    assert np.isnan(ref[0, 1, :j + 1]).all() and np.isfinite(ref[0, 0]).all()
    assert np.isfinite(ref[1:]).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int4"])
def test_nan_query(fmt):
    """The first draft's row: the drafts behind it are not seen by it."""
    c = Case(32, [300, 40, 3], 6, 2, 64, T=3, fmt=fmt)
    c.q[0, 0, 1, 5] = c.q[2, 1, 4, 0] = 0x7FC0
    ref = check(c)
    assert np.isnan(ref[0, 0, :298]).all() and np.isfinite(ref[0, 0, 298:]).all()
    assert np.isnan(ref[2, 1, :2]).all() and np.isfinite(ref[2, 1, 2])


@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_key(sign):
    """A score of +inf makes its row NaN; one of -inf is a weight of zero."""
    c = Case(33, [500, 90], 4, 2, 64, T=2, fmt="bf16")
    q = np.abs(O.bf16_bits_to_f64(c.q).astype(np.float32))
    q[..., 0] = sign * (q[..., 0] + 0.5)
    c.q = W.f32_to_bf16_bits(q)
    spoil_key(c, 0, 77, 0, np.inf)
    with np.errstate(invalid="ignore"):
        ref = check(c)
    assert np.isnan(ref).any() == (sign > 0)


def test_every_seen_score_minus_infinity():
    """No finite score in a row: its softmax is NaN."""
    c = Case(34, [2, 35], 2, 1, 64, T=2, fmt="bf16")
    q = np.abs(O.bf16_bits_to_f64(c.q).astype(np.float32))
    q[..., 0] += 0.5
    c.q = W.f32_to_bf16_bits(q)
    spoil_key(c, 0, 0, 0, -np.inf)                  # row 0 sees entry 0 alone
    ref = check(c)
    assert np.isnan(ref[0, 0, 0]) and np.isfinite(ref[0, 0, 1])


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_bad_block_beside_a_nan_key(fmt):
    """Entries of a block outside the pool are skipped, even by a row that is NaN."""
    c = Case(35, [100], 2, 1, 64, fmt=fmt)
    spoil_key(c, 0, 5, 0, np.nan)
    c.tables[0, 2] = c.NB + 4
    w = torch.ones((1, 1, 112), device="cuda")
    pa.accumulate_weights(to_dev(c.q), to_dev(c.k), to_dev(c.tables), to_dev(c.lens), w,
                          max_context_len=100, scale=c.scale,
                          k_scale=None if fmt == "bf16" else to_dev(c.k_scale))
    assert pa.get_device_error() == 5
    x = w[0, 0].cpu()
    assert (x[32:48] == 1).all() and (x[100:] == 1).all()
    assert torch.isnan(x[:32]).all() and torch.isnan(x[48:100]).all()


@pytest.mark.parametrize("fmt", ["fp8", "int4"])
@pytest.mark.parametrize("octaves", [98, 118])
def test_queries_near_the_largest_bf16(fmt, octaves):
    """Query rows up to 2^120 against keys as small: ordinary scores."""
    c = Case(36, [300, 40, 3], 6, 2, 64, T=3, fmt=fmt, power_of_two=True)
    c.q = W.f32_to_bf16_bits((O.bf16_bits_to_f64(c.q) * 2.0 ** octaves).astype(np.float32))
    c.k_scale = (c.k_scale * 2.0 ** -95).astype(np.float32)
    c.scale *= 2.0 ** (95 - octaves)
    assert np.isfinite(check(c)).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("octaves", [26, 60, 80])
def test_scores_past_what_fp32_resolves(fmt, octaves):
    """Scores so large that their rounding is octaves: the largest one takes all the weight."""
    c = Case(37, [300, 40, 2000], 4, 2, 64, fmt=fmt)
    c.q = W.f32_to_bf16_bits((O.bf16_bits_to_f64(c.q) * 2.0 ** octaves).astype(np.float32))
    w = torch.zeros((3, 2, 2000), device="cuda")
    pa.accumulate_weights(to_dev(c.q), to_dev(c.k), to_dev(c.tables), to_dev(c.lens), w,
                          max_context_len=2000, scale=c.scale,
                          k_scale=None if fmt == "bf16" else to_dev(c.k_scale))
    assert pa.get_device_error() == 0
    for b, n in enumerate(c.lens):
        for g in range(2):
            K = c.rows(c.k, b, g, int(n), "k")
            ref = np.zeros(2000)
            for h in (2 * g, 2 * g + 1):
                x = O.bf16_bits_to_f64(c.q[b, 0, h])
                s, size = K @ x, (np.abs(K) @ np.abs(x)).max()
                top = np.sort(s)[-2:]
                # a score errs by 2^-20 of sum |q k|; the second one is over 100 octaves down
                assert top[1] - top[0] > 2.0 ** -18 * size and size > 20 * 2.0 ** octaves
                ref[np.argmax(s)] += 1.0
            np.testing.assert_array_equal(w[b, g].cpu().numpy(), ref)
