"""INT4 pages on the GPU against the fp64 oracle: writes and reads code for code, attention
within a bound derived from the roundings it makes."""
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
from gpu_util import bits, to_dev  # noqa: E402
from oracle import fp8 as F  # noqa: E402
from oracle import int4 as Q4  # noqa: E402
from oracle import oracle as O  # noqa: E402


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert pa.get_device_error() == 0, "device error word was set"


class Dev:
    def __init__(self, c):
        for name in ("q", "k", "v", "k_scale", "v_scale", "tables", "lens", "new_key",
                     "new_value", "slots"):
            setattr(self, name, to_dev(getattr(c, name)))
        self.c = c

    def attend(self, append=False, **kw):
        new = {"new_key": self.new_key, "new_value": self.new_value} if append else {}
        kw.setdefault("max_context_len", max(1, int(self.c.lens.max())))
        return pa.attention_int4(self.q, self.k, self.v, self.k_scale, self.v_scale, self.tables,
                                 self.lens, scale=self.c.scale, **new, **kw)


def bound(c, k, v, ref, mag, window):
    """Largest error the roundings allow.  Output: half a bf16 step, 2^-8 of it.  A weight is
    rounded to f16 (2^-11), times an E4M3 scale rounded again (2^-11); the codes enter as u = value
    / (scale head_scale) + 8 and the 8 is taken back with the weight times the scale unrounded,
    so the second rounding also counts for 8 scale head_scale: 2^-11 * 8 * sum_j p_j s_j.  The
    weights' sum is that of the rounded weights.  Scores err by fp32 accumulation, at most
    2^-20 of sum |q k|, and so does a weight (exp).  Below 2^-14 of a row's reference weight (the
    largest weight is at least 1) a rounding is 2^-25 absolute, before the scale and after it,
    times codes up to 15 and the head scale."""
    keys = [[c.rows(k, b, g, int(n), "k") for g in range(c.Hkv)] for b, n in enumerate(c.lens)]
    score = 2.0 ** -20 * c.score_size(keys)
    sc = Q4.unpack(v, c.D)[1]
    s_max = np.nanmax(F.decode(sc))
    small = int(c.lens.max()) * 2.0 ** -25 * 15 * (s_max + 1) * float(c.v_scale.max())
    # sum_j p_j s_j: attention over the values of code 9 (value = scale)
    nine = Q4.pack(np.full((*sc.shape[:-1], c.D), 9, dtype=np.uint8), sc)
    step, _ = Q4.attention(c.q, k, nine, c.k_scale, c.v_scale, c.tables, c.lens, c.scale, window)
    return (2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 2.0 ** -16 + score) * mag +
            2.0 ** -11 * 8 * step + small)


def check(out, c, k=None, v=None, window=0):
    k, v = c.k if k is None else k, c.v if v is None else v
    ref, mag = Q4.attention(c.q, k, v, c.k_scale, c.v_scale, c.tables, c.lens, c.scale, window)
    got = out.float().cpu().double().numpy()
    assert np.isfinite(got).all()
    over = np.abs(got - ref) - bound(c, k, v, ref, mag, window)
    assert over.max() <= 0, f"error exceeds its bound by {over.max():.3e}"
    return got, ref


# ------------------------------------------------------------------------------- pages
def special_rows(D):
    x = np.zeros((8, D), dtype=np.float32)
    x[1, 3], x[2, 5], x[3, 7], x[4, 31] = np.nan, np.inf, -np.inf, 1e30
    x[2:, 0] = 1.0
    x[5] = np.linspace(-7, 7, D)
    x[6] = 1e-30
    x[7, ::2] = -0.0
    return W.f32_to_bf16_bits(x)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
@pytest.mark.parametrize("n", [1, 5, 33, 300])
def test_store_is_exact_and_leaves_the_rest(D, Hkv, n):
    rng = np.random.default_rng(n * Hkv + D)
    NB = n // 16 + 4
    k, v = (rng.integers(0, 256, (NB, Hkv, Q4.page_bytes(D)), dtype=np.uint8) for _ in range(2))
    key, value = (W.f32_to_bf16_bits((rng.standard_normal((n, Hkv, D)) *
                                      np.exp2(rng.integers(-8, 8, (n, Hkv, 1)))
                                      ).astype(np.float32)) for _ in range(2))
    key[:min(n, 8), 0] = special_rows(D)[:min(n, 8)]
    value[:min(n, 8), -1] = special_rows(D)[:min(n, 8)]
    # coarse grids: many ties of the codes and of the scales
    value[n // 2:] = W.f32_to_bf16_bits((rng.integers(-64, 65, value[n // 2:].shape) / 8)
                                        .astype(np.float32))
    ks = rng.uniform(0.01, 1, Hkv).astype(np.float32)
    vs = np.exp2(rng.integers(-5, 1, Hkv)).astype(np.float32)
    slots = rng.permutation(NB * 16)[:n].astype(np.int64)
    slots[::7] = -1 if n > 1 else slots[0]
    dk, dv = to_dev(k), to_dev(v)
    pa.reshape_and_cache_int4(to_dev(key), to_dev(value), dk, dv, to_dev(slots), to_dev(ks),
                              to_dev(vs))
    rk, rv = Q4.reshape_and_cache(key, value, k, v, slots, ks, vs)
    np.testing.assert_array_equal(dk.cpu().numpy(), rk)
    np.testing.assert_array_equal(dv.cpu().numpy(), rv)

    gk, gv = pa.gather_cache_int4(dk, dv, to_dev(slots), to_dev(ks), to_dev(vs))
    for got, pool, s in ((gk, rk, ks), (gv, rv, vs)):
        got = got.float().cpu().double().numpy()
        codes, sc = Q4.unpack(pool, D)
        for i, slot in enumerate(slots):
            if slot < 0:
                assert (got[i] == 0).all()
                continue
            for h in range(Hkv):
                ref = Q4.dequantize(codes[slot // 16, h, slot % 16], sc[slot // 16, h, slot % 16],
                                    s[h])
                # the product of code, scale and head scale is rounded to fp32, then to bf16
                np.testing.assert_allclose(got[i, h], ref, rtol=2.0 ** -8 + 2.0 ** -22, atol=0)


def test_many_tokens_round_trip():
    """Enough tokens for the form that reads several per thread, not a multiple of them."""
    n, Hkv, D = 2503, 8, 128
    gen = torch.Generator("cuda").manual_seed(0)
    x = torch.randint(-7, 8, (2, n, Hkv, D), generator=gen, device="cuda").bfloat16()
    x[..., ::32] = 7                                        # every group reaches 7: scale 1
    NB = n // 16 + 2
    pools = [torch.zeros((NB, Hkv, pa.int4_page_bytes(D)), dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    one = torch.ones(Hkv, device="cuda")
    slots = torch.randperm(NB * 16, generator=gen, device="cuda")[:n]
    slots[::11] = -1
    pa.reshape_and_cache_int4(x[0], x[1], *pools, slots, one, one)
    live = (slots >= 0)[:, None, None]
    for got, want in zip(pa.gather_cache_int4(*pools, slots, one, one), x):
        assert torch.equal(got, torch.where(live, want, torch.zeros_like(want)))


def test_empty_calls():
    c = Case(0, [5], 2, 2, 64)
    d = Dev(c)
    z = d.new_key[:0]
    pa.reshape_and_cache_int4(z, z, d.k, d.v, d.slots[:0], d.k_scale, d.v_scale)
    k, v = pa.gather_cache_int4(d.k, d.v, d.slots[:0], d.k_scale, d.v_scale)
    assert k.shape == (0, 2, 64) and v.shape == (0, 2, 64)
    out = pa.attention_int4(d.q[:0], d.k, d.v, d.k_scale, d.v_scale, d.tables[:0], d.lens[:0], 5)
    assert out.shape == (0, 1, 2, 64)
    np.testing.assert_array_equal(d.k.cpu().numpy(), c.k)


def test_slots_outside_the_pool_are_reported():
    c = Case(1, [20], 2, 2, 64)
    d = Dev(c)
    slots = torch.tensor([c.NB * 16, 3, 2 ** 40], device="cuda")
    x = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    pa.reshape_and_cache_int4(x, x, d.k, d.v, slots, d.k_scale, d.v_scale)
    assert pa.get_device_error() == 5
    one = W.f32_to_bf16_bits(np.ones((1, 2, 64), dtype=np.float32))
    rk, _ = Q4.reshape_and_cache(one, one, c.k, c.v, [3], c.k_scale, c.v_scale)
    np.testing.assert_array_equal(d.k.cpu().numpy(), rk)
    k, _ = pa.gather_cache_int4(d.k, d.v, slots, d.k_scale, d.v_scale)
    assert pa.get_device_error() == 5
    assert (k[0] == 0).all() and (k[2] == 0).all() and (k[1] != 0).all()


# ------------------------------------------------------------------------------- attention
EDGE = [1, 2, 15, 16, 17, 31, 33, 64, 100, 257]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (5, 1), (16, 2), (24, 1)])
def test_decode_edge_lengths(D, Hq, Hkv):
    c = Case(D + Hq, EDGE, Hq, Hkv, D)
    check(Dev(c).attend(), c)


@pytest.mark.parametrize("T,Hq,Hkv", [(2, 4, 2), (3, 5, 1), (5, 8, 2), (5, 4, 1), (7, 8, 2),
                                      (16, 2, 1), (33, 1, 1), (64, 1, 1), (13, 4, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_verify_rows(T, Hq, Hkv, D):
    """Every tile layout: 4 to 64 query rows per kv head, odd counts, context of drafts alone."""
    c = Case(T + Hq + D, [T, T + 1, T + 15, T + 16, 130], Hq, Hkv, D, T=T)
    check(Dev(c).attend(), c)


@pytest.mark.parametrize("psize", [16, 32, 64, 0])
@pytest.mark.parametrize("T", [1, 3])
def test_partitions(psize, T):
    c = Case(psize + T, [3, 16, 17, 48, 300, 1100], 8, 2, 128, T=T)
    d = Dev(c)
    got, _ = check(d.attend(partition_size=psize), c)
    # without scratch the library takes whole sequences
    if psize == 0:
        small = torch.empty(0, dtype=torch.uint8, device="cuda")
        with pytest.raises(pa.PagedAttnError):
            d.attend(partition_size=16, workspace=small)


@pytest.mark.parametrize("window", [1, 3, 16, 17, 40, 1000])
@pytest.mark.parametrize("T,psize", [(1, 0), (5, 0), (1, 16), (5, 32)])
def test_window(window, T, psize):
    c = Case(window, [T, 16, 18, 47, 300], 4, 2, 64, T=T)
    check(Dev(c).attend(window_size=window, partition_size=psize), c, window=window)


@pytest.mark.parametrize("psize", [0, 32])
def test_nan_outside_every_window(psize):
    """NaN K and V in entries that no query token sees, inside a page that is read."""
    c = Case(21, [300, 55], 4, 2, 64, T=2)
    for name in ("k", "v"):
        codes, sc = Q4.unpack(getattr(c, name), 64)
        sc = np.array(sc, copy=True)
        for b, n in enumerate(c.lens):
            for j in range(n - 2 - 20 + 1):
                sc[c.tables[b, j // 16], :, j % 16] = 0x7F
        setattr(c, name, Q4.pack(codes, sc))
    got = Dev(c).attend(window_size=20, partition_size=psize)
    assert torch.isfinite(got.float()).all()
    d = Case(21, [300, 55], 4, 2, 64, T=2)
    check(got, d, window=20)


@pytest.mark.parametrize("T,D,psize", [(1, 64, 0), (1, 128, 16), (5, 128, 0), (18, 64, 32)])
def test_append_equals_store_then_attend(T, D, psize):
    c = Case(T + D, [T, T + 1, 40, 65, 200], 4, 2, D, T=T)
    one, two = Dev(c), Dev(c)
    a = one.attend(append=True, partition_size=psize)
    pa.reshape_and_cache_int4(two.new_key, two.new_value, two.k, two.v, two.slots, two.k_scale,
                              two.v_scale)
    b = two.attend(partition_size=psize)
    assert torch.equal(one.k, two.k) and torch.equal(one.v, two.v)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    rk, rv = Q4.reshape_and_cache(c.new_key, c.new_value, c.k, c.v, c.slots, c.k_scale, c.v_scale)
    np.testing.assert_array_equal(one.k.cpu().numpy(), rk)
    check(a, c, rk, rv)


@pytest.mark.parametrize("factor", [2.0 ** -90, 2.0 ** -20, 2.0 ** 6])
def test_query_magnitudes(factor):
    """Query rows of any size: tiny ones give uniform weights, large ones a single entry."""
    c = Case(11, [40, 100], 4, 2, 128)
    x = O.bf16_bits_to_f64(c.q)
    x[0, :, 1] *= 2.0 ** -10                      # rows of one tile differ in size
    c.q = W.f32_to_bf16_bits((x * factor).astype(np.float32))
    check(Dev(c).attend(), c)


def test_spread_of_value_scales():
    """V groups between the largest E4M3 scale and its subnormals; the largest ones late."""
    c = Case(12, [150, 33], 4, 2, 64, power_of_two=True)
    codes, sc = Q4.unpack(c.v, 64)
    sc = np.array(sc, copy=True)
    rng = np.random.default_rng(12)
    pick = rng.choice(np.array([1, 3, 8, 0x30, 0x7E], dtype=np.uint8), sc.shape)
    sc = np.where(sc == 0x7F, sc, pick)
    c.v = Q4.pack(codes, sc)
    x = O.bf16_bits_to_f64(c.q) * 4
    c.q = W.f32_to_bf16_bits(x.astype(np.float32))
    check(Dev(c).attend(), c)


def test_rising_scores_move_the_reference():
    """Keys that grow along the context: the running maximum moves at almost every page."""
    c = Case(13, [400], 4, 1, 64)
    codes, sc = Q4.unpack(c.k, 64)
    sc = np.array(sc, copy=True)
    q = O.bf16_bits_to_f64(c.q[0, 0, 0])
    for j in range(400):
        at = (c.tables[0, j // 16], 0, j % 16)
        codes[at] = np.where(q > 0, 15, 1)
        sc[at] = F.encode(np.array([j / 40.0 + 0.01]))[0]
    c.k = Q4.pack(codes, sc)
    c.q = np.broadcast_to(c.q[:, :, :1], c.q.shape).copy()
    check(Dev(c).attend(), c)


def test_bad_block_id_is_reported_and_skipped():
    c = Case(14, [100, 60], 4, 2, 64)
    d = Dev(c)
    good = d.attend()
    d.tables[0, 3] = c.NB
    out = d.attend()
    assert pa.get_device_error() == 5
    assert torch.equal(out[1], good[1]) and torch.isfinite(out.float()).all()
    d.tables[0, 3] = -1
    d.attend(append=True)
    assert pa.get_device_error() == 5


def test_bad_lengths_are_reported_and_skipped():
    c = Case(15, [100, 60, 33], 4, 2, 64, T=2)
    d = Dev(c)
    good = d.attend()
    d.lens[0], d.lens[2] = 101, 1                 # above the bound; below the query tokens
    out = torch.full_like(good, 7.0)
    before = d.k.clone()
    d.attend(out=out, append=True, max_context_len=100)
    assert pa.get_device_error() == 5
    assert (out[0] == 7).all() and (out[2] == 7).all()
    changed = (before != d.k).any(-1).any(-1).nonzero().flatten().tolist()
    assert set(changed) <= set(c.tables[1].tolist())


def test_outputs_of_one_call_do_not_depend_on_the_batch():
    c = Case(16, [500, 37, 64], 8, 2, 128)
    d = Dev(c)
    out = d.attend(partition_size=64, max_context_len=512 if c.mbs * 16 >= 512 else 500)
    for b in range(3):
        one = pa.attention_int4(d.q[b:b + 1], d.k, d.v, d.k_scale, d.v_scale,
                                d.tables[b:b + 1].contiguous(), d.lens[b:b + 1], 500,
                                c.scale, 64)
        assert torch.equal(one[0], out[b])


def reference(q, k, v, ks, vs, tables, lens, scale, window=0):
    """fp64 attention on the device, sequence by sequence, for sizes the host oracle is slow at:
    (out, bound) with the bound's terms as in bound()."""
    B, T, Hq, D = q.shape
    Hkv, J = k.shape[1], tables.shape[1] * 16
    table = torch.tensor(F.DECODE_TABLE, device=q.device)

    def rows(pool, s, ids, n):
        page = pool[ids.long()]                                     # [M, Hkv, bytes]
        code = page[..., :8 * D].unflatten(-1, (16, D // 2)).long()
        code = torch.stack([code & 15, code >> 4], -1).flatten(-2).double() - 8
        unit = table[page[..., 8 * D:].long()].unflatten(-1, (16, D // 32))
        unit = (unit * s.double()[:, None, None]).repeat_interleave(32, -1)
        x, u = ((y.transpose(0, 1).flatten(1, 2)[:, :n]) for y in (code * unit, unit))
        return x, u                                                 # [Hkv, n, D]

    out, tol = torch.zeros(q.shape, dtype=torch.float64, device=q.device), None
    tol = torch.zeros_like(out)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        K, _ = rows(k, ks, tables[b, :-(-n // 16)], n)
        V, U = rows(v, vs, tables[b, :-(-n // 16)], n)
        qq = q[b].double().view(T, Hkv, Hq // Hkv, D).permute(1, 0, 2, 3)
        s = torch.einsum("htgd,hjd->htgj", qq, K) * scale
        size = torch.einsum("htgd,hjd->htgj", qq.abs(), K.abs()).max() * scale * 1.4427
        j, last = torch.arange(n, device=q.device), n - T + torch.arange(T, device=q.device)
        see = j <= last[:, None]
        if window:
            see &= j > last[:, None] - window
        s = s.masked_fill(~see[None, :, None], -float("inf"))
        p = torch.softmax(s, -1)
        put = lambda x: x.permute(1, 0, 2, 3).reshape(T, Hq, D)     # noqa: E731
        out[b] = put(torch.einsum("htgj,hjd->htgd", p, V))
        mag = put(torch.einsum("htgj,hjd->htgd", p, V.abs()))
        step = put(torch.einsum("htgj,hjd->htgd", p, U))
        small = n * 2.0 ** -25 * 15 * float(U.max() + vs.max())
        tol[b] = (2.0 ** -8 * out[b].abs() + (2.0 ** -10 + 2.0 ** -16 + 2.0 ** -20 * size) * mag +
                  2.0 ** -11 * 8 * step + small)
    return out, tol


def random_cache(gen, B, lens, Hkv, D):
    need = [-(-n // 16) for n in lens]
    NB = sum(need) + 2
    ids = torch.randperm(NB, generator=gen, device="cuda").int()
    tables = torch.zeros((B, max(max(need), 1)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = ids[at:at + n]
        at += n
    scales = [torch.rand(Hkv, generator=gen, device="cuda") * 0.2 + 0.02 for _ in range(2)]
    pools = [torch.zeros((NB, Hkv, pa.int4_page_bytes(D)), dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    slots = torch.arange(NB * 16, device="cuda")
    x = [torch.randn((NB * 16, Hkv, D), generator=gen, device="cuda").bfloat16()
         for _ in range(2)]
    pa.reshape_and_cache_int4(*x, *pools, slots, *scales)
    return pools, scales, tables, torch.tensor(lens, dtype=torch.int32, device="cuda")


def against_reference(gen, lens, Hq, Hkv, D, T=1, window=0, **kw):
    B = len(lens)
    (k, v), (ks, vs), tables, dl = random_cache(gen, B, lens, Hkv, D)
    q = torch.randn((B, T, Hq, D), generator=gen, device="cuda").bfloat16()
    out = torch.full_like(q, 7.0)
    pa.attention_int4(q, k, v, ks, vs, tables, dl, max(max(lens), T), out=out, window_size=window,
                      **kw)
    ok = dl >= T
    ref, tol = reference(q, k, v, ks, vs, tables, torch.where(ok, dl, 0), D ** -0.5, window)
    over = (out.double() - ref).abs()[ok] - tol[ok]
    assert torch.isfinite(out.float()).all() and over.max() <= 0, f"by {over.max():.3e}"
    assert (out[~ok] == 7).all()                  # sequences out of range are left alone
    return out


@pytest.mark.parametrize("B,lo,hi", [(1, 20000, 20000), (2, 1, 9000), (33, 1, 400),
                                     (257, 1, 700), (300, 250, 300), (1030, 1, 300)])
@pytest.mark.parametrize("Hq,Hkv,D,T", [(8, 2, 128, 1), (6, 2, 64, 1), (8, 1, 128, 3)])
def test_balanced_runs(B, lo, hi, Hq, Hkv, D, T):
    """Batches around the chunks of lengths a warp holds, past the size up to which runs are
    balanced, one long sequence over all workers, and one long among short ones."""
    gen = torch.Generator("cuda").manual_seed(B + hi)
    lens = torch.randint(lo, hi + 1, (B,), generator=gen, device="cuda").tolist()
    lens[0], lens[-1] = max(T, lo), hi
    if B == 33:
        lens[17] = 12345
    lens = [max(T, n) for n in lens]
    against_reference(gen, lens, Hq, Hkv, D, T)


@pytest.mark.parametrize("window", [100, 700])
def test_balanced_window(window):
    gen = torch.Generator("cuda").manual_seed(window)
    against_reference(gen, [5, 90, 3000, 5000, 17, 2049], 8, 2, 128, T=2, window=window)


def test_balanced_runs_skip_sequences_out_of_range():
    """Lengths below the query tokens (an idle row of a batch) take no part."""
    gen = torch.Generator("cuda").manual_seed(5)
    against_reference(gen, [0, 900, 1, 0, 2, 400, 0], 8, 2, 64, T=2)
    assert pa.get_device_error() == 5
    # nothing at all to do
    against_reference(gen, [0, 1, 0, 300], 8, 2, 64, T=2)
    assert pa.get_device_error() == 5


def test_two_calls_at_once():
    """Two streams, a workspace each: overlapping calls do not disturb one another."""
    gen = torch.Generator("cuda").manual_seed(6)
    lens = torch.randint(300, 3000, (16,), generator=gen, device="cuda").tolist()
    (k, v), (ks, vs), tables, dl = random_cache(gen, 16, lens, 4, 128)
    qs = [torch.randn((16, 1, 16, 128), generator=gen, device="cuda").bfloat16()
          for _ in range(2)]
    mcl = max(lens)
    want = [pa.attention_int4(q, k, v, ks, vs, tables, dl, mcl) for q in qs]
    need = pa.int4_workspace_size(16, 16, 4, 1, mcl, 128)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                pa.attention_int4(qs[i], k, v, ks, vs, tables, dl, mcl, workspace=ws[i],
                                  out=outs[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_three_dim_query_and_out():
    c = Case(17, [9, 50], 4, 2, 64)
    d = Dev(c)
    ref = d.attend()
    q = d.q.squeeze(1)
    out = torch.empty_like(q)
    got = pa.attention_int4(q, d.k, d.v, d.k_scale, d.v_scale, d.tables, d.lens, 50, c.scale,
                            out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, ref.squeeze(1))
    # no bound given: the library reads the lengths
    assert torch.equal(pa.attention_int4(q, d.k, d.v, d.k_scale, d.v_scale, d.tables, d.lens,
                                         scale=c.scale), got)


def test_graphs_and_streams():
    """Two captured graphs with a workspace each, replayed in turn and on another stream."""
    c = Case(18, [700, 90], 8, 2, 128)
    d = Dev(c)
    want = d.attend(partition_size=64, append=True).clone()
    need = pa.int4_workspace_size(2, 8, 2, 1, 700, 128, 64)
    graphs = []
    for _ in range(2):
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(d.q)
        d.attend(partition_size=64, append=True, workspace=ws, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            d.attend(partition_size=64, append=True, workspace=ws, out=out)
        graphs.append((g, out, ws))
    side = torch.cuda.Stream()
    for _ in range(3):
        for g, out, _ in graphs:
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for _, out, _ in graphs)
        with torch.cuda.stream(side):
            for g, out, _ in graphs:
                out.zero_()
                g.replay()
            eager = d.attend(partition_size=64)
        side.synchronize()
        assert all(torch.equal(out, want) for _, out, _ in graphs) and torch.equal(eager, want)


def test_offsets_past_32_bits():
    """Pages at the end of pools of more than 2^32 bytes."""
    c = Case(19, [200, 77], 4, 2, 128)
    d = Dev(c)
    want = d.attend()
    NB = (2 ** 32 // (2 * 1088)) + 4096
    k = torch.zeros((NB, 2, 1088), dtype=torch.uint8, device="cuda")
    v = torch.zeros((NB, 2, 1088), dtype=torch.uint8, device="cuda")
    k[NB - c.NB:], v[NB - c.NB:] = d.k, d.v
    d.k, d.v, d.tables = k, v, d.tables + (NB - c.NB)
    assert torch.equal(d.attend(), want)
    slots = d.slots + (NB - c.NB) * 16
    pa.reshape_and_cache_int4(d.new_key, d.new_value, k, v, slots, d.k_scale, d.v_scale)
    got, _ = pa.gather_cache_int4(k, v, slots, d.k_scale, d.v_scale)
    x = O.bf16_bits_to_f64(c.new_key[:, 0])
    codes, sc = Q4.quantize(c.new_key[:, 0], c.k_scale[0])
    ref = Q4.dequantize(codes, sc, c.k_scale[0])
    np.testing.assert_allclose(got[:, 0].float().cpu().numpy(), ref, rtol=2.0 ** -8 + 2.0 ** -22)
    assert np.abs(ref - x).max() < 0.5


def test_binding_refusals():
    c = Case(20, [9], 4, 2, 64)
    d = Dev(c)
    with pytest.raises(ValueError, match="INT4 pools"):
        pa.attention_int4(d.q, d.k[..., :500].contiguous(), d.v[..., :500].contiguous(),
                          d.k_scale, d.v_scale, d.tables, d.lens, 9)
    with pytest.raises(ValueError):
        pa.attention_int4(d.q[..., :32].contiguous(), d.k, d.v, d.k_scale, d.v_scale, d.tables,
                          d.lens, 9)
    with pytest.raises(TypeError):
        pa.attention_int4(d.q.half(), d.k, d.v, d.k_scale, d.v_scale, d.tables, d.lens, 9)
    with pytest.raises(ValueError, match="contiguous"):
        pa.attention_int4(torch.cat([d.q, d.q], -1)[..., ::2], d.k, d.v, d.k_scale, d.v_scale,
                          d.tables, d.lens, 9)
    with pytest.raises(ValueError, match="together"):
        d.attend(new_key=d.new_key)
    with pytest.raises(ValueError):
        pa.reshape_and_cache_int4(d.new_key, d.new_value, d.k, d.v, d.slots, d.k_scale[:1],
                                  d.v_scale)
    assert bits(d.q).shape == c.q.shape
