"""Accumulated attention weights of batches whose runs hold many whole jobs: every
(sequence, kv head) is normalised by its own maximum and sum, in every page format."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():          # collected on CPU-only hosts, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import __graft_entry__  # noqa: E402

__graft_entry__.build()

import paged_kv_cache_221_gb300 as pa  # noqa: E402
from oracle import fp8 as F  # noqa: E402


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert pa.get_device_error() == 0, "device error word was set"


def log_spread(n, lo, hi):
    return [round(lo * (hi / lo) ** (i / (n - 1))) for i in range(n)]


def spread(n, lo, hi):
    return [round(lo + (hi - lo) * i / (n - 1)) for i in range(n)]


# Lengths whose list gives every warp a run of several short sequences' heads.
BATCHES = {
    "512 of 64": [64] * 512,
    "64 of 1-4096": spread(64, 1, 4096),
    "256 of 128-8192": log_spread(256, 128, 8192),
    "short behind long": [6000] * 12 + [1, 17, 40] * 100 + [5000, 3],
}


def cache(gen, fmt, lens, Hkv, D):
    """(K pool, k_scale or None, tables, lens, fp64 keys of a sequence and its kv heads)."""
    need = [-(-n // 16) for n in lens]
    NB = sum(need) + 1
    ids = torch.randperm(NB, generator=gen, device="cuda").int()
    tables = torch.zeros((len(lens), max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = ids[at:at + n]
        at += n
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x = torch.randn((NB * 16, Hkv, D), generator=gen, device="cuda").bfloat16()
    scale = torch.rand(Hkv, generator=gen, device="cuda") * 0.2 + 0.02
    slots = torch.arange(NB * 16, device="cuda")
    table = torch.tensor(F.DECODE_TABLE, device="cuda")
    if fmt == "bf16":
        k = x.view(NB, 16, Hkv, D).transpose(1, 2).contiguous()
        page = lambda i: k[i].double()                                      # noqa: E731
        scale = None
    elif fmt == "fp8":
        k = torch.zeros((NB, Hkv, 16, D), dtype=torch.uint8, device="cuda")
        v = torch.zeros((NB, Hkv, D, 16), dtype=torch.uint8, device="cuda")
        pa.reshape_and_cache_fp8(x, x, k, v, slots, scale, scale)
        page = lambda i: table[k[i].long()] * scale.double()[:, None, None]  # noqa: E731
    else:
        k = torch.zeros((NB, Hkv, pa.int4_page_bytes(D)), dtype=torch.uint8, device="cuda")
        pa.reshape_and_cache_int4(x, x, k, k.clone(), slots, scale, scale)

        def page(i):
            code = k[i][..., :8 * D].unflatten(-1, (16, D // 2)).long()
            code = torch.stack([code & 15, code >> 4], -1).flatten(-2).double() - 8
            unit = table[k[i][..., 8 * D:].long()].unflatten(-1, (16, D // 32))
            return code * (unit * scale.double()[:, None, None]).repeat_interleave(32, -1)

    def keys(b):
        n = lens[b]
        return page(tables[b, :need[b]].long()).transpose(0, 1).flatten(1, 2)[:, :n]
    return k, scale, tables, dl, keys


def check(fmt, lens, Hq, Hkv, D, T):
    gen = torch.Generator("cuda").manual_seed(len(lens) + Hq + T)
    lens = [max(T, n) for n in lens]
    k, scale, tables, dl, keys = cache(gen, fmt, lens, Hkv, D)
    B, hi = len(lens), max(lens)
    q = torch.randn((B, T, Hq, D), generator=gen, device="cuda").bfloat16()
    w = torch.full((B, Hkv, hi), 3.0, device="cuda")
    pa.accumulate_weights(q, k, tables, dl, w, max_context_len=hi, decay=0.0, k_scale=scale)
    wrong = []
    for b, n in enumerate(lens):
        K = keys(b)
        x = q[b].double().view(T, Hkv, Hq // Hkv, D).permute(1, 0, 2, 3)
        s = torch.einsum("htgd,hjd->htgj", x, K) * D ** -0.5
        size = torch.einsum("htgd,hjd->htgj", x.abs(), K.abs()).max() * D ** -0.5 * 1.4427
        last = n - T + torch.arange(T, device="cuda")
        see = torch.arange(n, device="cuda") <= last[:, None]
        p = torch.softmax(s.masked_fill(~see[None, :, None], -float("inf")), -1)
        ref = p.sum((1, 2))
        # scores err by 2^-20 of sum |q k| (log2 domain), ex2 and the sums by 2^-19 together
        tol = (2.0 ** -20 * size + 2.0 ** -19) * ref + 1e-37
        over = ((w[b, :, :n].double() - ref).abs() <= tol).all(-1)
        wrong += [(b, g) for g in range(Hkv) if not over[g]]
        assert (w[b, :, n:] == 3).all()
    assert not wrong, f"{len(wrong)} of {B * Hkv} (sequence, kv head) pairs, first {wrong[:4]}"


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("batch", BATCHES)
def test_whole_jobs_in_one_run(fmt, batch):
    check(fmt, BATCHES[batch], 16, 8, 64, 1)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("group,T", [(4, 3), (3, 7), (5, 6), (8, 5), (1, 64)])
def test_whole_jobs_in_one_run_every_tile(fmt, group, T):
    """12 to 64 query rows per kv head, both row columns among them."""
    check(fmt, BATCHES["512 of 64"], 4 * group, 4, 128, T)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_whole_and_cut_jobs_of_two_row_columns(fmt):
    check(fmt, BATCHES["short behind long"], 8, 1, 128, 5)
