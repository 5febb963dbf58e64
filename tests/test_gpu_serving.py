"""Batches served on the device from prompts to scored drafts: block tables and slots, copies,
stores, attention and log probabilities of one step after another."""
import random

import numpy as np
import pytest
import torch

import paged_kv_cache_221_gb300 as pa
from prompt_cases import check
from step_cases import Batch
from test_gpu_score import run as score

pytestmark = pytest.mark.gpu
HQ, HKV, D, V = 8, 2, 128, 1000


class Server:
    """One layer over a paged cache, beside the K and V rows of every sequence."""

    def __init__(self, batch, fp8, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*shape):
            return torch.randn(shape, generator=g, device="cuda")
        self.batch, self.fp8 = batch, fp8
        self.embed, self.head = rand(V, HQ + 2 * HKV, D).bfloat16(), rand(V, HQ * D) / 16
        kind = dict(dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
        self.k = torch.full((batch.NB, HKV, 16, D), 255 if fp8 else float("nan"), **kind)
        self.v = torch.full((batch.NB, HKV, D, 16) if fp8 else self.k.shape,
                            255 if fp8 else float("nan"), **kind)
        self.scales = (dict(k_scale=torch.tensor([0.01, 0.02], device="cuda"),
                            v_scale=torch.tensor([0.02, 0.01], device="cuda")) if fp8 else {})
        self.rows = {}                          # by sequence: (K, V) in 64 bits, [Hkv, n, D]

    def store(self, key, value, slots, copies):
        if self.fp8:                            # the bytes of a page, as bf16 words
            flat = [x.view(torch.bfloat16).view(-1, HKV, 16, D // 2) for x in (self.k, self.v)]
            pa.copy_blocks(*flat, copies)
            pa.reshape_and_cache_fp8(key, value, self.k, self.v, slots, **self.scales)
        else:
            pa.copy_blocks(self.k, self.v, copies)
            pa.reshape_and_cache(key, value, self.k, self.v, slots)

    def layer(self, state, tokens, new, total, most):
        """Everything that runs on the device; takes no length from it."""
        starts, slots, positions, copies = pa.extend_sequences(*state, new, total)
        x = self.embed[tokens]
        q, key, value = (t.contiguous() for t in x.split([HQ, HKV, HKV], 1))
        self.store(key, value, slots, copies)
        out = pa.prompt_attention(q, self.k, self.v, state[0], state[1], starts, most,
                                  out=torch.zeros_like(q), **self.scales)
        return starts, slots, positions, copies, q, key, value, out

    def stored(self, slots):
        ids, at = slots // 16, slots % 16
        if not self.fp8:
            return self.k[ids, :, at].double(), self.v[ids, :, at].double()
        k, v = (x.view(torch.float8_e4m3fn).double() for x in (self.k, self.v))
        s = [self.scales[n].double()[:, None] for n in ("k_scale", "v_scale")]
        return k[ids, :, at] * s[0], v[ids, :, :, at] * s[1]

    def verify(self, state, new, total, got):
        """A step's results against the oracle's tables and every sequence's own rows."""
        starts, slots, positions, copies, q, key, value, out = got
        assert pa.get_device_error() == 0
        for a, b in zip(got[:4], self.batch.extend(new, total)):
            assert np.array_equal(a.cpu().numpy(), b)
        for a, b in zip(state, self.batch.arrays()):
            assert np.array_equal(a.cpu().numpy(), b)
        used = sum(new)
        for mine, given in zip(self.stored(slots[:used]), (key, value)):
            given = given[:used].double()
            # E4M3: half a step of 2^-3, or of 2^-9 scales below the normal numbers
            assert ((mine - given).abs() <= (given.abs() * 2.0 ** -4 + 2.0 ** -10 * 0.02
                                             if self.fp8 else 0.0)).all()
        want, size = (torch.zeros_like(out, dtype=torch.float64) for _ in range(2))
        at = 0
        for b, n in zip(self.batch.ids, new):
            k, v = self.stored(slots[at:at + n])
            old = self.rows.get(b, (k[:0], v[:0]))
            k, v = self.rows[b] = (torch.cat((old[0], k)), torch.cat((old[1], v)))
            L = len(k)
            s = torch.einsum("nhd,lhd->hnl", q[at:at + n].double(),
                             k.repeat_interleave(HQ // HKV, 1)) * D ** -0.5
            s += torch.ones(n, L, device="cuda").triu(L - n + 1).double() * -1e9
            w = s.softmax(-1)
            vv = v.repeat_interleave(HQ // HKV, 1)
            want[at:at + n] = torch.einsum("hnl,lhd->nhd", w, vv)
            size[at:at + n] = torch.einsum("hnl,lhd->nhd", w, vv.abs())
            at += n
        check(out, want, size)

    def step(self, state, r, new, spare=0):
        total = sum(new) + spare
        tokens = torch.tensor([r.randrange(V) for _ in range(total)], device="cuda")
        got = self.layer(state, tokens, torch.tensor(new, dtype=torch.int32, device="cuda"), total,
                         self.batch.mbs * 16)
        self.verify(state, new, total, got)
        # the model's log probability of every token that follows
        logits = got[-1].flatten(1).float() @ self.head.t()
        score(logits, torch.cat((tokens[1:], tokens[:1] * 0 - 1)).int(), 5)

    def keep(self, state, lens):
        pa.truncate_sequences(*state, torch.tensor(lens, dtype=torch.int32, device="cuda"))
        assert pa.get_device_error() == 0
        self.batch.truncate(lens)
        self.rows = {b: (k[:n], v[:n]) for (b, (k, v)), n in zip(sorted(self.rows.items()), lens)}
        for a, b in zip(state, self.batch.arrays()):
            assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("fp8", [False, True])
def test_prompts_forks_and_drafts(fp8):
    r = random.Random(1 + fp8)
    batch = Batch(200, 30)
    for _ in range(6):
        batch.add(0)
    s = Server(batch, fp8)
    state = batch.upload()
    s.step(state, r, [37, 1, 128, 0, 300, 16], 3)                 # prompts
    s.step(state, r, [20, 0, 1, 5, 40, 16])                       # a chunk behind them
    for parent in (0, 0, 4):                                      # samples of the same prompt
        batch.fork(parent)
        s.rows[len(batch.ids) - 1] = s.rows[parent]
    state = batch.upload()
    for _ in range(4):                                            # drafts, some of them rejected
        before = [batch.m.tokens[b] for b in batch.ids]
        s.step(state, r, [5] * 9)
        s.keep(state, [n + r.randint(1, 5) for n in before])
    s.keep(state, [0] * 8 + [batch.m.tokens[8]])                  # all but one have finished
    s.step(state, r, [60, 1, 0, 0, 0, 0, 0, 0, 1])


@pytest.mark.parametrize("fp8", [False, True])
def test_steps_replayed_from_a_graph(fp8):
    """One captured step serves batches whose lengths are known to the device alone."""
    r = random.Random(5)
    batch = Batch(150, 20)
    for n in range(5):
        batch.add(0)
    batch.fork(4)
    s = Server(batch, fp8, 7)
    state, total = batch.upload(), 40
    tokens = torch.zeros(total, dtype=torch.long, device="cuda")
    new = torch.zeros(6, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.layer(state, tokens, new, total, batch.mbs * 16)        # nothing is taken in
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.layer(state, tokens, new, total, batch.mbs * 16)
    for lens in ([7, 0, 1, 16, 8, 8], [1] * 6, [0] * 6, [30, 0, 0, 0, 5, 5], [6, 7, 8, 9, 10, 0]):
        tokens.copy_(torch.tensor([r.randrange(V) for _ in range(total)]))
        new.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        s.verify(state, lens, total, got)
