"""Packed prompts over random paged caches, and their attention in 64 bits."""
import numpy as np
import torch

BLOCK = 16


class Prompts:
    """Sequences with ``new`` query tokens behind ``cached`` ones each, on the GPU.

    Slots that hold no token, blocks of no sequence and the rows of q behind the last sequence
    hold NaN.
    """

    def __init__(self, seed, new, cached, Hq, Hkv, D, fp8=False, behind=0, extra_blocks=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.new, self.cached = list(new), list(cached)
        self.lens = [a + b for a, b in zip(new, cached)]
        self.Hq, self.Hkv, self.D, self.fp8 = Hq, Hkv, D, fp8
        need = [-(-n // BLOCK) for n in self.lens]
        self.mbs = max(max(need, default=0), 1) + extra_blocks
        self.NB = sum(need) + 3
        ids = torch.randperm(self.NB, generator=g, device="cuda").int()
        # entries behind a sequence's blocks name no block
        self.tables = torch.full((len(new), self.mbs), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = ids[at:at + n]
            at += n
        self.N = sum(new) + behind
        self.q = torch.randn((self.N, Hq, D), generator=g, device="cuda").bfloat16()
        self.q[sum(new):] = float("nan")
        self.starts = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
        self.ctx = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.most = max(1, max(self.lens, default=1))
        self.k_scale = self.v_scale = None
        used = torch.zeros((self.NB, BLOCK), dtype=torch.bool, device="cuda")
        for b, n in enumerate(self.lens):
            j = torch.arange(n, device="cuda")
            used[self.tables[b, j // BLOCK].long(), j % BLOCK] = True
        pools = []
        for i in range(2):
            x = torch.randn((self.NB, Hkv, BLOCK, D), generator=g, device="cuda")
            if fp8:
                s = torch.rand(Hkv, generator=g, device="cuda") / 96 + 1 / 96
                x = (x / s[:, None, None]).clamp(-448, 448)
                x.transpose(1, 2)[~used] = float("nan")
                x = x.to(torch.float8_e4m3fn).view(torch.uint8)
                x = x.transpose(-1, -2).contiguous() if i else x
                if i:
                    self.v_scale = s
                else:
                    self.k_scale = s
            else:
                x = x.bfloat16()
                x.transpose(1, 2)[~used] = float("nan")
            pools.append(x)
        self.k, self.v = pools

    def kv(self, b):
        """K and V of sequence b in 64 bits, [Hkv, L, D]."""
        ids = self.tables[b, :-(-self.lens[b] // BLOCK)].long()
        out = []
        for i, (pool, scale) in enumerate(((self.k, self.k_scale), (self.v, self.v_scale))):
            x = pool[ids]
            if self.fp8:
                x = x.view(torch.float8_e4m3fn).double() * scale.double()[:, None, None]
                x = x.transpose(-1, -2) if i else x
            out.append(x.double().transpose(0, 1).flatten(1, 2)[:, :self.lens[b]])
        return out

    def exact(self, scale=None, window=0):
        """(outputs, sums of weight times |value|), [N, Hq, D] in 64 bits; rows of no sequence
        are zero.  A key that a query token must not see has no part in it, whatever it holds."""
        scale = self.D ** -0.5 if scale is None else scale
        out = torch.zeros((self.N, self.Hq, self.D), dtype=torch.float64, device="cuda")
        size = torch.zeros_like(out)
        G, row = self.Hq // self.Hkv, 0
        for b, (n, L) in enumerate(zip(self.new, self.lens)):
            if n == 0:
                continue
            k, v = (x.repeat_interleave(G, 0) for x in self.kv(b))
            q = self.q[row:row + n].double().transpose(0, 1)              # [Hq, n, D]
            pos = torch.arange(L - n, L, device="cuda")[:, None]
            j = torch.arange(L, device="cuda")
            see = j <= pos
            if window:
                see &= j > pos - window
            s = (q @ k.transpose(1, 2) * scale).masked_fill(~see, -float("inf"))
            w = torch.softmax(s, -1)
            if bool(torch.isfinite(v).all()):
                o = w @ v
            else:                                                          # 0 * inf is NaN
                o = torch.where(see[None, :, :, None], w[..., None] * v[:, None], 0.0).sum(2)
            out[row:row + n] = o.transpose(0, 1)
            size[row:row + n] = (w @ v.abs().nan_to_num(0.0, 0.0, 0.0)).transpose(0, 1)
            row += n
        return out, size


def bound(out, size):
    """A weight and the output are rounded to bf16 once each, 2^-8 of the value at most; what
    fp32 arithmetic adds (scores, exponentials, sums) stays below a sixteenth of that."""
    return 2.0 ** -8 * (size + out.abs()) * (1 + 2.0 ** -4) + 1e-30


def check(got, out, size, rows=None):
    got = got.double()
    if rows is not None:
        got, out, size = got[rows], out[rows], size[rows]
    fine = torch.isfinite(out)
    assert torch.equal(torch.isnan(got), torch.isnan(out))
    odd = ~fine & ~torch.isnan(out)
    assert torch.equal(got[odd], out[odd])
    over = (got - out).abs()[fine] - bound(out, size)[fine]
    assert over.numel() == 0 or over.max() <= 0, f"over the bound by {over.max().item():.3e}"
