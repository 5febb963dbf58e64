"""Cases of the operators that take whole prompts through the paged cache.

Three kinds of case:

prompt   causal attention of packed prompts of different lengths over their pages; each
         sequence's query tokens are the newest positions of its context, so that a prompt can
         continue a cached prefix
step     the block tables, reference counts, lengths, slots and positions of a batch extended by
         each request's new tokens, and for drafts cut back to the accepted ones
score    the log probabilities of given tokens with the entropy and the most probable
         alternatives of every row of logits

With `own` false `run` is the plain form in elementary torch operations; with `own` true it
calls the package.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # two short prompts, 4 kv heads of 64 dims: nothing but latency
        {"name": "prompt_tiny", "op": "prompt", "batch": 2, "q_heads": 4, "kv_heads": 4, "dim": 64,
         "cached_lo": 0, "cached_hi": 0, "lo": 37, "hi": 100, "window": 0, "pages": "bf16"},
        # the prompts that arrive together at a serving batch, 128 to 2048 tokens each
        {"name": "prompt_batch", "op": "prompt", "batch": 24, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "cached_lo": 0, "cached_hi": 0, "lo": 128, "hi": 2048, "window": 0,
         "pages": "bf16"},
        # one long document
        {"name": "prompt_long", "op": "prompt", "batch": 1, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "cached_lo": 0, "cached_hi": 0, "lo": 16384, "hi": 16384, "window": 0,
         "pages": "bf16"},
        # the next 512 tokens of prompts that are taken in chunks, eight query heads per kv head
        {"name": "prompt_chunk", "op": "prompt", "batch": 4, "q_heads": 64, "kv_heads": 8,
         "dim": 128, "cached_lo": 4096, "cached_hi": 32000, "lo": 512, "hi": 512, "window": 0,
         "pages": "bf16"},
        # a short question about a long cached document
        {"name": "prompt_question", "op": "prompt", "batch": 1, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "cached_lo": 65519, "cached_hi": 65519, "lo": 33, "hi": 33, "window": 0,
         "pages": "bf16"},
        # layers that look at the last thousand tokens only
        {"name": "prompt_window", "op": "prompt", "batch": 4, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "cached_lo": 0, "cached_hi": 0, "lo": 4001, "hi": 8191, "window": 1000,
         "pages": "bf16"},
        # prompts into an 8-bit cache
        {"name": "prompt_fp8", "op": "prompt", "batch": 12, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "cached_lo": 0, "cached_hi": 0, "lo": 512, "hi": 4096, "window": 0,
         "pages": "fp8"},
        # five drafts per sequence taken in and the rejected ones given back, every verify step
        {"name": "step_drafts", "op": "step", "batch": 256, "lo": 128, "hi": 8192, "new_lo": 5,
         "new_hi": 5, "forked": 16, "blocks": 90000, "mbs": 520, "spare": 0, "reject": True},
        # a burst of prompts, some of them over forked prefixes, into a large pool
        {"name": "step_prompts", "op": "step", "batch": 512, "lo": 0, "hi": 2000, "new_lo": 1,
         "new_hi": 1000, "forked": 40, "blocks": 262144, "mbs": 200, "spare": 1000,
         "reject": False},
        # the logits of one decode step, a tenth of them masked
        {"name": "score_step", "op": "score", "rows": 64, "vocab": 128256, "type": "fp32", "top": 5,
         "masked": True},
        # a prompt scored token by token with twenty alternatives each
        {"name": "score_prompt", "op": "score", "rows": 2048, "vocab": 128256, "type": "bf16",
         "top": 20, "masked": False},
        # an odd vocabulary, rows without alignment
        {"name": "score_odd", "op": "score", "rows": 1000, "vocab": 32003, "type": "fp16", "top": 1,
         "masked": False},
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "step", "score"])
    if op == "step":
        batch, mbs = _between(rng, 1, 512), _between(rng, 8, 520)
        hi, new = rng.randint(0, 8 * mbs), _between(rng, 1, 8 * mbs)
        new = min(new, max(1, 500000 // batch))
        return {"op": op, "batch": batch, "lo": rng.randint(0, hi), "hi": hi,
                "new_lo": rng.randint(0, new), "new_hi": new, "forked": rng.randint(0, batch // 2),
                "blocks": batch * mbs + rng.randint(0, 1000), "mbs": mbs,
                "spare": rng.choice([0, 0, 7, 100]), "reject": rng.random() < 0.5}
    if op == "score":
        vocab = rng.choice([_between(rng, 2, 262144), 32000, 128256, 50257])
        return {"op": op, "rows": _between(rng, 1, max(1, min(4096, 2048 * 128256 // vocab))),
                "vocab": vocab, "type": rng.choice(["bf16", "fp16", "fp32"]),
                "top": min(vocab, rng.choice([0, 1, 5, 20, 32])), "masked": rng.random() < 0.3}
    kv, group = rng.choice([1, 2, 4, 8, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    hi = _between(rng, 1, 16384)
    cached = 0 if rng.random() < 0.5 else _between(rng, 1, 65536)
    most = 2 ** 32 // (hi * (hi + cached) * kv * group)      # half of the longest listed case
    while most < 1:
        hi, cached = max(1, hi // 2), cached // 2
        most = 2 ** 32 // (hi * (hi + cached) * kv * group)
    return {"op": op, "batch": _between(rng, 1, min(64, most)), "q_heads": kv * group,
            "kv_heads": kv, "dim": rng.choice([64, 128, 128]),
            "cached_lo": rng.randint(0, cached), "cached_hi": cached, "lo": rng.randint(0, hi),
            "hi": hi, "window": _between(rng, 1, hi + cached) if rng.random() < 0.25 else 0,
            "pages": rng.choice(["bf16", "bf16", "fp8"])}


def _spread(lo, hi, n, turn=0):
    """n whole numbers evenly spaced over [lo, hi], its ends included, in an order by `turn`."""
    x = [hi] if n == 1 else [lo + round((hi - lo) * i / (n - 1)) for i in range(n)]
    step = 1 + 2 * turn
    while math.gcd(step, n) > 1:
        step += 1
    return [x[i * step % n] for i in range(n)]


def _lens(case):
    """(new tokens, context length) of every sequence of a prompt case."""
    new = _spread(case["lo"], case["hi"], case["batch"], 3)
    cached = _spread(case["cached_lo"], case["cached_hi"], case["batch"], 1)
    return new, [a + b for a, b in zip(new, cached)]


# ------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return {"prompt": _prepare_prompt, "step": _prepare_step, "score": _prepare_score}[case["op"]](
        case, seed, g)


def _prepare_prompt(case, seed, g):
    B, Hkv, D = case["batch"], case["kv_heads"], case["dim"]
    new, lens = _lens(case)
    mbs = max(1, (max(lens) + BLOCK - 1) // BLOCK)
    NB = B * mbs + 3
    tables = torch.randperm(NB, generator=g, device=DEV)[:B * mbs].view(B, mbs).int()
    st = {"case": case, "tables": tables, "most": max(1, max(lens))}
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["starts"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEV)
    st["longest"] = max(new)
    st["q"] = torch.randn((sum(new), case["q_heads"], D), generator=g, device=DEV).bfloat16()
    # slots behind a context's end hold what an earlier sequence left there, here NaN
    at = torch.arange(mbs * BLOCK, device=DEV)
    dead = (at >= st["lens"][:, None]).view(B, mbs, BLOCK)
    b, m, t = dead.nonzero(as_tuple=True)
    for name in ("k", "v"):
        x = torch.randn((NB, Hkv, BLOCK, D), generator=g, device=DEV)
        if case["pages"] == "bf16":
            x = x.bfloat16()
            x[tables[b, m].long(), :, t] = math.nan
        else:
            st[name + "_scale"] = torch.rand(Hkv, generator=g, device=DEV) / 96 + 1 / 96
            x = (x / st[name + "_scale"][:, None, None]).clamp(-448, 448)
            x[tables[b, m].long(), :, t] = math.nan
            x = x.to(torch.float8_e4m3fn).view(torch.uint8)
            x = x.transpose(-1, -2).contiguous() if name == "v" else x
        st[name] = x
    return st


def _prepare_step(case, seed, g):
    r = np.random.default_rng(seed)
    B, mbs, NB = case["batch"], case["mbs"], case["blocks"]
    lens = np.array(_spread(case["lo"], case["hi"], B, 2))
    new = np.array(_spread(case["new_lo"], case["new_hi"], B, 5))
    order = r.permutation(B)
    lens, new = lens[order], new[order]
    for i in range(case["forked"]):                     # sequence 2i + 1 is a fork of 2i
        lens[2 * i + 1] = lens[2 * i]
    have = -(-lens // BLOCK)
    tables = np.full((B, mbs), -1)
    # blocks have come and gone: the sequences' own lie among the first ones in any order
    ids = r.permutation(min(NB, int(have.sum()) * 5 // 4 + 1))
    refs = np.zeros(NB, dtype=np.int64)
    used = 0
    for b in range(B):
        if b % 2 and b // 2 < case["forked"]:
            tables[b] = tables[b - 1]
        else:
            tables[b, :have[b]] = ids[used:used + have[b]]
            used += have[b]
        refs[tables[b, :have[b]]] += 1
    total = int(new.sum()) + case["spare"]
    kept = torch.from_numpy(np.concatenate([lens, tables.ravel(), refs]).astype(np.int32)).to(DEV)
    live = kept.clone()
    keep = lens + new - r.integers(0, new + 1)
    return {"case": case, "kept": kept, "live": live, "lens": live[:B],
            "tables": live[B:B + B * mbs].view(B, mbs), "refs": live[B + B * mbs:],
            "new": torch.from_numpy(new.astype(np.int32)).to(DEV), "total": total,
            "keep": torch.from_numpy(keep.astype(np.int32)).to(DEV)}


def _prepare_score(case, seed, g):
    N, V = case["rows"], case["vocab"]
    x = torch.randn((N, V), generator=g, device=DEV)
    # most rows have a few likely tokens, some are nearly flat
    x *= 0.5 + 3 * torch.rand((N, 1), generator=g, device=DEV)
    if case["masked"]:
        x[torch.rand((N, V), generator=g, device=DEV) < 0.1] = -math.inf
        x[:, 0] = 0.25
    tokens = torch.randint(0, V, (N,), generator=g, device=DEV)
    best = torch.rand(N, generator=g, device=DEV) < 0.5
    tokens = torch.where(best, x.argmax(-1), tokens).int()
    return {"case": case, "logits": x.to(TYPES[case["type"]]), "tokens": tokens}


# ------------------------------------------------------------------------------- plain forms
def _entries(st, case):
    """K and V of every sequence, [B, Hkv, J, D] in 32 bits, V zero behind the context."""
    out = []
    for name in ("k", "v"):
        x = st[name][st["tables"].long()]               # [B, M, Hkv, ...]
        if case["pages"] == "fp8":
            x = x.view(torch.float8_e4m3fn).float() * st[name + "_scale"][:, None, None]
            x = x.transpose(-1, -2) if name == "v" else x
        out.append(x.float().transpose(1, 2).flatten(2, 3))
    live = torch.arange(out[1].shape[2], device=DEV) < st["lens"][:, None]
    out[1] = torch.where(live[:, None, :, None], out[1], 0.0)
    return out


def _plain_prompt(st, case):
    """Padded to the longest prompt: rows of all sequences in one batch of products."""
    B, Hkv, D, T = case["batch"], case["kv_heads"], case["dim"], st["longest"]
    G = case["q_heads"] // Hkv
    first, count = st["starts"][:-1].long(), st["starts"].diff().long()
    t = torch.arange(T, device=DEV)
    real = t < count[:, None]                           # [B, T]
    rows = torch.where(real, first[:, None] + t, 0)
    q = st["q"][rows].float().view(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4).flatten(2, 3)
    keys, values = _entries(st, case)
    s = (q @ keys.transpose(-1, -2)).mul_(1 / math.sqrt(D)).view(B, Hkv, G, T, -1)
    j = torch.arange(keys.shape[2], device=DEV)
    last = (st["lens"].long() - count)[:, None] + t     # [B, T]
    hidden = (j > last[..., None]) | (j >= st["lens"][:, None, None])
    if case["window"]:
        hidden |= j <= last[..., None] - case["window"]
    s.masked_fill_(hidden[:, None, None], -math.inf)
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    s.div_(s.sum(-1, keepdim=True))
    o = (s.flatten(2, 3) @ values).view(B, Hkv, G, T, D).permute(0, 3, 1, 2, 4).flatten(2, 3)
    return o[real].bfloat16()


def _plain_extend(st, case):
    B, mbs, NB, N = case["batch"], case["mbs"], case["blocks"], st["total"]
    lens, new = st["lens"].long(), st["new"].long()
    tables, refs = st["tables"].long(), st["refs"].long()
    b = torch.arange(B, device=DEV)
    have, want = (lens + 15) // BLOCK, (lens + new + 15) // BLOCK
    end = (have - 1).clamp(min=0)
    last = tables[b, end]
    writes = (lens % BLOCK > 0) & (new > 0)             # into its last block
    before = (last[:, None] == last) & writes & (b < b[:, None])
    copied = writes & (refs[last.clamp(min=0)] - before.sum(1) > 1)
    need = want - have + copied
    at = need.cumsum(0) - need
    free = refs == 0
    ids = torch.zeros(NB + 1, dtype=torch.long, device=DEV)
    ids.scatter_(0, torch.where(free, free.cumsum(0) - 1, NB), torch.arange(NB, device=DEV))
    j = torch.arange(mbs, device=DEV)
    fresh = (j >= have[:, None]) & (j < want[:, None])
    fresh |= copied[:, None] & (j == end[:, None])
    pick = at[:, None] + copied[:, None] + j - have[:, None]
    tables = torch.where(fresh, ids[pick.clamp(0, NB)], tables)
    copies = torch.where(copied[:, None], torch.stack([last, tables[b, end]], 1), 0)
    refs = refs + torch.zeros(NB + 1, dtype=torch.long, device=DEV).index_add_(
        0, torch.where(fresh, tables, NB).flatten(), torch.ones(B * mbs, dtype=torch.long,
                                                                device=DEV))[:NB]
    refs.index_add_(0, last.clamp(min=0), -copied.long())
    starts = torch.zeros(B + 1, dtype=torch.long, device=DEV)
    starts[1:] = new.cumsum(0)
    i = torch.arange(N, device=DEV)
    seq = torch.searchsorted(starts[1:].contiguous(), i, right=True)
    real, seq = seq < B, seq.clamp(max=B - 1)
    pos = lens[seq] + i - starts[seq]
    slots = tables[seq, (pos // BLOCK).clamp(0, mbs - 1)] * BLOCK + pos % BLOCK
    st["tables"].copy_(tables)
    st["refs"].copy_(refs)
    st["lens"].copy_(lens + new)
    return (starts.int(), torch.where(real, slots, -1), torch.where(real, pos, -1).int(),
            copies.int())


def _plain_truncate(st, case):
    lens, keep, tables = st["lens"].long(), st["keep"].long(), st["tables"].long()
    j = torch.arange(case["mbs"], device=DEV)
    drop = (j >= (keep[:, None] + 15) // BLOCK) & (j < (lens[:, None] + 15) // BLOCK)
    gone = torch.zeros(case["blocks"] + 1, dtype=torch.int32, device=DEV).index_add_(
        0, torch.where(drop, tables, case["blocks"]).flatten(),
        torch.ones(tables.numel(), dtype=torch.int32, device=DEV))
    st["refs"].sub_(gone[:-1])
    st["tables"].masked_fill_(drop, -1)
    st["lens"].copy_(st["keep"])


def _plain_score(st, case):
    x = st["logits"].float()
    m = x.amax(-1, keepdim=True)
    d = x - m
    e = d.exp()
    z = e.sum(-1)
    spread = torch.where(e > 0, d * e, 0.0).sum(-1)
    at = x.gather(-1, st["tokens"].long()[:, None])[:, 0]
    shift = m[:, 0] + z.log()
    out = [(at - m[:, 0]) - z.log(), z.log() - spread / z]
    if case["top"]:
        v, i = x.sort(dim=-1, descending=True, stable=True)
        out += [v[:, :case["top"]] - shift[:, None], i[:, :case["top"]].int()]
    return out


def run(state):
    st, case = state, state["case"]
    if case["op"] == "prompt":
        if own:
            import paged_kv_cache_221_gb300 as pa
            return pa.prompt_attention(st["q"], st["k"], st["v"], st["tables"], st["lens"],
                                       st["starts"], st["most"], window_size=case["window"],
                                       k_scale=st.get("k_scale"), v_scale=st.get("v_scale"))
        return _plain_prompt(st, case)
    if case["op"] == "step":
        # the pass is made on the same batch again and again: the state as it was before
        st["live"].copy_(st["kept"])
        if own:
            import paged_kv_cache_221_gb300 as pa
            made = pa.extend_sequences(st["tables"], st["lens"], st["refs"], st["new"], st["total"])
            if case["reject"]:
                pa.truncate_sequences(st["tables"], st["lens"], st["refs"], st["keep"])
        else:
            made = _plain_extend(st, case)
            if case["reject"]:
                _plain_truncate(st, case)
        return [*made, st["tables"], st["lens"], st["refs"]]
    if own:
        import paged_kv_cache_221_gb300 as pa
        out = pa.token_logprobs(st["logits"], st["tokens"], case["top"])
        return list(out) if case["top"] else list(out[:2])
    return _plain_score(st, case)


# ------------------------------------------------------------------------------- 64 bits
def _exact_prompt(st, case):
    """One sequence, one kv head and a few query tokens after the other."""
    new, lens = _lens(case)
    visible = sum(n * (c - n) + n * n // 2 for n, c in zip(new, lens))
    if 4.0 * visible * case["q_heads"] * case["dim"] > 8e12:
        return None
    Hkv, D, W = case["kv_heads"], case["dim"], case["window"]
    G = case["q_heads"] // Hkv
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
    row = 0
    for b in range(case["batch"]):
        n, L = new[b], lens[b]
        ids = st["tables"][b, :(L + 15) // 16].long()
        k, v = st["k"][ids], st["v"][ids]
        if case["pages"] == "fp8":
            k = k.view(torch.float8_e4m3fn).double() * st["k_scale"].double()[None, :, None, None]
            v = v.view(torch.float8_e4m3fn).double().permute(0, 1, 3, 2)
            v = v * st["v_scale"].double()[None, :, None, None]
        k = k.double().permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :L]
        v = v.double().permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :L]
        for t0 in range(0, n, 1024):
            t1 = min(n, t0 + 1024)
            p0, p1 = L - n + t0, L - n + t1             # positions of these query tokens
            a = max(0, p0 - W + 1) if W else 0
            pos = torch.arange(p0, p1, device=DEV)[:, None]
            j = torch.arange(a, p1, device=DEV)
            see = (j <= pos) & (j > pos - W if W else True)
            for h in range(case["q_heads"]):
                q = st["q"][row + t0:row + t1, h].double()
                s = q @ k[h // G, a:p1].T / D ** 0.5
                w = torch.softmax(s.masked_fill(~see, -math.inf), -1)
                out[row + t0:row + t1, h] = w @ v[h // G, a:p1]
        row += n
    return out


def _exact_step(st, case):
    """Token by token in the order of the batch, with the lowest free block each time."""
    B, mbs = case["batch"], case["mbs"]
    kept = st["kept"].cpu().numpy().astype(np.int64)
    lens, tables, refs = kept[:B].copy(), kept[B:B + B * mbs].reshape(B, mbs).copy(), \
        kept[B + B * mbs:].copy()
    new, keep = st["new"].cpu().numpy(), st["keep"].cpu().numpy()
    free = iter(np.flatnonzero(refs == 0).tolist())
    starts, slots, positions = [0], [], []
    copies = np.zeros((B, 2), dtype=np.int64)
    for b in range(B):
        row, at = tables[b], int(lens[b])
        for _ in range(int(new[b])):
            i = at // BLOCK
            if at % BLOCK == 0:
                row[i] = next(free)
                refs[row[i]] = 1
            elif refs[row[i]] > 1:
                fresh = next(free)
                refs[fresh], refs[row[i]] = 1, refs[row[i]] - 1
                copies[b] = row[i], fresh
                row[i] = fresh
            slots.append(int(row[i]) * BLOCK + at % BLOCK)
            positions.append(at)
            at += 1
        lens[b] = at
        starts.append(len(slots))
    behind = st["total"] - len(slots)
    if case["reject"]:
        for b in range(B):
            for i in range(-(-int(keep[b]) // BLOCK), -(-int(lens[b]) // BLOCK)):
                refs[tables[b, i]] -= 1
                tables[b, i] = -1
        lens = keep
    return [torch.tensor(starts, dtype=torch.int32), torch.tensor(slots + [-1] * behind),
            torch.tensor(positions + [-1] * behind, dtype=torch.int32),
            torch.tensor(copies, dtype=torch.int32), torch.tensor(tables, dtype=torch.int32),
            torch.tensor(lens, dtype=torch.int32), torch.tensor(refs, dtype=torch.int32)]


def _exact_score(st, case):
    parts = []
    for x, t in zip(st["logits"].split(256), st["tokens"].split(256)):
        x = x.double()
        lp = x - torch.logsumexp(x, -1, keepdim=True)
        part = [lp[torch.arange(len(t), device=DEV), t.long()],
                -torch.where(lp > -math.inf, lp.exp() * lp, 0.0).sum(-1)]
        if case["top"]:
            order = torch.argsort(x, dim=-1, descending=True, stable=True)[:, :case["top"]]
            part += [lp.gather(-1, order), order.int()]
        parts.append(part)
    return [torch.cat(p) for p in zip(*parts)]


def exact(case, seed):
    st = prepare(case, seed)
    return {"prompt": _exact_prompt, "step": _exact_step, "score": _exact_score}[case["op"]](
        st, case)


# ------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "prompt":
        new, lens = _lens(case)
        W, D = case["window"], case["dim"]
        pairs = entries = 0
        for n, L in zip(new, lens):
            c = L - n                                   # position of the first query token
            if not W:
                pairs += n * c + n * (n + 1) // 2
                entries += L if n else 0
            else:
                short = max(0, min(n, W - 1 - c))       # query tokens that see their whole past
                pairs += short * c + short * (short + 1) // 2 + (n - short) * W
                entries += min(L, n + W - 1) if n else 0
        size = 1 if case["pages"] == "fp8" else 2
        return {"bytes": 4 * sum(new) * case["q_heads"] * D
                + 2 * size * entries * case["kv_heads"] * D + 4 * (entries // BLOCK),
                "flops": 4 * D * case["q_heads"] * pairs}
    if case["op"] == "step":
        B = case["batch"]
        new = sum(_spread(case["new_lo"], case["new_hi"], B, 5))
        # lengths, new lengths, starts, copies, a slot and a position per row, the reference
        # counts up to the free blocks, and an entry and a count per new block
        return {"bytes": 24 * B + 12 * (new + case["spare"]) + 4 * min(case["blocks"], new)
                + 8 * (new // BLOCK), "flops": 0}
    size = 4 if case["type"] == "fp32" else 2
    n = case["rows"] * case["vocab"]
    return {"bytes": size * n + case["rows"] * (12 + 8 * case["top"]), "flops": 5 * n}
