"""Cases of the compressed-cache operators: 4-bit pages, the attention that reads them, and
eviction by accumulated attention weight.

Four kinds of case:

attend   attention of T query tokens per sequence over 4-bit pages, with or without the query
         tokens' K/V appended by the call; the appended tokens are read back as values
store    new tokens' K/V quantised into 4-bit pages and read back as bf16
observe  the attention weights of T query tokens added to each cache entry's running sum
evict    the entries with the smallest sums dropped and the cache closed up; with "step" the
         whole per-token loop of a bounded cache: evict one entry, append and attend, observe

A 4-bit page holds 16 tokens of one kv head: 16 rows of D/2 bytes (dim d in byte d/2, even d in
the low nibble; value code - 8), then 16 rows of D/32 E4M3 scales, one for 32 dims.  A value is
(code - 8) * scale * head_scale.

With `own` false `run` is the plain form in elementary torch operations; with `own` true it
calls the package.
"""
import math

import torch

own = False

BLOCK = 16
GROUP = 32
DEV = "cuda"


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # two short chats, 4 kv heads of 64 dims: nothing but latency
        {"name": "attend_tiny", "op": "attend", "batch": 2, "q_heads": 4, "kv_heads": 4,
         "dim": 64, "tokens": 1, "lo": 37, "hi": 100, "log": False, "window": 0,
         "append": False},
        # a decode step of a mid-sized serving batch, grouped-query attention 4 to 1
        {"name": "attend_decode", "op": "attend", "batch": 64, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "tokens": 1, "lo": 512, "hi": 4096, "log": False, "window": 0,
         "append": False},
        # a decode step of a large batch with very uneven contexts, new tokens appended
        {"name": "attend_batch", "op": "attend", "batch": 256, "q_heads": 64, "kv_heads": 8,
         "dim": 128, "tokens": 1, "lo": 128, "hi": 8192, "log": True, "window": 0,
         "append": True},
        # verification of five drafts per sequence, drafts appended
        {"name": "attend_verify", "op": "attend", "batch": 32, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "tokens": 5, "lo": 2048, "hi": 16384, "log": False, "window": 0,
         "append": True},
        # one user with a very long document
        {"name": "attend_long", "op": "attend", "batch": 1, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "tokens": 1, "lo": 131071, "hi": 131071, "log": False, "window": 0,
         "append": False},
        # layers that look at the last thousand tokens only
        {"name": "attend_window", "op": "attend", "batch": 64, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "tokens": 1, "lo": 2048, "hi": 16384, "log": False, "window": 1000,
         "append": False},
        # the prompts of several requests written in one chunk, with padding rows
        {"name": "store_prompt", "op": "store", "count": 16389, "kv_heads": 8, "dim": 128,
         "pad": 37},
        # the new tokens of one decode step
        {"name": "store_step", "op": "store", "count": 256, "kv_heads": 8, "dim": 128,
         "pad": 0},
        # the statistics of a decode step over a bf16 cache
        {"name": "observe_decode", "op": "observe", "batch": 64, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "tokens": 1, "lo": 512, "hi": 4096, "log": False, "pages": "bf16",
         "decay": 1.0},
        # the statistics of five verified tokens over a 4-bit cache, with fading
        {"name": "observe_verify", "op": "observe", "batch": 32, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "tokens": 5, "lo": 2048, "hi": 16384, "log": False, "pages": "int4",
         "decay": 0.9},
        # prompts of up to 8192 tokens cut to 2048 entries before decoding starts
        {"name": "evict_prompt", "op": "evict", "batch": 16, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "tokens": 1, "lo": 4096, "hi": 8192, "log": False, "pages": "bf16",
         "budget": 2048, "recent": 256, "step": False},
        # the loop of a bounded 4-bit cache: one entry out, one in, attend, observe
        {"name": "evict_step", "op": "evict", "batch": 64, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "tokens": 1, "lo": 2049, "hi": 2049, "log": False, "pages": "int4",
         "budget": 2048, "recent": 512, "step": True},
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "store", "observe", "observe", "evict"])
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8, 8])
    if op == "store":
        return {"op": op, "count": _between(rng, 1, 16389), "kv_heads": kv, "dim": dim,
                "pad": rng.choice([0, 0, 3, 37])}
    tokens = rng.choice([1, 1, 1, 2, 3, 5, 7])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if g * tokens <= 64])
    hi = _between(rng, max(tokens, 16), 131071)
    most = 256 * 1940 * 8 * 128 // 4                # a quarter of the largest listed case
    batch = _between(rng, 1, max(1, min(256, most // (hi * kv * dim))))
    case = {"op": op, "batch": batch, "q_heads": kv * group, "kv_heads": kv, "dim": dim,
            "tokens": tokens, "lo": rng.randint(tokens, hi), "hi": hi,
            "log": rng.random() < 0.3}
    if op == "attend":
        return {**case, "window": _between(rng, 1, hi) if rng.random() < 0.25 else 0,
                "append": rng.random() < 0.5}
    case["pages"] = rng.choice(["bf16", "fp8", "int4", "int4"])
    if op == "observe":
        return {**case, "decay": rng.choice([1.0, 1.0, 0.9, 0.0])}
    budget = rng.randint(1, max(1, hi - 1))
    case.update(tokens=1, q_heads=kv * min(group, 8), budget=budget,
                recent=rng.randint(0, budget), step=False)
    return case


def _lens(case):
    """Context lengths: evenly spaced quantiles of the case's range, its ends included."""
    B, lo, hi = case["batch"], case["lo"], case["hi"]
    if B == 1:
        return [hi]
    if case["log"]:
        a, b = math.log(lo), math.log(hi)
        return [min(hi, max(lo, round(math.exp(a + (b - a) * i / (B - 1))))) for i in range(B)]
    return [lo + round((hi - lo) * i / (B - 1)) for i in range(B)]


# ------------------------------------------------------------------------------- formats
def _pack4(x, head_scale):
    """[..., Hkv, 16, D] values to 4-bit pages [..., Hkv, 8 D + D / 2] (uint8)."""
    x = x.float()
    D = x.shape[-1]
    g = x.unflatten(-1, (D // GROUP, GROUP))
    s = g.abs().amax(-1) / (7 * head_scale[:, None, None])
    s8 = s.clamp(max=448.0).to(torch.float8_e4m3fn)
    step = (s8.float() * head_scale[:, None, None])[..., None]
    code = torch.where(step > 0, g / step, torch.zeros_like(g)).round().clamp(-7, 7) + 8
    code = code.to(torch.uint8).flatten(-2)
    rows = code[..., 0::2] | (code[..., 1::2] << 4)
    return torch.cat([rows.flatten(-2), s8.view(torch.uint8).flatten(-2)], -1)


def _parts4(pages, D):
    """Views of 4-bit pages: code rows [..., 16, D / 2] and scales [..., 16, D / 32]."""
    return (pages[..., :8 * D].unflatten(-1, (BLOCK, D // 2)),
            pages[..., 8 * D:].unflatten(-1, (BLOCK, D // GROUP)))


def _values4(rows, scales, head_scale):
    """The values [..., D] of code rows [..., D / 2] and E4M3 scales [..., D / 32], 32 bits."""
    s = scales.contiguous().view(torch.float8_e4m3fn).float() * head_scale
    code = torch.stack([rows & 15, rows >> 4], -1).flatten(-2).float() - 8
    return (code.unflatten(-1, (s.shape[-1], GROUP)) * s[..., None]).flatten(-2)


def _unpack4(pages, head_scale, D):
    """4-bit pages [..., Hkv, bytes] to values [..., Hkv, 16, D] in 32 bits."""
    return _values4(*_parts4(pages, D), head_scale[:, None, None])


def _keys(st, case):
    """The K entries [B, Hkv, J, D] of every sequence, in 32 bits."""
    k = st["k"][st["tables"].long()]                # [B, M, Hkv, ...]
    if case["pages"] == "int4":
        k = _unpack4(k, st["k_scale"], case["dim"])
    elif case["pages"] == "fp8":
        k = k.view(torch.float8_e4m3fn).float() * st["k_scale"][:, None, None]
    return k.float().transpose(1, 2).flatten(2, 3)


def _probs(st, case, keys, lens, window=0):
    """Softmax weights [B, Hkv, T, G, J] in 32 bits, zero where a query token does not see."""
    q, T = st["q"].float(), case["tokens"]
    B, _, Hq, D = q.shape
    Hkv, J = keys.shape[1], keys.shape[2]
    q = q.view(B, T, Hkv, Hq // Hkv, D).transpose(1, 2).flatten(2, 3)
    s = (q @ keys.transpose(-1, -2)).view(B, Hkv, T, Hq // Hkv, J) / math.sqrt(D)
    j = torch.arange(J, device=DEV)
    last = lens[:, None].long() - T + torch.arange(T, device=DEV)        # [B, T]
    see = j <= last[..., None]
    if window:
        see &= j > last[..., None] - window
    s = torch.where(see[:, None, :, None], s, torch.full_like(s, -math.inf))
    e = (s - s.amax(-1, keepdim=True)).exp()
    return e / e.sum(-1, keepdim=True)


def _plain_attend(st, case, lens):
    B, T, Hq, D = st["q"].shape
    keys = _keys(st, case)
    p = _probs(st, case, keys, lens, case.get("window", 0))
    del keys
    v = _unpack4(st["v"][st["tables"].long()], st["v_scale"], D).transpose(1, 2).flatten(2, 3)
    live = torch.arange(v.shape[2], device=DEV) < lens[:, None]
    v = torch.where(live[:, None, :, None], v, torch.zeros_like(v))
    o = p.flatten(2, 3) @ v
    return o.view(B, v.shape[1], T, Hq // v.shape[1], D).transpose(1, 2).flatten(2, 3).bfloat16()


def _plain_store(st, D):
    """Quantise st["key"] / st["value"] into their slots; negative slots are skipped."""
    at = st["slots"][st["slots"] >= 0]
    b, t = at // BLOCK, at % BLOCK
    for pool, new, scale in (("k", "key", "k_scale"), ("v", "value", "v_scale")):
        x = st[new][st["slots"] >= 0].unsqueeze(-2)             # [n, Hkv, 1, D]
        page = _pack4(x, st[scale])                             # one row and its scales
        rows, scales = _parts4(st[pool], D)
        rows[b, :, t], scales[b, :, t] = page[..., :D // 2], page[..., D // 2:]


def _plain_gather(st, D, slots):
    """The values in the slots, bf16 [N, Hkv, D]; zeros for negative slots."""
    b, t = slots.clamp(min=0) // BLOCK, slots.clamp(min=0) % BLOCK
    out = []
    for pool, scale in (("k", "k_scale"), ("v", "v_scale")):
        rows, scales = (x[b, :, t] for x in _parts4(st[pool], D))
        x = _values4(rows, scales, st[scale][:, None])
        out.append(torch.where((slots >= 0)[:, None, None], x, torch.zeros_like(x)).bfloat16())
    return out


def _plain_observe(st, case, lens, before, after):
    """after = decay * before + the weights of st["q"]; entries behind a context stay."""
    T = case["tokens"]
    p = _probs(st, case, _keys(st, case), lens).sum((2, 3))
    J = before.shape[-1]
    j = torch.arange(J, device=DEV)
    old = torch.where((j < lens[:, None] - T)[:, None], before * case.get("decay", 1.0),
                      torch.zeros_like(before))
    live = (j < lens[:, None])[:, None]
    after.copy_(torch.where(live, old + p[..., :J], after))
    new = live & (j >= lens[:, None] - T)[:, None]
    pos = (st["seen"] - lens)[:, None] + j
    st["positions"].copy_(torch.where(new, pos[:, None].int(), st["positions"]))


def _plain_evict(st, case):
    budget, w, pos, lens = case["budget"], st["weights"], st["positions"], st["lens"]
    J = w.shape[-1]
    j = torch.arange(J, device=DEV)
    live = (j < lens[:, None])[:, None].expand_as(w)
    newest = torch.where(live, pos, torch.full_like(pos, -2 ** 31)).amax(-1, keepdim=True)
    safe = live & (pos > newest - case["recent"])
    order = torch.where(live, w, torch.full_like(w, -math.inf)).sort(
        dim=-1, descending=True, stable=True).indices
    kind = torch.gather(safe.int() + live.int(), -1, order)
    order = torch.gather(order, -1, kind.sort(dim=-1, descending=True, stable=True).indices)
    kept = torch.zeros_like(live).scatter(-1, order[..., :budget], True) & live
    src = (kept & (j >= budget)).nonzero()
    dst = (live & ~kept & (j < budget)).nonzero()
    b, h = src[:, 0], src[:, 1]
    tab = st["tables"].long()
    bs, ts, bd, td = (x for i in (src[:, 2], dst[:, 2]) for x in (tab[b, i // BLOCK], i % BLOCK))
    D = case["dim"]
    for name in ("k", "v"):
        pool = st[name]
        if case["pages"] == "int4":
            views = _parts4(pool, D)
        elif case["pages"] == "fp8" and name == "v":
            views = [pool.transpose(-1, -2)]
        else:
            views = [pool]
        for x in views:
            x[bd, h, td] = x[bs, h, ts]
    w[b, h, dst[:, 2]] = w[b, h, src[:, 2]]
    pos[b, h, dst[:, 2]] = pos[b, h, src[:, 2]]
    return lens.clamp(max=budget)


# ------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).bfloat16()

    def head_scales():
        # powers of two of a calibration, between 1/16 and 1/4
        return torch.exp2(torch.randint(-4, -1, (case["kv_heads"],), generator=gen,
                                        device=DEV).float())

    D, Hkv = case["dim"], case["kv_heads"]
    st = {"case": case, "k_scale": head_scales(), "v_scale": head_scales()}
    if case["op"] == "store":
        n, NB = case["count"], -(-case["count"] // BLOCK) + 3
        st["key"], st["value"] = normal(n, Hkv, D), normal(n, Hkv, D)
        start = torch.randint(0, 3 * BLOCK, (1,), generator=gen, device=DEV)
        slots = start + torch.arange(n, device=DEV)              # a run of whole blocks ...
        perm = torch.randperm(NB, generator=gen, device=DEV)
        slots = perm[slots // BLOCK] * BLOCK + slots % BLOCK     # ... placed anywhere
        if case["pad"]:
            slots[::case["pad"]] = -1
        st["slots"] = slots
        page = 8 * D + D // 2
        st["k"] = torch.zeros((NB, Hkv, page), dtype=torch.uint8, device=DEV)
        st["v"] = torch.zeros((NB, Hkv, page), dtype=torch.uint8, device=DEV)
        return st

    pages = case.get("pages", "int4")
    st["case"] = case = {**case, "pages": pages}
    B, T = case["batch"], case["tokens"]
    perm = torch.randperm(B, generator=gen, device=DEV)
    lens = torch.tensor(_lens(case), device=DEV, dtype=torch.int32)[perm]
    M = -(-case["hi"] // BLOCK)
    need = (lens.long() + BLOCK - 1) // BLOCK
    total = sum(-(-n // BLOCK) for n in _lens(case))
    NB = total + total // 4 + 1                                  # a pool 1.25x the need
    ids = torch.randperm(NB, generator=gen, device=DEV).int()
    first = need.cumsum(0) - need
    col = torch.arange(M, device=DEV)
    at = (first[:, None] + col).clamp(max=NB - 1)
    st["tables"] = torch.where(col < need[:, None], ids[at], torch.zeros_like(ids[at]))
    step = case["op"] == "evict" and case["step"]
    st["lens"], st["seen"] = lens, (lens + 1000 + step).int()    # tokens seen so far
    st["q"] = normal(B, T, case["q_heads"], D)
    for name in ("k", "v"):
        scale = st[name + "_scale"]
        x = normal(NB, Hkv, BLOCK, D)
        if pages == "int4":
            x = _pack4(x, scale)
        elif pages == "fp8":
            x = (x.float() / scale[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            x = x.view(torch.uint8)
            x = x.transpose(-1, -2).contiguous() if name == "v" else x
        st[name] = x
    if case["op"] == "attend" and not case["append"]:
        return st
    # the newest T tokens of every sequence, and their slots
    j = (lens[:, None] - T + torch.arange(T, device=DEV)).long()
    slots = torch.gather(st["tables"].long(), 1, j // BLOCK) * BLOCK + j % BLOCK
    st["slots"] = slots.flatten()
    st["key"], st["value"] = normal(B * T, Hkv, D), normal(B * T, Hkv, D)
    if case["op"] == "attend":
        return st
    J = M * BLOCK
    w = torch.randn((B, Hkv, J), generator=gen, device=DEV).mul(2).exp()   # heavy tails ...
    drop = torch.rand((B, Hkv, J), generator=gen, device=DEV) < 0.05       # ... and some zeros
    st["weights0"] = torch.where(drop, torch.zeros_like(w), w)
    st["weights"] = st["weights0"].clone()
    # entries hold tokens in order, 1000 of them evicted from the front earlier on
    st["positions0"] = (torch.arange(J, device=DEV, dtype=torch.int32) + 1000).expand(
        B, Hkv, J).contiguous()
    st["positions"] = st["positions0"].clone()
    if step:
        _plain_store(st, D)                          # what the loop's last append has left
    elif case["op"] == "evict" and pages == "int4":
        # the slots of the entries that stay, to read the cut cache back
        j = torch.arange(case["budget"], device=DEV).expand(B, -1)
        slots = torch.gather(st["tables"].long(), 1, j // BLOCK) * BLOCK + j % BLOCK
        st["kept"] = torch.where(j < lens[:, None], slots, torch.full_like(slots, -1)).flatten()
    return st


# ------------------------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    return (_run_own if own else _run_plain)(st, case, case["op"], case["dim"])


def _run_plain(st, case, op, D):
    if op == "store":
        _plain_store(st, D)
        return _plain_gather(st, D, st["slots"])
    if op == "attend":
        if not case["append"]:
            return _plain_attend(st, case, st["lens"])
        _plain_store(st, D)
        return [_plain_attend(st, case, st["lens"]), *_plain_gather(st, D, st["slots"])]
    if op == "observe":
        _plain_observe(st, case, st["lens"], st["weights0"], st["weights"])
        return [st["weights"], st["positions"]]
    st["weights"].copy_(st["weights0"])
    st["positions"].copy_(st["positions0"])
    lens = _plain_evict(st, case)
    if not case["step"]:
        if case["pages"] == "int4":
            return [lens, st["weights"], st["positions"], *_plain_gather(st, D, st["kept"])]
        return [lens, st["weights"], st["positions"], *_values(st, case)]
    _plain_store(st, D)
    lens = lens + 1
    out = _plain_attend(st, case, lens)
    _plain_observe(st, case, lens, st["weights"], st["weights"])
    return [lens, out, st["weights"], st["positions"]]


def _run_own(st, case, op, D):
    import paged_kv_cache_221_gb300 as pa
    cache = (st["k"], st["v"])
    scales = {"k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    if op == "store":
        pa.reshape_and_cache_int4(st["key"], st["value"], *cache, st["slots"], **scales)
        return list(pa.gather_cache_int4(*cache, st["slots"], **scales))
    k_scale = None if case["pages"] == "bf16" else st["k_scale"]
    if op == "attend":
        new = {"new_key": st["key"], "new_value": st["value"]} if case["append"] else {}
        out = pa.attention_int4(st["q"], *cache, st["k_scale"], st["v_scale"], st["tables"],
                                st["lens"], case["hi"], window_size=case["window"], **new)
        if not case["append"]:
            return out
        return [out, *pa.gather_cache_int4(*cache, st["slots"], **scales)]
    if op == "observe":
        pa.accumulate_weights(st["q"], st["k"], st["tables"], st["lens"], st["weights0"],
                              st["positions"], st["seen"], case["hi"], decay=case["decay"],
                              k_scale=k_scale, out=st["weights"])
        return [st["weights"], st["positions"]]
    st["weights"].copy_(st["weights0"])
    st["positions"].copy_(st["positions0"])
    lens = pa.evict_tokens(*cache, st["tables"], st["lens"], st["weights"], st["positions"],
                           case["budget"], case["recent"], case["hi"])
    if not case["step"]:
        if case["pages"] == "int4":
            return [lens, st["weights"], st["positions"],
                    *pa.gather_cache_int4(*cache, st["kept"], **scales)]
        return [lens, st["weights"], st["positions"], *_values(st, case)]
    lens = lens + 1
    bound = case["budget"] + 1
    out = pa.attention_int4(st["q"], *cache, st["k_scale"], st["v_scale"], st["tables"], lens,
                            bound, new_key=st["key"], new_value=st["value"])
    pa.accumulate_weights(st["q"], st["k"], st["tables"], lens, st["weights"], st["positions"],
                          st["seen"], bound, k_scale=k_scale)
    return [lens, out, st["weights"], st["positions"]]


def _values(st, case):
    """The cache as it stands, bf16 or FP8 pages."""
    if case["pages"] == "fp8":
        return [st["k"].view(torch.float8_e4m3fn), st["v"].view(torch.float8_e4m3fn)]
    return [st["k"], st["v"]]


# ------------------------------------------------------------------------------- work
def work(case):
    D, Hkv = case["dim"], case["kv_heads"]
    int4 = D // 2 + D // GROUP
    if case["op"] == "store":
        live = case["count"] - (-(-case["count"] // case["pad"]) if case["pad"] else 0)
        # bf16 in, pages out, pages in, bf16 out, for K and V; one slot for each of the two
        return {"bytes": 2 * Hkv * (2 * live * 2 * int4 // 2 + (live + case["count"]) * D * 2)
                + 16 * case["count"], "flops": 4 * live * Hkv * D}
    B, T, Hq, lens = case["batch"], case["tokens"], case["q_heads"], _lens(case)
    if case.get("window"):
        seen = sum(min(n, case["window"] + T - 1) for n in lens)
    else:
        seen = sum(lens)
    if case["op"] == "evict" and case["step"]:
        seen = B * (case["budget"] + 1)
    tables = 4 * -(-seen // BLOCK) + 4 * B
    rows = B * T * Hq * D * 2
    attend = 2 * seen * Hkv * int4 + 2 * rows + tables
    row = {"bf16": 2 * D, "fp8": D, "int4": int4}[case.get("pages", "int4")]
    observe = seen * Hkv * (row + 8) + rows + tables
    if case["op"] == "attend":
        if case["append"]:
            # new K/V in, the appended rows out and read back as bf16
            attend += 2 * B * T * Hkv * (4 * D + 2 * int4)
        return {"bytes": attend, "flops": 4 * seen * T * Hq * D}
    if case["op"] == "observe":
        return {"bytes": observe + 4 * B * T * Hkv, "flops": 2 * seen * T * Hq * D}
    moved = 0.0
    for n in lens:
        if n > case["budget"]:
            tail, free = n - case["budget"], n - case["recent"]
            r = min(case["recent"], tail)
            moved += r + (tail - r) * (case["budget"] - case["recent"]) / max(1, free)
    # the sums and positions in; the moved rows, sums and positions in and out
    evict = 8 * Hkv * sum(lens) + int(moved * Hkv * (4 * row + 16)) + 8 * B
    # the statistics laid fresh for the pass
    evict += 16 * B * Hkv * BLOCK * -(-case["hi"] // BLOCK)
    if not case["step"]:
        if case["pages"] == "int4":
            evict += 2 * Hkv * (sum(min(n, case["budget"]) for n in lens) * int4
                                + B * case["budget"] * 2 * D)
        return {"bytes": evict, "flops": Hkv * sum(lens)}
    return {"bytes": evict + attend + observe + 2 * B * T * Hkv * (2 * D + int4),
            "flops": 6 * seen * T * Hq * D}


# ------------------------------------------------------------------------------- 64 bits
_E4M3 = [(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
         for e in range(16) for m in range(8)][:127]


def _nearest(x):
    """Index of the E4M3 value nearest to each x >= 0: ties to the even index, 448 at most."""
    t = torch.tensor(_E4M3, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(t, x.contiguous()).clamp(1, 126)
    lo = hi - 1
    a, b = x - t[lo], t[hi] - x
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def _values64(x, head_scale):
    """What 4-bit storage makes of x [n, Hkv, D]."""
    n, Hkv, D = x.shape
    out = torch.empty((n, Hkv, D), dtype=torch.float64, device=x.device)
    t = torch.tensor(_E4M3, dtype=torch.float64, device=x.device)
    for h in range(Hkv):
        for g in range(0, D, GROUP):
            part = x[:, h, g:g + GROUP].double()
            unit = t[_nearest(part.abs().max(1).values / 7 / head_scale[h].double())]
            unit = unit * head_scale[h].double()
            q = part / torch.where(unit > 0, unit, torch.ones_like(unit))[:, None]
            out[:, h, g:g + GROUP] = torch.round(q).clamp(-7, 7) * unit[:, None]
    return out


def _entries64(st, case, name, b, h, upto):
    """Entries [0, upto) of sequence b and head h in 64 bits."""
    D = case["dim"]
    ids = st["tables"][b, :-(-upto // BLOCK)].long()
    page = st[name][ids, h]
    if case["pages"] == "bf16":
        x = page.double().reshape(-1, D)
    else:
        t = torch.tensor(_E4M3 + [math.nan], dtype=torch.float64, device=page.device)
        t = torch.cat([t, -t])
        scale = st[name + "_scale"][h].double()
        if case["pages"] == "fp8":
            page = page if name == "k" else page.permute(0, 2, 1)
            x = t[page.reshape(-1, D).long()] * scale
        else:
            codes = page[:, :8 * D].reshape(-1, D // 2).long()
            x = torch.empty((codes.shape[0], D), dtype=torch.float64, device=page.device)
            x[:, 0::2] = (codes % 16 - 8).double()
            x[:, 1::2] = (codes // 16 - 8).double()
            unit = t[page[:, 8 * D:].reshape(-1, D // GROUP).long()] * scale
            for g in range(D // GROUP):
                x[:, g * GROUP:(g + 1) * GROUP] *= unit[:, g:g + 1]
    return x[:upto]


def _softmax64(st, case, b, h, keys, window=0):
    """[T, G, L] softmax weights of sequence b's query tokens over the L entries."""
    T, D = case["tokens"], case["dim"]
    G, L = case["q_heads"] // case["kv_heads"], keys.shape[0]
    q = st["q"][b, :, h * G:(h + 1) * G].double()
    s = torch.einsum("tgd,jd->tgj", q, keys) / D ** 0.5
    for t in range(T):
        last = L - T + t
        s[t, :, last + 1:] = -math.inf
        if window:
            s[t, :, :max(0, last - window + 1)] = -math.inf
    return torch.softmax(s, -1)


def exact(case, seed):
    st = prepare(case, seed)
    case, op, D = st["case"], st["case"]["op"], case["dim"]
    if op == "store":
        live = (st["slots"] >= 0)[:, None, None]
        return [_values64(st[n], st[s]) * live for n, s in (("key", "k_scale"),
                                                            ("value", "v_scale"))]
    lens = st["lens"].tolist()
    B, T, Hkv = case["batch"], case["tokens"], case["kv_heads"]
    G = case["q_heads"] // Hkv
    keep = {}
    if op == "evict":
        new_w, new_pos = st["weights0"].clone(), st["positions0"].clone()
        for b in range(B):
            for h in range(Hkv):
                n, k = lens[b], case["budget"]
                src = list(range(min(n, k)))
                if n > k:
                    w, pos = st["weights0"][b, h, :n].double(), st["positions0"][b, h, :n]
                    rank = torch.where(pos > pos.max() - case["recent"],
                                       torch.full_like(w, math.inf), w)   # the newest first
                    order = torch.argsort(-rank, stable=True)[:k]
                    mark = torch.zeros(n, dtype=torch.bool, device=DEV)
                    mark[order] = True
                    moved = (torch.nonzero(mark[k:]).flatten() + k).tolist()
                    holes = torch.nonzero(~mark[:k]).flatten().tolist()
                    for i, x in zip(holes, moved):
                        src[i] = x
                at = torch.tensor(src, device=DEV)
                keep[b, h] = at
                new_w[b, h, :len(src)] = st["weights0"][b, h][at]
                new_pos[b, h, :len(src)] = st["positions0"][b, h][at]
        new_lens = torch.tensor([min(n, case["budget"]) for n in lens], dtype=torch.int32,
                                device=DEV)
        if not case["step"]:
            # the cache itself is moved, not computed: nothing of it has a value in 64 bits
            if case["pages"] != "int4":
                return [new_lens, new_w.double(), new_pos, None, None]
            kept = []
            for name in ("k", "v"):
                x = torch.zeros((B, case["budget"], Hkv, D), dtype=torch.float64, device=DEV)
                for (b, h), at in keep.items():
                    x[b, :at.numel(), h] = _entries64(st, case, name, b, h, lens[b])[at]
                kept.append(x.flatten(0, 1))
            return [new_lens, new_w.double(), new_pos, *kept]
    out = torch.zeros((B, T, case["q_heads"], D), dtype=torch.float64, device=DEV)
    weights = (new_w if op == "evict" else st["weights"] if op == "observe" else out).double()
    fresh = {}
    if op != "observe" and "key" in st:
        fresh = {n: _values64(st[x], st[n + "_scale"]).view(B, T, Hkv, D)
                 for n, x in (("k", "key"), ("v", "value"))}
    for b in range(B):
        L = case["budget"] + 1 if op == "evict" else lens[b]
        for h in range(Hkv):
            kv = []
            for name in ("k", "v") if op != "observe" else ("k",):
                x = _entries64(st, case, name, b, h, lens[b])
                if op == "evict":
                    x = torch.cat([x[keep[b, h]], fresh[name][b, :, h]])
                elif fresh:
                    x[L - T:] = fresh[name][b, :, h]
                kv.append(x)
            p = _softmax64(st, case, b, h, kv[0], case.get("window", 0))
            if op != "observe":
                # entries that no query token sees may hold anything
                out[b, :, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", p, kv[1])
            if op != "attend":
                before = (new_w if op == "evict" else st["weights0"])[b, h, :L].double()
                before = before * (case.get("decay", 1.0))
                before[L - T:] = 0
                weights[b, h, :L] = before + p.sum((0, 1))
    if op == "attend":
        return out if not fresh else [out, *(fresh[n].reshape(B * T, Hkv, D)
                                             for n in ("k", "v"))]
    pos = (new_pos if op == "evict" else st["positions"]).clone()
    for b in range(B):
        L = case["budget"] + 1 if op == "evict" else lens[b]
        for t in range(T):
            pos[b, :, L - T + t] = int(st["seen"][b]) - T + t
    if op == "observe":
        return [weights, pos]
    return [new_lens + 1, out, weights, pos]
