"""Operators of a cache that takes less memory, as they are called, and their plain forms.

A cache held in 4 bits (rows quantised as they are appended, attention of the
last tokens over it), and a cache that is trimmed by what attention looked at
(the weights that the last tokens give to every slot, summed up, and the
eviction of the slots with the least). ``listed`` and ``draw`` give cases,
``prepare`` their inputs, ``run`` one pass (the plain form in elementary torch
operations, or, with ``own`` set, the framework's calls), ``work`` the bytes and
operations that a pass cannot do without, ``exact`` the results in 64 bits.

A cache is [pages, Hkv, page_size, row] (with a leading layer dimension where a
step takes every layer) under ``page_table`` int32 [rows, max_pages] (-1: no
page), or the static [rows, Hkv, slots, row]. A row in 4 bits is D/2 + 16 bytes:
four groups of D/4 features, each with 16 codes from its least value in steps of
its scale; the codes two a byte (the even feature in the low half; D = 64: the
bytes of groups 0 and 1, and of 2 and 3, by turns), then the four scales and the
four least values in fp16.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SCRATCH = 256 << 20  # bytes of the workspace that a serving program keeps per stream


# ---- cases --------------------------------------------------------------------

def _append(name=None, **kw):
    c = dict(op="append_q4", dtype="bf16", layers=1, B=8, Hkv=8, D=128, T=1, cap=1024, page=16, chosen=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _decode(name=None, **kw):
    c = dict(op="decode_q4", dtype="bf16", B=8, Hq=32, Hkv=8, D=128, T=1, cap=8192, page=16, lo=1, window=0, sinks=0)
    c.update(kw)
    return dict(c, name=name) if name else c


def _weights(name=None, **kw):
    c = dict(op="weights", dtype="bf16", q4=False, B=8, Hq=32, Hkv=8, D=128, T=1, cap=8192, page=16, lo=1, window=0,
             sinks=0)
    c.update(kw)
    return dict(c, name=name) if name else c


def _evict(name=None, **kw):
    c = dict(op="evict", dtype="bf16", layers=1, B=8, Hkv=8, D=128, cap=8192, page=16, lo=1, budget=2048, sinks=4,
             recent=256)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the step's token of a serving batch goes into every layer's 4-bit pages
        _append("append token 4-bit", layers=32, B=32),
        # a prompt's keys and values go into the 4-bit pages of one layer
        _append("append prompt 4-bit", B=4, T=8192, cap=16384, page=64),
        # one request's token over a 4-bit static cache of 8192 slots: latency alone
        _decode("decode one 4-bit", B=1, Hq=16, Hkv=2, D=64, page=0),
        # a serving batch over 4-bit pages, requests of any length up to 32768
        _decode("decode batch 4-bit", B=32, cap=32768),
        # a chain of drafted tokens, already appended, is checked over very long contexts
        _decode("decode chain 4-bit", B=4, T=8, cap=131072, page=64, lo=65536),
        # what a step's token looked at, in a batch of short requests over the static cache
        _weights("weights of a token", B=8, Hq=16, Hkv=2, D=64, page=0),
        # what the last 32 tokens of two long prompts looked at, before the first eviction
        _weights("weights of prompts", B=2, T=32, cap=32768, page=64, lo=16384),
        # what the step's tokens of a batch looked at, over 4-bit pages
        _weights("weights batch 4-bit", B=32, cap=32768, q4=True),
        # a long prompt of one layer is cut to what it will be served with
        _evict("evict one prompt", B=1, cap=32768, page=64, lo=32768, budget=4096),
        # a batch that has grown past its budget is cut back in a few layers
        _evict("evict batch", layers=4, B=16, budget=2048),
        # a static cache that has run full gives up a few slots, in every layer
        _evict("evict a few", layers=8, B=4, cap=1024, lo=1024, page=0, budget=960, recent=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append_q4", "decode_q4", "decode_q4", "decode_q4", "weights", "weights", "evict", "evict"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([0, 1, 8, 16, 16, 24, 32, 64, 128])
    if op == "append_q4":
        chosen = rng.random() < 0.4
        T = _log(rng, 1, 64) if chosen else _log(rng, 1, 4096)
        return _append(dtype=dtype, layers=rng.choice([1, 2, 8]) if T < 256 else 1, B=min(_log(rng, 1, 16), 16384 // T),
                       Hkv=Hkv, D=D, T=T, cap=T + _log(rng, 1, 512), page=page, chosen=chosen)
    if op in ("decode_q4", "weights"):
        cap = _log(rng, 1, 65536)
        T = min(cap, _log(rng, 1, 48), 100000000 // (cap * Hq))
        B = max(1, min(_log(rng, 1, 48), 262144 // cap, 100000000 // (cap * Hq * T)))
        kw = dict(dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, D=D, T=T, cap=cap, page=page,
                  window=rng.choice([0, 0, _log(rng, 1, 4096)]), sinks=rng.choice([0, 1, 4, 64]))
        return _decode(**kw) if op == "decode_q4" else _weights(q4=rng.random() < 0.4, **kw)
    cap = _log(rng, 32, 32768)
    budget = _log(rng, 16, cap)
    sinks = min(budget, rng.choice([0, 1, 4, 16]))
    layers = min(rng.choice([1, 2, 4]), max(1, 49152 // cap))
    return _evict(dtype=dtype, layers=layers, B=max(1, min(_log(rng, 1, 32), 49152 // (cap * layers))), Hkv=Hkv, D=D,
                  cap=cap, page=page, lo=rng.choice([1, cap // 2 + 1, cap]), budget=budget, sinks=sinks,
                  recent=rng.randint(0, budget - sinks))


# ---- a row in 4 bits --------------------------------------------------------------

def _quantise(x):
    """Rows [..., D] as records [..., D/2 + 16] of bytes. Every step is one operation in 32 bits."""
    D = x.shape[-1]
    x = x.float().unflatten(-1, (4, D // 4))
    least = x.amin(-1).clamp(-65504.0, 65504.0).half() + 0.0  # (+ 0: no negative zero)
    lo = least.float()
    scale = ((x.amax(-1) - lo) * (1.0 / 15.0)).clamp(0.0, 65504.0).half()
    step = scale.float()[..., None]
    code = torch.where(step > 0, (x - lo[..., None]) / step, torch.zeros_like(x)).round().clamp(0.0, 15.0)
    code = code.to(torch.uint8).unflatten(-1, (D // 8, 2))
    byte = code[..., 0] | (code[..., 1] << 4)  # [..., 4, D/8]
    if D == 64:
        byte = byte.unflatten(-2, (2, 2)).transpose(-1, -2)
    params = torch.cat([scale, least], -1).contiguous().view(torch.uint8)
    return torch.cat([byte.flatten(len(x.shape) - 2), params], -1)


def _values(rec, dtype=torch.float32):
    """What records [..., D/2 + 16] stand for, [..., D]."""
    H = rec.shape[-1] - 16
    byte, par = rec[..., :H], rec[..., H:].contiguous().view(torch.float16).to(dtype)
    byte = byte.unflatten(-1, (2, 8, 2)).transpose(-1, -2).flatten(-3, -2) if H == 32 else byte.unflatten(-1, (4, 16))
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).to(dtype)  # [..., 4, D/4]
    return (par[..., :4, None] * code + par[..., 4:, None]).flatten(-2)


# ---- inputs -------------------------------------------------------------------

def _dev():
    return torch.device("cuda")


def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=_dev(), dtype=torch.float32).to(dtype)


def _fill(gen, shape, dtype):
    """A large cache's values: bounded memory whatever its size."""
    return torch.empty(shape, device=_dev(), dtype=dtype).normal_(generator=gen)


def _records(gen, shape, D):
    """A large 4-bit cache [..., D/2 + 16]: quantised normal values, some features larger than the others."""
    out = torch.empty((math.prod(shape), D // 2 + 16), device=_dev(), dtype=torch.uint8)
    gain = torch.exp(torch.randn(D, generator=gen, device=_dev()) * 0.5)
    for at in range(0, out.shape[0], 1 << 18):
        n = min(1 << 18, out.shape[0] - at)
        out[at:at + n] = _quantise(_randn(gen, (n, D), torch.float32) * gain)
    return out.view(*shape, D // 2 + 16)


def _table(rng, lens, page, max_pages, pages):
    """A page table over a shuffled pool of `pages` pages: rows of ceil(len / page) of them, -1 behind."""
    order = list(range(pages))
    rng.shuffle(order)
    table, at = torch.full((len(lens), max(1, max_pages)), -1, dtype=torch.int32), 0
    for r, n in enumerate(lens):
        m = -(-n // page)
        table[r, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
        at += m
    return table


def prepare(case, seed):
    gen = torch.Generator(device=_dev()).manual_seed(seed)
    rng = random.Random(seed * 7919 + 17)
    op, dt, D, Hkv, B, cap, page = (case[x] for x in ("op", "dtype", "D", "Hkv", "B", "cap", "page"))
    dt, L = DTYPES[dt], case.get("layers", 1)
    s = dict(case, scale=1.0 / math.sqrt(D), scratch=torch.empty(SCRATCH, dtype=torch.uint8, device=_dev()))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=_dev())  # noqa: E731
    if op == "append_q4":
        lens = [rng.randint(0, cap - case["T"]) for _ in range(B)]
        held = [n + case["T"] for n in lens]
    else:
        lens = [rng.randint(case["lo"], cap) for _ in range(B)]
        held = lens
    if page:
        # (a pool that is an output has one size whatever the lengths)
        pages = (B * -(-cap // page) if op in ("append_q4", "evict") else sum(-(-n // page) for n in held)) + 3
        s["table"], shape = _table(rng, held, page, -(-cap // page), pages).to(_dev()), (pages, Hkv, page)
    else:
        s["table"], shape = None, (B, Hkv, cap)
    s["kv_len"] = i32(lens)
    if op == "append_q4":
        T = case["T"]
        rec = (L, *shape, D // 2 + 16)
        s["k"] = torch.randint(0, 256, rec, generator=gen, device=_dev(), dtype=torch.uint8)
        s["v"] = torch.randint(0, 256, rec, generator=gen, device=_dev(), dtype=torch.uint8)
        # the new keys and values as a projection leaves them: [L, B, T, Hkv, D]
        s["k_new"] = _randn(gen, (L, B, T, Hkv, D), dt).transpose(2, 3)
        s["v_new"] = _randn(gen, (L, B, T, Hkv, D), dt).transpose(2, 3)
        s["kv_len_out"] = torch.empty_like(s["kv_len"])
        s["index"] = s["count"] = None
        if case["chosen"]:  # an accepted path: ascending drafts, a few of them
            counts = [min(T, rng.choice([1, 2, 2, 3, 4, 5])) for _ in range(B)]
            paths = [sorted(rng.sample(range(T), c)) for c in counts]
            s["index"] = i32([p + [0] * (T - len(p)) for p in paths])
            s["count"] = i32(counts)
        return s
    if op == "evict":
        s["k"], s["v"] = _fill(gen, (L, *shape, D), dt), _fill(gen, (L, *shape, D), dt)
        # summed weights: a few slots have most of them, some have none
        w = torch.exp(torch.randn((L, B, Hkv, cap), generator=gen, device=_dev()) * 2.0 - 4.0)
        w = torch.where(torch.rand((L, B, Hkv, cap), generator=gen, device=_dev()) < 0.05, torch.zeros_like(w), w)
        s["weight"] = w * (torch.arange(cap, device=_dev()) < s["kv_len"][:, None, None])
        s["weight_out"] = s["weight"].clone()
        s["kv_len_out"] = torch.empty_like(s["kv_len"])
        return s
    Hq, T = case["Hq"], case["T"]
    s["q"] = _randn(gen, (B, Hq, T, D), dt)
    if op == "decode_q4":
        s["k"], s["v"] = _records(gen, shape, D), _records(gen, shape, D)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, Hq, T), dtype=torch.float32, device=_dev())
        return s
    s["k"] = _records(gen, shape, D) if case["q4"] else _fill(gen, (*shape, D), dt)
    s["weight"] = torch.rand((B, Hkv, cap), generator=gen, device=_dev(), dtype=torch.float32)
    # what the attention call over the same cache has left
    s["lse"] = torch.stack([torch.logsumexp(_scores(s, b), -1).reshape(Hq, T) for b in range(B)])
    return s


# ---- the plain forms ------------------------------------------------------------

def _cached(s, x, b):
    """All slots of request b of the cache x, [Hkv, cap, row] (any row where there is no page)."""
    if s["table"] is None:
        return x[b]
    ids = s["table"][b].clamp(min=0).long()
    return x[ids].transpose(0, 1).flatten(1, 2)[:, :s["cap"]]


def _scores(s, b):
    """Scores [Hkv, Hq/Hkv * T, cap] of request b's last T tokens in 32 bits, -inf where a slot is not seen."""
    Hq, T, D = s["q"].shape[1:]
    k = _cached(s, s["k"], b)
    k = _values(k) if k.dtype == torch.uint8 else k.float()
    sc = torch.matmul(s["q"][b].float().view(s["Hkv"], -1, D), k.transpose(1, 2)) * s["scale"]
    j = torch.arange(s["cap"], device=k.device)
    pos = (s["kv_len"][b] - T + torch.arange(T, device=k.device))[:, None]
    sees = j <= pos
    if s["window"]:
        sees = sees & ((pos - j < s["window"]) | (j < s["sinks"]))
    return sc.masked_fill(~sees.repeat(Hq // s["Hkv"], 1), -math.inf)


def _plain_decode(s):
    Hq, T, D = s["q"].shape[1:]
    for b in range(s["B"]):
        sc = _scores(s, b)
        m = sc.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        p = torch.exp(sc - m)
        l = p.sum(-1, keepdim=True)
        out = torch.matmul(p, _values(_cached(s, s["v"], b))) / torch.where(l > 0, l, torch.ones_like(l))
        s["out"][b] = out.view(Hq, T, D).to(s["out"].dtype)
        s["lse"][b] = (torch.log(l) + m).view(Hq, T)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_weights(s):
    Hq, T, _ = s["q"].shape[1:]
    for b in range(s["B"]):
        lse = s["lse"][b].reshape(s["Hkv"], -1, 1)
        p = torch.exp(_scores(s, b) - torch.where(lse == -math.inf, torch.zeros_like(lse), lse))
        s["weight"][b] += torch.where(lse == -math.inf, torch.zeros_like(p), p).sum(1)
    return {"weight": s["weight"]}


def _plain_append(s):
    L, B, Hkv, T, D = s["k_new"].shape
    t = torch.arange(T, device=s["k"].device)
    count = s["count"].long() if s["count"] is not None else torch.full((B,), T, device=s["k"].device)
    pick = s["index"].long() if s["index"] is not None else t.expand(B, T)
    b, t = torch.nonzero(t < count[:, None], as_tuple=True)
    pos = s["kv_len"].long()[b] + t
    row, slot = b, pos
    if s["table"] is not None:
        row, slot = s["table"].long()[b, pos // s["page"]], pos % s["page"]
    s["k"][:, row, :, slot] = _quantise(s["k_new"][:, b, :, pick[b, t]])
    s["v"][:, row, :, slot] = _quantise(s["v_new"][:, b, :, pick[b, t]])
    torch.add(s["kv_len"], count.int(), out=s["kv_len_out"])
    return {"k": s["k"], "v": s["v"], "kv_len": s["kv_len_out"]}


def _plain_evict(s):
    """Requests longer than the budget keep their first and their last slots and, of each head's others, those of the
    largest weight (of equal ones the first), in their order."""
    n, budget, cap = s["kv_len"], s["budget"], s["cap"]
    L, B, Hkv, _ = s["weight"].shape
    dev = n.device
    j = torch.arange(cap, device=dev)
    ln = n[:, None, None]
    w = torch.where((j < s["sinks"]) | (j >= ln - s["recent"]), torch.full((), math.inf, device=dev), s["weight"])
    w = torch.where(j < ln, w, torch.full((), -math.inf, device=dev))
    keep = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget].sort(-1).values
    over = ln > budget
    for b in torch.nonzero(n > budget).view(-1).tolist():
        h = torch.arange(Hkv, device=dev)[:, None]
        d = torch.arange(budget, device=dev)
        for layer in range(L):
            i = keep[layer, b]  # [Hkv, budget]
            row, slot, to, at = b, i, b, d
            if s["table"] is not None:
                t = s["table"][b].long()
                row, slot, to, at = t[i // s["page"]], i % s["page"], t[d // s["page"]], d % s["page"]
            for x in (s["k"][layer], s["v"][layer]):
                x[to, h, at] = x[row, h, slot]
    kept = torch.zeros_like(s["weight"])
    kept[..., :budget] = torch.gather(s["weight"], -1, keep)
    s["weight_out"].copy_(torch.where(over & (j < ln), kept, s["weight"]))
    torch.clamp(n, max=budget, out=s["kv_len_out"])
    return {"k": s["k"], "v": s["v"], "weight": s["weight_out"], "kv_len": s["kv_len_out"]}


# ---- one pass -------------------------------------------------------------------

def _own_run(s):
    import masked_gqa_attention_gb300 as M
    op = s["op"]
    if op == "append_q4":
        M.masked_gqa_cache_append_q4(s["k"], s["v"], s["k_new"], s["v_new"], s["kv_len"], s["kv_len_out"],
                                     index=s["index"], count=s["count"], page_table=s["table"])
        return {"k": s["k"], "v": s["v"], "kv_len": s["kv_len_out"]}
    if op == "decode_q4":
        M.masked_gqa_attn_decode_q4(s["q"], s["k"], s["v"], s["kv_len"], s["out"], window=s["window"],
                                    sinks=s["sinks"], page_table=s["table"], workspace=s["scratch"],
                                    scale=s["scale"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "weights":
        M.masked_gqa_attn_cache_weights(s["q"], s["k"], s["kv_len"], s["lse"], s["weight"], window=s["window"],
                                        sinks=s["sinks"], page_table=s["table"], scale=s["scale"])
        return {"weight": s["weight"]}
    M.masked_gqa_cache_evict(s["k"], s["v"], s["weight"], s["kv_len"], budget=s["budget"], sinks=s["sinks"],
                             recent=s["recent"], page_table=s["table"], weight_out=s["weight_out"],
                             kv_len_out=s["kv_len_out"], workspace=s["scratch"])
    return {"k": s["k"], "v": s["v"], "weight": s["weight_out"], "kv_len": s["kv_len_out"]}


_PLAIN = {"append_q4": _plain_append, "decode_q4": _plain_decode, "weights": _plain_weights, "evict": _plain_evict}


def run(state):
    return _own_run(state) if own else _PLAIN[state["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------

def _seen(case):
    """Means over the lengths: cached keys that some of the T queries sees, and (query, key) pairs."""
    lo, hi, T, W = case["lo"], case["cap"], case["T"], case["window"]
    num = min(256, hi - lo + 1)
    keys = pairs = 0.0
    for n in (lo + (hi - lo) * i // max(1, num - 1) for i in range(num)):
        first = max(0, n - T)
        a = max(0, first - W + 1) if W else 0
        keys += n - a + min(case["sinks"], a)
        for p in range(first, n):
            a = max(0, p - W + 1) if W else 0
            pairs += p + 1 - a + min(case["sinks"], a)
    return keys / num, pairs / num


def work(case):
    op, e, D, Hkv, B = case["op"], 4 if case["dtype"] == "fp32" else 2, case["D"], case["Hkv"], case["B"]
    rec = D // 2 + 16
    if op == "append_q4":
        rows = case["layers"] * Hkv * B * (min(case["T"], 17 / 6) if case["chosen"] else case["T"])
        return {"bytes": 2.0 * rows * (e * D + rec) + 8.0 * B, "flops": 0}
    if op in ("decode_q4", "weights"):
        keys, pairs = _seen(case)
        Hq, T = case["Hq"], case["T"]
        if op == "decode_q4":
            return {"bytes": B * (2.0 * rec * Hkv * keys + 2 * e * D * Hq * T + 4 * Hq * T),
                    "flops": 4.0 * D * B * Hq * pairs}
        row = rec if case["q4"] else e * D
        return {"bytes": B * ((row + 8.0) * Hkv * keys + e * D * Hq * T + 4 * Hq * T), "flops": 2.0 * D * B * Hq * pairs}
    lo, hi, budget = case["lo"], case["cap"], case["budget"]
    above = range(max(lo, budget + 1), hi + 1)
    share, mean = len(above) / (hi - lo + 1), (above[0] + above[-1]) / 2 if len(above) else 0
    # every kept row behind the first one that goes moves: of the middle, all but the share kept in a row at its front
    middle = budget - case["sinks"] - case["recent"]
    part = middle / max(1.0, mean - case["sinks"] - case["recent"])
    moved = max(0.0, budget - case["sinks"] - part / max(1e-9, 1 - part)) if part < 1 else 0.0
    heads = case["layers"] * B * Hkv * share
    return {"bytes": heads * (4.0 * e * D * moved + 8.0 * mean) + 8.0 * B, "flops": 0}


# ---- the results in 64 bits -------------------------------------------------------

def _rounded(x, t):
    return x.to(t).double()


def _exact_records(x):
    """The records of rows x [n, D]: the definition's steps in 64 bits, each rounded once to 32 (or to fp16)."""
    n, D = x.shape
    f32, f16 = torch.float32, torch.float16
    out = torch.zeros(n, D // 2 + 16, dtype=torch.uint8, device=x.device)
    par = torch.zeros(n, 8, dtype=f16, device=x.device)
    fifteenth = float(torch.tensor(1.0 / 15.0, dtype=f32))
    for g in range(4):
        y = x[:, g * (D // 4):(g + 1) * (D // 4)].double()
        lo = y.min(1).values.clamp(-65504, 65504)
        lo = _rounded(lo, f16)
        lo = torch.where(lo == 0, torch.zeros_like(lo), lo)
        sc = _rounded(_rounded(y.max(1).values - lo, f32) * fifteenth, f32).clamp(0, 65504)
        sc = _rounded(sc, f16)
        par[:, g], par[:, 4 + g] = sc.half(), lo.half()
        quot = _rounded(_rounded(y - lo[:, None], f32) / torch.where(sc > 0, sc, torch.ones_like(sc))[:, None], f32)
        code = torch.where(sc[:, None] > 0, torch.round(quot).clamp(0, 15), torch.zeros_like(quot)).to(torch.uint8)
        two = code[:, 0::2] + 16 * code[:, 1::2]
        at = slice(16 * g, 16 * g + 16) if D == 128 else slice(16 * (g // 2) + g % 2, 16 * (g // 2) + 16, 2)
        out[:, at] = two
    out[:, D // 2:] = par.view(torch.uint8)
    return out


def _exact_values(rec):
    """What records [n, D/2 + 16] stand for, in 64 bits."""
    D = 2 * (rec.shape[-1] - 16)
    par = rec[:, D // 2:].contiguous().view(torch.float16).double()
    x = torch.empty(rec.shape[0], D, dtype=torch.float64, device=rec.device)
    for g in range(4):
        at = slice(16 * g, 16 * g + 16) if D == 128 else slice(16 * (g // 2) + g % 2, 16 * (g // 2) + 16, 2)
        y = x[:, g * (D // 4):(g + 1) * (D // 4)]
        y[:, 0::2] = par[:, g, None] * (rec[:, at] % 16).double() + par[:, 4 + g, None]
        y[:, 1::2] = par[:, g, None] * (rec[:, at] // 16).double() + par[:, 4 + g, None]
    return x


def _exact_append(s):
    L, B, Hkv, T, D = s["k_new"].shape
    k, v = s["k"].clone(), s["v"].clone()
    lens = s["kv_len"].tolist()
    counts = s["count"].tolist() if s["count"] is not None else [T] * B
    for b in range(B):
        rows = s["index"][b, :counts[b]].long() if s["index"] is not None else torch.arange(counts[b], device=k.device)
        at = lens[b] + torch.arange(counts[b], device=k.device)
        page, slot = (b, at) if s["table"] is None else (s["table"][b].long()[at // s["page"]], at % s["page"])
        for layer in range(L):
            for g in range(Hkv):
                for to, new in ((k, s["k_new"]), (v, s["v_new"])):
                    to[layer, page, g, slot] = _exact_records(new[layer, b, g, rows])
    return {"k": k, "v": v, "kv_len": torch.tensor([a + c for a, c in zip(lens, counts)], dtype=torch.int32)}


def exact(case, seed):
    op = case["op"]
    if op == "evict" or work(case)["flops"] > 4e11 or case.get("layers", 1) * case["B"] * case["Hkv"] > 2048:
        return None  # (rows that are moved as they are; or a long calculation)
    s = prepare(case, seed)
    if op == "append_q4":
        return _exact_append(s)
    B, Hq, T, D = s["q"].shape
    Hkv, W, S, dev = s["Hkv"], s["window"], s["sinks"], s["q"].device
    r = Hq // Hkv
    out = torch.zeros(B, Hq, T, D, dtype=torch.float64, device=dev)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=dev)
    weight = s["weight"].double() if op == "weights" else None
    for b in range(B):
        n = int(s["kv_len"][b])
        j = torch.arange(n, device=dev)
        at = n - T + torch.arange(T, device=dev)
        ahead = at[:, None] - j
        vis = (ahead >= 0) & ((ahead < W) | (j < S) if W else ahead >= 0)
        page, slot = (b, j) if s["table"] is None else (s["table"][b].long()[j // s["page"]], j % s["page"])
        for g in range(Hkv):
            k = s["k"][page, g, slot]
            k = _exact_values(k) if k.dtype == torch.uint8 else k.double()
            v = _exact_values(s["v"][page, g, slot]) if op == "decode_q4" else None
            for h in range(g * r, (g + 1) * r):
                sc = s["q"][b, h].double() @ k.T * s["scale"]
                sc[~vis] = -math.inf
                if op == "weights":
                    have = s["lse"][b, h].double()[:, None]
                    p = torch.exp(sc - have)
                    weight[b, g, :n] += torch.where(have == -math.inf, torch.zeros_like(p), p).sum(0)
                else:
                    lse[b, h] = torch.logsumexp(sc, -1)
                    some = lse[b, h][:, None] > -math.inf
                    p = torch.where(some, torch.exp(sc - torch.where(some, lse[b, h][:, None], torch.zeros_like(sc))),
                                    torch.zeros_like(sc))
                    out[b, h] = p @ v
    return {"weight": weight} if op == "weights" else {"out": out, "lse": lse}
