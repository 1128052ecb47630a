"""The cache operators of a serving loop as they are called, and their plain forms.

Attention with a sliding window and sinks (whole sequences, and one token over
a cache), attention for a tree of drafted tokens over a cache, and the cache's
own steps: appending accepted rows, forking / freeing / reserving rows of pages,
and compacting the pages. ``listed`` and ``draw`` give cases, ``prepare`` their
inputs, ``run`` one pass (the plain form in elementary torch operations, or,
with ``own`` set, the framework's calls), ``work`` the bytes and operations that
a pass cannot do without, ``exact`` the attention results in 64 bits.

A cache is K and V as [pages, Hkv, page_size, D] (with a leading layer dimension
for the steps that move every layer) and ``page_table`` int32 [rows, max_pages]
(-1: no page); without a table it is the static [rows, Hkv, slots, D].
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SCRATCH = 256 << 20  # bytes of the workspace that a serving program keeps per stream


# ---- cases --------------------------------------------------------------------

def _prefill(name=None, **kw):
    c = dict(op="prefill_window", dtype="bf16", B=1, Hq=16, Hkv=8, D=128, Lq=1024, Lk=1024, window=256, sinks=4,
             causal=True, padded=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _decode(name=None, **kw):
    c = dict(op="decode_window", dtype="bf16", B=8, Hq=16, Hkv=2, D=64, cap=8192, page=0, window=1024, sinks=4)
    c.update(kw)
    return dict(c, name=name) if name else c


def _tree(name=None, **kw):
    c = dict(op="decode_tree", dtype="bf16", B=8, Hq=32, Hkv=8, D=128, T=16, cap=8192, page=16, lo=1, window=0,
             sinks=0, ragged=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _append(name=None, **kw):
    c = dict(op="cache_append", dtype="bf16", layers=1, B=8, Hkv=8, D=128, T=8, cap=1024, page=16, chosen=True)
    c.update(kw)
    return dict(c, name=name) if name else c


def _fork(name=None, **kw):
    c = dict(op="cache_fork", dtype="bf16", layers=4, rows=64, n=16, Hkv=8, D=128, page=16, cap=1024, extra=8)
    c.update(kw)
    return dict(c, name=name) if name else c


def _compact(name=None, **kw):
    c = dict(op="cache_compact", dtype="bf16", layers=4, rows=64, pages=1024, Hkv=8, D=128, page=16, used=0.4)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # two guidance rows (1000 keys, and 384 padded to that length) through a windowed decoder: a short call
        _prefill("prefill padded 1000", B=2, Lq=1000, Lk=1000, window=256, padded=True),
        # a long prompt through a windowed layer
        _prefill("prefill long 32768", Hq=32, Lq=32768, Lk=32768, window=4096),
        # one request's token over the static 8192-slot cache: latency alone
        _decode("decode one static", B=1),
        # a full serving batch over pages, rows of any length up to 32768
        _decode("decode batch paged", B=64, Hq=32, Hkv=8, D=128, cap=32768, page=16, window=4096),
        # one request verifies a few drafts
        _tree("tree of 8", B=1, Hq=16, Hkv=2, D=64, T=8, cap=4096, dtype="fp16"),
        # a batch with ragged trees, as a draft model proposes them
        _tree("trees ragged batch", B=16, T=24, cap=8192, page=64, ragged=True),
        # large trees over very long contexts
        _tree("trees of 61 long", B=4, T=61, cap=131072, page=64, lo=65536),
        # the accepted drafts of a step go into every layer's cache
        _append("append accepted", layers=32, B=8, T=8),
        # a prompt's keys and values go into the pages of one layer
        _append("append prompt", B=4, T=8192, cap=16384, page=64, chosen=False),
        # a few samples continue from one prompt
        _fork("fork few", rows=16, n=4, cap=512),
        # beams of a full batch are reordered and finished ones are freed
        _fork("fork batch", rows=256, n=128, page=64),
        # a fragmented pool is packed to its low end
        _compact("compact pool", rows=256, pages=4096, page=32, used=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill_window", "decode_window", "decode_tree", "decode_tree", "cache_append", "cache_fork",
                     "cache_compact"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    if op == "prefill_window":
        L = _log(rng, 1, 4096 if dtype == "fp32" else 16384)
        Lq = L if rng.random() < 0.6 else rng.randint(1, L)
        return _prefill(dtype=dtype, B=rng.randint(1, 2), Hq=min(Hq, 16) // Hkv * Hkv or Hkv, Hkv=Hkv, D=D, Lq=Lq,
                        Lk=L, window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 130]),
                        causal=rng.random() < 0.8, padded=rng.random() < 0.3)
    if op == "decode_window":
        cap = _log(rng, 1, 32768)
        return _decode(dtype=dtype, B=_log(rng, 1, 48), Hq=Hq, Hkv=Hkv, D=D, cap=cap, page=rng.choice([0, page]),
                       window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 64]))
    if op == "decode_tree":
        cap = _log(rng, 128, 65536)
        B = max(1, min(_log(rng, 1, 32), 262144 // cap))
        return _tree(dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, D=D, T=_log(rng, 1, 64), cap=cap, page=rng.choice([0, page]),
                     lo=0, window=rng.choice([0, 0, _log(rng, 1, 4096)]), sinks=rng.choice([0, 4]),
                     ragged=rng.random() < 0.5)
    if op == "cache_append":
        chosen = rng.random() < 0.5
        T = _log(rng, 1, 64) if chosen else _log(rng, 1, 4096)
        return _append(dtype=dtype, layers=rng.choice([1, 2, 8]), B=_log(rng, 1, 16), Hkv=Hkv, D=D, T=T,
                       cap=T + _log(rng, 1, 512), page=rng.choice([0, page]), chosen=chosen)
    if op == "cache_fork":
        rows = _log(rng, 4, 256)
        return _fork(dtype=dtype, layers=rng.choice([1, 2, 4]), rows=rows, n=rng.randint(1, rows // 2), Hkv=Hkv, D=D,
                     page=page, cap=_log(rng, 16, 700), extra=rng.choice([0, 1, 40]))
    return _compact(dtype=dtype, layers=rng.choice([1, 2, 4]), rows=_log(rng, 1, 128), pages=_log(rng, 16, 4096),
                    Hkv=Hkv, D=D, page=min(page, 32), used=rng.choice([0.1, 0.4, 0.8, 1.0]))


# ---- inputs -------------------------------------------------------------------

def _dev():
    return torch.device("cuda")


def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=_dev(), dtype=torch.float32).to(dtype)


def _fill(gen, shape, dtype):
    """A large cache's values: bounded memory whatever its size."""
    x = torch.empty(shape, device=_dev(), dtype=dtype)
    return x.normal_(generator=gen)


def _pages_for(rng, lens, page, max_pages, pages):
    """A page table over a shuffled pool of `pages` pages: rows of ceil(len / page) of them, -1 behind."""
    need = [-(-n // page) for n in lens]
    order = list(range(pages))
    rng.shuffle(order)
    table, at = torch.full((len(lens), max(1, max_pages)), -1, dtype=torch.int32), 0
    for r, m in enumerate(need):
        table[r, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
        at += m
    return table


def _lens(case, rng, lo, hi):
    return [rng.randint(lo, hi) for _ in range(case["B"])]


def _tree_of(rng, T):
    """Ancestor masks of a random tree in its order of drafting: bit s of word row t is set where t sees s."""
    rows = []
    for t in range(T):
        parent = rng.randint(max(-1, t - 6), t - 1)
        rows.append((rows[parent] if parent >= 0 else 0) | (1 << t))
    W = -(-T // 32)
    words = [[(r >> (32 * w)) & 0xFFFFFFFF for w in range(W)] for r in rows]
    return [[x - (1 << 32) if x >= 1 << 31 else x for x in row] for row in words]


def prepare(case, seed):
    gen = torch.Generator(device=_dev()).manual_seed(seed)
    rng = random.Random(seed * 7919 + 13)
    op, dt, D, Hkv = case["op"], DTYPES[case["dtype"]], case["D"], case["Hkv"]
    s = dict(case, scale=1.0 / math.sqrt(D), scratch=torch.empty(SCRATCH, dtype=torch.uint8, device=_dev()))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=_dev())  # noqa: E731
    if op == "prefill_window":
        B, Hq, Lq, Lk = case["B"], case["Hq"], case["Lq"], case["Lk"]
        s["q"] = _randn(gen, (B, Hq, Lq, D), dt)
        s["k"] = _randn(gen, (B, Hkv, Lk, D), dt)
        s["v"] = _randn(gen, (B, Hkv, Lk, D), dt)
        s["kv_len"] = i32([Lk] + [max(1, (Lk * 3) // 8)] * (B - 1)) if case["padded"] else None
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, Hq, Lq), dtype=torch.float32, device=_dev())
        return s
    page = case.get("page", 0)
    if op in ("decode_window", "decode_tree"):
        B, Hq, cap = case["B"], case["Hq"], case["cap"]
        T = case.get("T", 1)
        hi = cap if op == "decode_window" else max(0, cap - T)
        lens = _lens(case, rng, min(case.get("lo", 1), hi), hi)
        if page:
            mp = -(-cap // page)
            held = [n + (T if op == "decode_tree" else 0) for n in lens]
            pages = sum(-(-n // page) for n in held) + 3
            s["table"] = _pages_for(rng, held, page, mp, pages).to(_dev())
            shape = (pages, Hkv, page, D)
        else:
            s["table"], shape = None, (B, Hkv, cap, D)
        s["k"], s["v"] = _fill(gen, shape, dt), _fill(gen, shape, dt)
        s["kv_len"] = i32(lens)
        s["q"] = _randn(gen, (B, Hq, T, D), dt)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, Hq, T), dtype=torch.float32, device=_dev())
        if op == "decode_tree":
            # the drafts' keys and values as a projection leaves them: [B, T, Hkv, D]
            s["k_new"] = _randn(gen, (B, T, Hkv, D), dt).transpose(1, 2)
            s["v_new"] = _randn(gen, (B, T, Hkv, D), dt).transpose(1, 2)
            s["bits"] = i32([_tree_of(rng, T) for _ in range(B)])
            s["tree_len"] = i32([rng.randint(1, T) for _ in range(B)]) if case["ragged"] else None
        return s
    L = case["layers"]
    if op == "cache_append":
        B, T, cap = case["B"], case["T"], case["cap"]
        lens = _lens(case, rng, 0, cap - T)
        if page:
            mp = -(-cap // page)
            pages = B * mp + 3
            s["table"] = _pages_for(rng, [n + T for n in lens], page, mp, pages).to(_dev())
            shape = (L, pages, Hkv, page, D)
        else:
            s["table"], shape = None, (L, B, Hkv, cap, D)
        s["k"], s["v"] = _fill(gen, shape, dt), _fill(gen, shape, dt)
        s["k_new"] = _randn(gen, (L, B, T, Hkv, D), dt).transpose(2, 3)
        s["v_new"] = _randn(gen, (L, B, T, Hkv, D), dt).transpose(2, 3)
        s["kv_len"] = i32(lens)
        s["kv_len_out"] = torch.empty_like(s["kv_len"])
        s["index"] = s["count"] = None
        if case["chosen"]:  # an accepted path: ascending drafts, a few of them
            counts = [min(T, rng.choice([1, 2, 2, 3, 4, 5])) for _ in range(B)]
            paths = [sorted(rng.sample(range(T), c)) for c in counts]
            s["index"] = i32([p + [0] * (T - len(p)) for p in paths])
            s["count"] = i32(counts)
        return s
    if op == "cache_fork":
        rows, n, cap = case["rows"], case["n"], case["cap"]
        order = list(range(rows))
        rng.shuffle(order)
        dst, rest = order[:n], order[n:]
        lens = [0] * rows
        for r in order:
            lens[r] = rng.randint(0, cap) if r in rest or rng.random() < 0.5 else 0
        mp = -(-(cap + case["extra"]) // page) + 1
        pages = rows * -(-cap // page) + n * (2 + -(-case["extra"] // page))
        table = _pages_for(rng, lens, page, mp, pages)
        ref = torch.zeros(pages, dtype=torch.int32)
        ref[table[table >= 0].long()] = 1
        s["table"], s["ref"], s["kv_len"] = table.to(_dev()), ref.to(_dev()), i32(lens)
        s["src"] = i32([-1 if rng.random() < 0.1 else rng.choice(rest) for _ in dst])
        s["dst"] = i32(dst)
        shape = (L, pages, Hkv, page, D)
        s["k"], s["v"] = _fill(gen, shape, dt), _fill(gen, shape, dt)
        return s
    pages, rows = case["pages"], case["rows"]
    held = sorted(rng.sample(range(pages), max(0, min(pages, int(case["used"] * pages)))))
    rng.shuffle(held)
    mp = -(-len(held) // rows) + 2
    table = torch.full((rows, mp), -1, dtype=torch.int32)
    ref = torch.zeros(pages, dtype=torch.int32)
    for i, p in enumerate(held):
        table[i % rows, i // rows] = p
        ref[p] = 1
    if rows > 1 and held:  # a forked row shares the first row's pages
        table[rows - 1] = table[0]
        ref.zero_()
        ref.index_add_(0, table[table >= 0].long(), torch.ones(int((table >= 0).sum()), dtype=torch.int32))
    s["table"], s["ref"] = table.to(_dev()), ref.to(_dev())
    s["table_out"], s["ref_out"] = torch.empty_like(s["table"]), torch.empty_like(s["ref"])
    shape = (L, pages, Hkv, page, D)
    s["k"], s["v"] = _fill(gen, shape, dt), _fill(gen, shape, dt)
    return s


# ---- the plain forms ------------------------------------------------------------

def _softmax_values(sc, vis, v):
    """(out, lse) of scores sc with the visible keys vis, over the last axis; rows that see nothing: 0, -inf."""
    sc = sc.masked_fill(~vis, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(sc - m0)
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    return out, (torch.log(l) + m0).squeeze(-1)


def _plain_prefill(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    B, Hq, Lq, D = q.shape
    Hkv, Lk, W, S = k.shape[1], k.shape[2], s["window"], min(s["sinks"], k.shape[2])
    dev, r = q.device, Hq // Hkv
    blk = min(1024, Lq)
    nb = -(-Lq // blk)
    back = min(W - 1, Lk)
    span = min(Lk, blk + back + (0 if s["causal"] else min(W - 1, Lk)))
    first = (torch.arange(nb, device=dev) * blk + (Lk - Lq) - back).clamp(0, Lk - span)
    at = torch.cat([torch.arange(S, device=dev).expand(nb, S), first[:, None] + torch.arange(span, device=dev)], 1)
    pos = (torch.arange(nb * blk, device=dev) + (Lk - Lq)).view(nb, blk)
    kb, vb = k[:, :, at], v[:, :, at]  # [B, Hkv, nb, S + span, D]
    qb = torch.nn.functional.pad(q, (0, 0, 0, nb * blk - Lq)).view(B, Hkv, r, nb, blk, D)
    sc = torch.matmul(qb, kb.unsqueeze(2).transpose(-1, -2)) * s["scale"]
    d = pos[:, :, None] - at[:, None, :]
    vis = (d < W) & (d >= 0 if s["causal"] else d > -W)
    sink = torch.zeros(S + span, dtype=torch.bool, device=dev)
    sink[:S] = True
    vis = torch.where(sink, (d >= 0) if s["causal"] else torch.ones_like(vis), vis & (at >= S)[:, None, :])
    vis = vis.expand(B, 1, 1, nb, blk, S + span)
    if s["kv_len"] is not None:
        vis = vis & (at[None] < s["kv_len"][:, None, None])[:, None, None, :, None, :]
    out, lse = _softmax_values(sc, vis, vb.unsqueeze(2))
    out = out.reshape(B, Hq, nb * blk, D)[:, :, :Lq]
    return {"out": out.to(s["q"].dtype), "lse": lse.reshape(B, Hq, nb * blk)[:, :, :Lq]}


def _slots(s, x, pos):
    """Rows pos [B, n] of the cache x, as [B, Hkv, n, D] in 32 bits (any row where pos has no page)."""
    if s["table"] is None:
        b = torch.arange(pos.shape[0], device=pos.device)[:, None]
        return x[b, :, pos].transpose(1, 2).float()
    page = x.shape[2]
    held = torch.gather(s["table"].long(), 1, pos // page).clamp(min=0)
    return x[held, :, pos % page].transpose(1, 2).float()


def _visible_slots(s, last):
    """Positions [B, n] of the cache that some query may see and whether each counts; last: [B] positions whose
    window reaches furthest back."""
    W, S, cap = s["window"], s["sinks"], s["cap"]
    dev = s["kv_len"].device
    if W == 0 or W + S >= cap:
        pos = torch.arange(cap, device=dev).expand(s["B"], cap)
        return pos, pos < s["kv_len"][:, None]
    n = torch.arange(S + W, device=dev)
    pos = torch.where(n < S, n, last[:, None].long() - W + 1 + (n - S))
    ok = ((n < S) | (pos >= S)) & (pos >= 0) & (pos < s["kv_len"][:, None])
    return pos.clamp(0, cap - 1), ok


def _plain_decode(s):
    B, Hq, T, D = s["q"].shape
    Hkv = s["Hkv"]
    last = s["kv_len"] - 1
    pos, ok = _visible_slots(s, last)
    ok = ok & ((last[:, None] - pos < s["window"]) | (pos < s["sinks"]))
    k, v = _slots(s, s["k"], pos), _slots(s, s["v"], pos)
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    sc = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    out, lse = _softmax_values(sc, ok[:, None, None, :], v)
    return {"out": out.view(B, Hq, 1, D).to(s["q"].dtype), "lse": lse.view(B, Hq, 1)}


def _tree_sees(bits, T, tree_len):
    """[B, T, T] which drafts each draft sees, and its depth [B, T]."""
    n = torch.arange(T, device=bits.device)
    sees = (bits.long()[:, :, n // 32] >> (n % 32)) & 1 == 1
    if tree_len is not None:
        live = n < tree_len[:, None]
        sees = sees & live[:, None, :] & live[:, :, None]
    eye = torch.eye(T, dtype=torch.bool, device=bits.device)
    return sees, (sees & ~eye).sum(-1)


def _plain_tree(s):
    B, Hq, T, D = s["q"].shape
    Hkv, r, W, S = s["Hkv"], Hq // s["Hkv"], s["window"], s["sinks"]
    sees, depth = _tree_sees(s["bits"], T, s["tree_len"])
    at = s["kv_len"][:, None].long() + depth  # positions of the drafts
    pos, ok = _visible_slots(s, s["kv_len"])
    ok = ok[:, None, :].expand(B, T, pos.shape[1])
    if W:
        ok = ok & ((at[:, :, None] - pos[:, None, :] < W) | (pos < S)[:, None, :])
        sees = sees & ((at[:, :, None] - at[:, None, :] < W) | (at < S)[:, None, :])
    if s["tree_len"] is not None:
        ok = ok & (torch.arange(T, device=pos.device) < s["tree_len"][:, None])[:, :, None]
    k = torch.cat([_slots(s, s["k"], pos), s["k_new"].float()], 2)
    v = torch.cat([_slots(s, s["v"], pos), s["v_new"].float()], 2)
    q = s["q"].float().view(B, Hkv, r * T, D)
    sc = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    vis = torch.cat([ok, sees], 2)[:, None, None].expand(B, Hkv, r, T, k.shape[2]).reshape(B, Hkv, r * T, -1)
    out, lse = _softmax_values(sc, vis, v)
    return {"out": out.view(B, Hq, T, D).to(s["q"].dtype), "lse": lse.view(B, Hq, T)}


def _plain_append(s):
    L, B, Hkv, T, D = s["k_new"].shape
    dev = s["k"].device
    t = torch.arange(T, device=dev)
    count = s["count"].long() if s["count"] is not None else torch.full((B,), T, device=dev)
    pick = s["index"].long() if s["index"] is not None else t.expand(B, T)
    b, t = torch.nonzero(t < count[:, None], as_tuple=True)
    pos = s["kv_len"].long()[b] + t
    if s["table"] is None:
        row, slot = b, pos
    else:
        page = s["k"].shape[3]
        row, slot = s["table"].long()[b, pos // page], pos % page
    s["k"][:, row, :, slot] = s["k_new"][:, b, :, pick[b, t]]
    s["v"][:, row, :, slot] = s["v_new"][:, b, :, pick[b, t]]
    torch.add(s["kv_len"], count.int(), out=s["kv_len_out"])
    return {"k": s["k"], "v": s["v"], "kv_len": s["kv_len_out"]}


def _plain_fork(s):
    """dst rows release their pages and take over src's: full pages shared, the last one copied to a fresh page, and
    fresh pages up to `extra` more tokens; fresh pages are the lowest free ones in the order of the pairs."""
    table, ref, lens, ps = s["table"], s["ref"], s["kv_len"], s["page"]
    src, dst = s["src"].long(), s["dst"].long()
    n, mp = src.shape[0], table.shape[1]
    j = torch.arange(mp, device=table.device)
    held = table[dst]
    one = torch.ones((), dtype=torch.int32, device=table.device)
    ref.index_add_(0, held.clamp(min=0).view(-1).long(), -(held >= 0).int().view(-1))
    from_ = torch.where((src >= 0)[:, None], table[src.clamp(min=0)], -one)
    ln = torch.where(src >= 0, lens[src.clamp(min=0)], 0 * one)
    full = (ln // ps)[:, None]
    shared = j < full
    ref.index_add_(0, from_.clamp(min=0).view(-1).long(), shared.int().view(-1))
    part = (j == full) & (ln % ps > 0)[:, None]  # the page that is copied
    free = ref == 0
    free[from_[part].long()] = False
    fresh = (j >= full) & (j * ps < (ln + s["extra"])[:, None]) & (src >= 0)[:, None]
    got = torch.nonzero(free).view(-1)[: int(fresh.sum())]
    new = torch.where(shared, from_, -one)
    new[fresh] = got.int()
    ref[got] = 1
    table[dst], lens[dst] = new, ln
    i, c = torch.nonzero(part, as_tuple=True)
    keep = torch.arange(ps, device=table.device) < (ln[i] % ps)[:, None]  # slots of each copied page
    p, o = torch.nonzero(keep, as_tuple=True)
    a, b = from_[i, c].long()[p], new[i, c].long()[p]
    s["k"][:, b, :, o] = s["k"][:, a, :, o]
    s["v"][:, b, :, o] = s["v"][:, a, :, o]
    return {"k": s["k"], "v": s["v"], "table": table, "kv_len": lens, "ref": ref}


def _plain_compact(s):
    """The used pages behind the first `used` ones move, in order, to the free pages among those."""
    used = s["ref"] > 0
    n = used.sum()
    at = torch.arange(used.shape[0], device=used.device)
    src, dst = torch.nonzero(used & (at >= n)).view(-1), torch.nonzero(~used & (at < n)).view(-1)
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    to = at.int()
    to[src] = dst.int()
    s["ref_out"].copy_(s["ref"])
    s["ref_out"][dst] = s["ref"][src]
    s["ref_out"][src] = 0
    s["table_out"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()], s["table"]))
    return {"k": s["k"], "v": s["v"], "table": s["table_out"], "ref": s["ref_out"]}


# ---- one pass -------------------------------------------------------------------

def _own_run(s):
    import masked_gqa_attention_gb300 as M
    op = s["op"]
    if op == "prefill_window":
        M.masked_gqa_attn_prefill_window(s["q"], s["k"], s["v"], s["out"], window=s["window"], sinks=s["sinks"],
                                         causal=s["causal"], scale=s["scale"], kv_len=s["kv_len"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "decode_window":
        M.masked_gqa_attn_decode_window(s["q"], s["k"], s["v"], s["kv_len"], s["out"], window=s["window"],
                                        sinks=s["sinks"], page_table=s["table"], workspace=s["scratch"],
                                        scale=s["scale"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "decode_tree":
        M.masked_gqa_attn_decode_tree(s["q"], s["k"], s["v"], s["k_new"], s["v_new"], s["kv_len"], s["out"],
                                      tree_bits=s["bits"], tree_len=s["tree_len"], window=s["window"],
                                      sinks=s["sinks"], page_table=s["table"], workspace=s["scratch"],
                                      scale=s["scale"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "cache_append":
        M.masked_gqa_cache_append(s["k"], s["v"], s["k_new"], s["v_new"], s["kv_len"], s["kv_len_out"],
                                  index=s["index"], count=s["count"], page_table=s["table"])
        return {"k": s["k"], "v": s["v"], "kv_len": s["kv_len_out"]}
    if op == "cache_fork":
        M.masked_gqa_cache_fork(s["k"], s["v"], s["table"], s["kv_len"], s["ref"], s["src"], s["dst"],
                                extra=s["extra"], workspace=s["scratch"])
        return {"k": s["k"], "v": s["v"], "table": s["table"], "kv_len": s["kv_len"], "ref": s["ref"]}
    M.masked_gqa_cache_compact(s["k"], s["v"], s["table"], s["ref"], s["table_out"], s["ref_out"],
                               workspace=s["scratch"])
    return {"k": s["k"], "v": s["v"], "table": s["table_out"], "ref": s["ref_out"]}


_PLAIN = {"prefill_window": _plain_prefill, "decode_window": _plain_decode, "decode_tree": _plain_tree,
          "cache_append": _plain_append, "cache_fork": _plain_fork, "cache_compact": _plain_compact}


def run(state):
    return _own_run(state) if own else _PLAIN[state["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------

def _expected_visible(lo, hi, window, sinks):
    """Mean number of cached keys that a query behind a uniformly drawn length in [lo, hi] sees."""
    n = min(256, hi - lo + 1)
    ls = [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]
    return sum(L if window == 0 else min(L, window + min(sinks, max(0, L - window))) for L in ls) / n


def work(case):
    op, e = case["op"], 4 if case["dtype"] == "fp32" else 2
    D, Hkv = case["D"], case["Hkv"]
    if op == "prefill_window":
        B, Hq, Lq, Lk, W, S = case["B"], case["Hq"], case["Lq"], case["Lk"], case["window"], case["sinks"]
        kvl = [Lk] + [max(1, Lk * 3 // 8) if case["padded"] else Lk] * (B - 1)
        pairs, keys = 0, 0
        for n in sorted(set(kvl)):
            step = max(1, Lq // 4096)
            seen = 0
            for i in range(0, Lq, step):
                p = i + Lk - Lq
                a, b = max(0, p - W + 1), min(n, (p if case["causal"] else p + W - 1) + 1)
                top = min(n, p + 1) if case["causal"] else n
                seen += max(0, b - a) + max(0, min(S, a, top))
            pairs += kvl.count(n) * seen * Lq // len(range(0, Lq, step))
            a = max(0, Lk - Lq - W + 1)
            keys += kvl.count(n) * (max(0, n - a) + min(S, a, n))
        return {"bytes": e * D * (2 * B * Hq * Lq + 2 * Hkv * keys) + 4 * B * Hq * Lq, "flops": 4.0 * D * Hq * pairs}
    if op in ("decode_window", "decode_tree"):
        B, Hq, T = case["B"], case["Hq"], case.get("T", 1)
        hi = case["cap"] if op == "decode_window" else max(0, case["cap"] - T)
        seen = _expected_visible(min(case.get("lo", 1), hi), hi, case["window"], case["sinks"])
        live = (T + 1) / 2 if case.get("ragged") else T
        new = live if op == "decode_tree" else 0
        io = 2 * e * D * B * Hq * T + 2 * e * D * B * Hkv * new
        return {"bytes": io + 2 * e * D * B * Hkv * seen, "flops": 4.0 * D * B * Hq * live * (seen + new / 3)}
    if op == "cache_append":
        rows = case["B"] * (min(case["T"], 17 / 6) if case["chosen"] else case["T"])
        return {"bytes": 4.0 * e * D * Hkv * case["layers"] * rows, "flops": 0}
    if op == "cache_fork":
        ps = case["page"]
        mean = sum(n % ps for n in range(case["cap"] + 1)) / (case["cap"] + 1)
        meta = 12.0 * case["n"] * (-(-case["cap"] // ps))
        return {"bytes": 4.0 * e * D * Hkv * case["layers"] * 0.9 * case["n"] * mean + meta, "flops": 0}
    used, pages = max(0, min(case["pages"], int(case["used"] * case["pages"]))), case["pages"]
    moved = used * (1 - used / pages)
    return {"bytes": 4.0 * e * D * Hkv * case["layers"] * case["page"] * moved + 8.0 * (pages + used), "flops": 0}


# ---- the attention results in 64 bits ---------------------------------------------

def _exact_rows(q, k, v, vis, scale):
    """q [R, D] against k, v [n, D] where vis [R, n], in 64 bits."""
    sc = (q.double() @ k.double().T) * scale
    sc[~vis] = -math.inf
    lse = torch.logsumexp(sc, -1)
    p = torch.exp(sc - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None])
    return p @ v.double(), lse


def _exact_cached(s, x, b, n):
    """Slots [0, n) of row b of the cache x, [Hkv, n, D]."""
    if s["table"] is None:
        return x[b, :, :n]
    page = x.shape[2]
    ids = s["table"][b, : -(-n // page)].clamp(min=0).long()
    return x[ids].transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :n]


def exact(case, seed):
    op = case["op"]
    if op not in ("prefill_window", "decode_window", "decode_tree"):
        return None  # rows that are moved as they are, and whole numbers
    if work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    q = s["q"]
    B, Hq, Lq, D = q.shape
    r, W, S, dev = Hq // s["Hkv"], s["window"], s["sinks"], q.device
    out = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=dev)
    for b in range(B):
        n = int(s["kv_len"][b]) if s["kv_len"] is not None else case["Lk"]
        if op == "prefill_window":
            for i0 in range(0, Lq, 2048):
                p = torch.arange(i0, min(Lq, i0 + 2048), device=dev) + case["Lk"] - Lq
                a = max(0, int(p[0]) - W + 1)
                z = min(n, int(p[-1]) + (1 if case["causal"] else W))
                j = torch.cat([torch.arange(min(S, a, n), device=dev), torch.arange(a, max(a, z), device=dev)])
                if not case["causal"] and max(a, z) < min(S, n):  # sinks ahead of the band
                    j = torch.cat([j, torch.arange(max(a, z), min(S, n), device=dev)])
                if j.numel() == 0:
                    continue
                near = (p[:, None] - j < W) & (p[:, None] - j > -W)
                vis = near | (j < S)
                if case["causal"]:
                    vis &= j <= p[:, None]
                for h in range(Hq):
                    o, l = _exact_rows(q[b, h, i0:i0 + 2048], s["k"][b, h // r, j], s["v"][b, h // r, j], vis,
                                       s["scale"])
                    out[b, h, i0:i0 + 2048], lse[b, h, i0:i0 + 2048] = o, l
            continue
        k, v = _exact_cached(s, s["k"], b, n), _exact_cached(s, s["v"], b, n)
        j = torch.arange(n, device=dev)
        if op == "decode_window":
            vis = ((n - 1 - j < W) | (j < S))[None].expand(1, n)
        else:
            live = int(s["tree_len"][b]) if s["tree_len"] is not None else Lq
            t = torch.arange(Lq, device=dev)
            words = s["bits"][b].long() & 0xFFFFFFFF
            seen = torch.stack([(words[:, x // 32] >> (x % 32)) & 1 for x in range(Lq)], 1).bool()
            seen &= (t < live) & (t < live)[:, None]
            p = n + seen.sum(1) - seen.diagonal().int()
            vis = (t < live)[:, None].expand(Lq, n)
            if W:
                vis = vis & ((p[:, None] - j < W) | (j < S))
                seen &= (p[:, None] - p < W) | (p < S)
            vis = torch.cat([vis, seen], 1)
            k, v = torch.cat([k, s["k_new"][b]], 1), torch.cat([v, s["v_new"][b]], 1)
        for h in range(Hq):
            if k.shape[1]:
                out[b, h], lse[b, h] = _exact_rows(q[b, h], k[h // r], v[h // r], vis, s["scale"])
    return {"out": out, "lse": lse}
