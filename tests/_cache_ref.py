"""64-bit references of the windowed, tree and cache operators, with error
bounds derived from the types, and a sequential model of the page bookkeeping.

Bound of an attention output: with h = eps / 2 of the type (0 for the weights
of the fp32 path), weights are rounded by at most h relative (they are an
operand of the second product), the result by at most h relative, and a score
of D fp32 products and sums is off by at most delta = 2 (D + 8) 2^-24
scale sum|q||k|, which changes every weight by at most that much relative
(numerator and denominator: twice). With A = sum p |v| / sum p:
  |error| <= (h + 2 delta + n 2^-24 + 2^-20) A + h |out|    (1.01: products of the terms)
(n 2^-24: the sums over n keys; 2^-20: exponential, logarithm, division).
The log-sum is off by at most delta + n 2^-24 + 2^-20 (1 + |lse|).
"""
import math

import torch


def see_words(seen):
    """bool [B, T, T] -> int32 words [B, T, ceil(T/32)], bit s % 32 of word s // 32."""
    B, T, _ = seen.shape
    W = (T + 31) // 32
    pad = torch.zeros(B, T, W * 32, dtype=torch.int64)
    pad[:, :, :T] = seen.cpu().long()
    w = (pad.view(B, T, W, 32) << torch.arange(32)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).int()


def attention(q, k, v, vis, scale):
    """q [Hq, T, D], k / v [Hkv, n, D], vis [T, n]; returns (out, lse, A, delta) in 64 bits."""
    Hq, T, D = q.shape
    Hkv, n, _ = k.shape
    out = torch.zeros(Hq, T, D, dtype=torch.float64, device=q.device)
    A = torch.zeros_like(out)
    lse = torch.full((Hq, T), -math.inf, dtype=torch.float64, device=q.device)
    delta = torch.zeros(Hq, T, dtype=torch.float64, device=q.device)
    if n == 0:
        return out, lse, A, delta
    used = vis.any(0)  # keys that nobody sees may hold anything
    k = torch.where(used[None, :, None], k.double(), 0.0).repeat_interleave(Hq // Hkv, 0)
    v = torch.where(used[None, :, None], v.double(), 0.0).repeat_interleave(Hq // Hkv, 0)
    s = (q.double() @ k.transpose(1, 2)) * scale
    mag = (q.double().abs() @ k.abs().transpose(1, 2)) * abs(scale)
    s = s.masked_fill(~vis, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    delta = 2 * (D + 8) * 2.0 ** -24 * mag.masked_fill(~vis, 0.0).amax(-1)
    return p @ v, lse, p @ v.abs(), delta


def check(out, lse, want, n, what=""):
    """out [Hq, T, D], lse [Hq, T] of the GPU against attention()'s."""
    ref, rl, A, delta = want
    h = 0.0 if out.dtype == torch.float32 else torch.finfo(out.dtype).eps / 2
    hr = torch.finfo(out.dtype).eps / 2
    tol = 1.01 * ((h + 2 * delta + n * 2.0 ** -24 + 2.0 ** -20)[..., None] * A + hr * ref.abs()) + 1e-30
    if out.dtype == torch.float16:
        tol = tol + 2.0 ** -24 * (1 + A * 0 + (1 + n) * 2.0 ** -1)  # subnormal weights and results
    got = out.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    worst = ((got - ref).abs() / tol).max().item()
    assert worst <= 1.0, f"{what}: error {worst:.3g} times the bound"
    if lse is not None:
        none = rl == -math.inf
        assert torch.equal(lse.double() == -math.inf, none), f"{what}: which rows see nothing"
        assert (got[none] == 0).all(), f"{what}: rows that see nothing"
        err = (lse.double() - rl)[~none].abs()
        lt = (delta + n * 2.0 ** -24 + 2.0 ** -20 * (1 + rl.abs()))[~none]
        assert (err <= lt).all(), f"{what}: lse off by {(err / lt).max().item():.3g} times the bound"


# ---- page bookkeeping, one step after the other -----------------------------------

def fork_model(table, lens, ref, src, dst, extra, page):
    """What masked_gqa_cache_fork does to lists (table rows, lens, ref); returns
    (copies as (from, to, slots), errors found)."""
    old = [list(r) for r in table]
    old_len = list(lens)
    mp, npages, rows = len(table[0]), len(ref), len(table)
    good = lambda e: e if 0 <= e < npages else -1  # noqa: E731
    bad = False
    pairs, seen = [], set()
    for s, d in zip(src, dst):
        if d in seen or not (0 <= d < rows) or not (-1 <= s < rows):
            bad = True
        else:
            pairs.append((s, d))
        seen.add(d)
    for s, d in pairs:
        if s != d:
            for e in old[d]:
                if good(e) >= 0:
                    ref[e] -= 1
            if s >= 0:
                for e in old[s][:old_len[s] // page]:
                    if good(e) >= 0:
                        ref[e] += 1
    plans, busy = [], set()
    for s, d in pairs:
        n = old_len[s] if s >= 0 else 0
        full, need = n // page, -(-(n + extra) // page) if s >= 0 else 0
        row = [good(e) for e in old[s]] if s >= 0 else [-1] * mp
        fresh = []
        if need <= mp:
            for j in range(full, need):
                if s != d or row[j] < 0 or ref[row[j]] > 1:
                    fresh.append(j)
                    if j == full and n % page:
                        if row[j] >= 0:
                            busy.add(row[j])
                        else:
                            bad = True
        plans.append((s, d, n, full, need, row, fresh))
    free = [p for p in range(npages) if ref[p] <= 0 and p not in busy]
    at, copies, drop = 0, [], []
    for s, d, n, full, need, row, fresh in plans:
        off = at
        at += len(fresh)
        if need > mp or (fresh and at > len(free)):
            bad = True
            if s != d:
                for e in row[:full]:
                    if e >= 0:
                        drop.append(e)
                table[d] = [-1] * mp
                lens[d] = 0
            continue
        new = list(row) if s == d else [e if j < full else -1 for j, e in enumerate(row)]
        for i, j in enumerate(fresh):
            p = free[off + i]
            if j == full and n % page and row[j] >= 0:
                copies.append((row[j], p, n % page))
            if s == d and row[j] >= 0:
                drop.append(row[j])
            new[j] = p
            ref[p] = 1
        table[d], lens[d] = new, n
    for e in drop:
        ref[e] -= 1
    return copies, bad


def compact_model(table, ref):
    """(table, ref, moves, used) after packing."""
    used = [p for p, r in enumerate(ref) if r > 0]
    n = len(used)
    src, dst = [p for p in used if p >= n], [p for p in range(n) if ref[p] <= 0]
    to = dict(zip(src, dst))
    out = list(ref)
    for a, b in to.items():
        out[b], out[a] = ref[a], 0
    return [[to.get(e, e) for e in row] for row in table], out, to, n
