"""64-bit references of the cache in 4 bits, of the accumulated attention weights
and of the eviction, with error bounds derived from the arithmetic.

A record stands for x = scale u + least. The kernels multiply the codes and add the
least values' part beside them, so magnitudes below are of scale u + |least|, not of
x. With h = 2^-11 (a weight, or a weight times a scale, is one fp16 operand; two of
them, 2^-22, in fp32 calls), hr half a step of the output's type, and scores off by
at most delta = 2 (D + 8) 2^-24 scale sum |q| (scale u + |least|), which covers the
fp32 products and sums and the queries' two terms of 2^-22:
  |error| <= 1.01 ((h + 2 delta + n 2^-24 + 2^-20) A + hr |out|) + n F
where A = sum p (scale u + |least|) and F = 2^-39 (|least| + 30 scale), the largest
of each: a weight is held as up to 2^14, its fp16 rounding is at least 2^-25, and so
for its product with a scale, which is held relative to a power of two above every
scale. The log-sum is off by at most delta + n 2^-24 + 2^-20 (1 + |lse|).
"""
import math

import torch


def group_bytes(D, g):
    """Where group g's codes lie in a record of D features."""
    return slice(16 * g, 16 * g + 16) if D == 128 else slice(16 * (g // 2) + g % 2, 16 * (g // 2) + 16, 2)


def records(x):
    """Rows [..., D] as records, each step in 64 bits and rounded once to its type."""
    shape, D = x.shape[:-1], x.shape[-1]
    x = x.reshape(-1, D).double()
    r32 = lambda t: t.float().double()  # noqa: E731
    out = torch.zeros(x.shape[0], D // 2 + 16, dtype=torch.uint8, device=x.device)
    par = torch.zeros(x.shape[0], 8, dtype=torch.float16, device=x.device)
    for g in range(4):
        y = x[:, g * D // 4:(g + 1) * D // 4]
        lo = y.min(1).values.clamp(-65504, 65504).half().double()
        lo = torch.where(lo == 0, 0.0, lo)
        sc = r32(r32(y.max(1).values - lo) * r32(torch.tensor(1 / 15, dtype=torch.float64))).clamp(0, 65504).half()
        par[:, g], par[:, 4 + g] = sc, lo.half()
        sc = sc.double()[:, None]
        u = r32(r32(y - lo[:, None]) / torch.where(sc > 0, sc, 1.0))
        u = torch.where(sc > 0, u.round().clamp(0, 15), 0.0).to(torch.uint8)
        out[:, group_bytes(D, g)] = u[:, 0::2] + 16 * u[:, 1::2]
    out[:, D // 2:] = par.view(torch.uint8)
    return out.reshape(*shape, D // 2 + 16)


def values(rec):
    """(x, scale u + |least|) of records [..., D/2 + 16], in 64 bits."""
    shape, D = rec.shape[:-1], 2 * (rec.shape[-1] - 16)
    rec = rec.reshape(-1, rec.shape[-1])
    par = rec[:, D // 2:].contiguous().view(torch.float16).double()
    x = torch.empty(rec.shape[0], D, dtype=torch.float64, device=rec.device)
    mag = torch.empty_like(x)
    for g in range(4):
        b = rec[:, group_bytes(D, g)]
        u = torch.stack([b % 16, b // 16], -1).reshape(rec.shape[0], D // 4).double() * par[:, g, None]
        x[:, g * D // 4:(g + 1) * D // 4] = u + par[:, 4 + g, None]
        mag[:, g * D // 4:(g + 1) * D // 4] = u.abs() + par[:, 4 + g, None].abs()
    return x.reshape(*shape, D), mag.reshape(*shape, D)


def sees(n, T, window, sinks, device="cpu"):
    """[T, n]: which of n slots the last T tokens see."""
    j, pos = torch.arange(n, device=device), n - T + torch.arange(T, device=device)[:, None]
    vis = j <= pos
    return vis & ((pos - j < window) | (j < sinks)) if window else vis


def scores(q, k, kmag, vis, scale):
    """q [Hq, T, D], k [Hkv, n, D]: (scores with -inf where unseen, delta [Hq, T])."""
    Hq, T, D = q.shape
    rep = Hq // k.shape[0]
    s = (q.double() @ k.repeat_interleave(rep, 0).transpose(1, 2)) * scale
    mag = (q.double().abs() @ kmag.repeat_interleave(rep, 0).transpose(1, 2)) * abs(scale)
    delta = 2 * (D + 8) * 2.0 ** -24 * mag.masked_fill(~vis, 0.0).amax(-1) if k.shape[1] else mag.sum(-1)
    return s.masked_fill(~vis, -math.inf), delta


def check_attention(out, lse, q, krec, vrec, vis, scale, what=""):
    """out [Hq, T, D], lse [Hq, T] of the GPU for krec / vrec [Hkv, n, D/2 + 16]."""
    Hq, T, D = q.shape
    n = krec.shape[1]
    used = vis.any(0)  # records that nobody sees may hold anything
    clean = lambda r: torch.where(used[None, :, None], r, torch.zeros_like(r))  # noqa: E731
    (k, kmag), (v, vmag) = values(clean(krec)), values(clean(vrec))
    s, delta = scores(q, k, kmag, vis, scale)
    lse_ref = torch.logsumexp(s, -1) if n else torch.full((Hq, T), -math.inf, dtype=torch.float64, device=q.device)
    none = lse_ref == -math.inf
    p = torch.exp(s - torch.where(none, 0.0, lse_ref)[..., None])
    rep = Hq // k.shape[0]
    ref, A = p @ v.repeat_interleave(rep, 0), p @ vmag.repeat_interleave(rep, 0)
    par = clean(vrec)[..., D // 2:].contiguous().view(torch.float16).double().abs()
    floor = 2.0 ** -39 * (par[..., 4:].amax() + 30 * par[..., :4].amax()) if n else 0.0
    h = 2.0 ** -22 if out.dtype == torch.float32 else 2.0 ** -11
    hr = torch.finfo(out.dtype).eps / 2
    tol = 1.01 * ((h + 2 * delta + n * 2.0 ** -24 + 2.0 ** -20)[..., None] * A + hr * ref.abs()) + n * floor + 1e-30
    if out.dtype == torch.float16:
        tol = tol + 2.0 ** -25  # subnormal results
    got = out.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    worst = ((got - ref).abs() / tol).max().item()
    assert worst <= 1.0, f"{what}: error {worst:.3g} times the bound"
    if lse is not None:
        assert torch.equal(lse.double() == -math.inf, none), f"{what}: which rows see nothing"
        assert (got[none] == 0).all(), f"{what}: rows that see nothing"
        err = (lse.double() - lse_ref)[~none].abs()
        lt = (delta + n * 2.0 ** -24 + 2.0 ** -20 * (1 + lse_ref.abs()))[~none]
        assert (err <= lt).all(), f"{what}: lse off by {(err / lt).max().item():.3g} times the bound"


def check_weights(got, before, q, k, kmag, vis, lse, scale, what=""):
    """got, before [Hkv, >= n]: weights after and before the call; k, kmag [Hkv, n, D] in 64 bits.

    A weight is off by delta (its score), 2^-20 (the exponential) and 2^-23 (1 + |lse|
    log2 e) (the log-sum in base 2), relative; their sum of R terms and the one that is
    added by (R + 2) 2^-24."""
    Hkv, n = k.shape[:2]
    Hq, T, _ = q.shape
    used = vis.any(0)
    assert torch.equal(got[:, n:], before[:, n:]), f"{what}: weights behind the length"
    if n == 0:
        return
    assert torch.equal(got[:, :n][:, ~used], before[:, :n][:, ~used]), f"{what}: weights of slots that are not seen"
    z = lambda t: torch.where(used[None, :, None], t, torch.zeros_like(t))  # noqa: E731
    s, delta = scores(q, z(k), z(kmag), vis, scale)
    dead = lse.double() == -math.inf
    p = torch.exp(s - torch.where(dead, math.inf, lse.double())[..., None])
    rel = delta + 2.0 ** -20 + 2.0 ** -23 * (1 + torch.where(dead, 0.0, lse.double().abs()) * 1.4427)
    tol = (p * rel[..., None]).reshape(Hkv, -1, n).sum(1)
    add = p.reshape(Hkv, -1, n).sum(1)
    want = before[:, :n].double() + add
    tol = 1.01 * (tol + (Hq // Hkv * T + 2) * 2.0 ** -24 * want.abs()) + 1e-30
    err = (got[:, :n].double() - want).abs()[:, used]
    worst = (err / tol[:, used]).max().item() if used.any() else 0.0
    assert worst <= 1.0, f"{what}: weights off by {worst:.3g} times the bound"


def kept_slots(w, n, budget, sinks, recent):
    """Slots that stay of n with weights w [>= n] (on the CPU), in order."""
    if n <= budget:
        return list(range(n))
    mid = w[sinks:n - recent].double()
    mid = torch.where(mid.isnan(), -math.inf, mid)
    # (a NaN behind -inf: by whether it is one, then by weight; stable, so the first of equal ones)
    order = torch.sort(mid, descending=True, stable=True).indices
    order = order[torch.sort(w[sinks:n - recent][order].isnan().int(), stable=True).indices]
    middle = (order[:budget - sinks - recent] + sinks).tolist()
    return sorted(list(range(sinks)) + middle + list(range(n - recent, n)))
