"""Attention over 4-bit records whose rows share one scale: a rounding that is the same for
every key does not average out, so errors are bounded by the outputs themselves."""
import math

import pytest
import torch

from _q4_ref import group_bytes, sees, values

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
LEVEL = 0.05  # how much lower every second key's score is


@pytest.fixture(scope="module")
def M():
    import masked_gqa_attention_gb300 as M
    M.build_library()
    return M


def pack(u, scale, least):
    """Records of codes u [..., D] with one scale and least value a row ([...])."""
    D = u.shape[-1]
    rec = torch.zeros(*u.shape[:-1], D // 2 + 16, dtype=torch.uint8, device="cuda")
    for g in range(4):
        y = u[..., g * D // 4:(g + 1) * D // 4]
        rec[..., group_bytes(D, g)] = y[..., 0::2] + 16 * y[..., 1::2]
    par = torch.cat([x.half()[..., None].expand(*x.shape, 4) for x in (scale, least)], -1)
    rec[..., D // 2:] = par.contiguous().view(torch.uint8)
    return rec


def worst_scale(power):
    """The scale in [2^power, 2^(power + 1)) whose product with the lower level's weight loses most in fp16."""
    p = float(torch.tensor(2.0 ** 14 * math.exp(-LEVEL)).half())
    return 2.0 ** power * max((m / 1024 for m in range(1024, 2048)),
                              key=lambda s: abs(float(torch.tensor(p * s).half()) / (p * s) - 1))


@pytest.mark.parametrize("codes", ["even", "low", "high"])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,T,Hq,Hkv,power", [(1000, 1, 4, 1, 0), (4096, 1, 16, 1, 3), (100003, 1, 8, 2, -4),
                                              (60000, 8, 8, 2, 0)])
def test_keys_of_one_scale(M, codes, dtype, D, n, T, Hq, Hkv, power):
    """Keys of two scores, half of them each; values of one scale and random codes whose mean stands for 0.

    Keys of a score have one weight, and so one rounding of it (h = 2^-11; fp32 2^-22) and one of its product
    with the scale: the sum A of such keys' part of the output is off by h |A| from the first, and by h times
    what the codes are from their middle, |A| + W scale / 64 of weight W, from the second. Beside them half a
    step hr of the output's type, the scores' and exponentials' 2^-20 |A|, and 2^-20 of the largest terms for
    the fp32 sums."""
    g = torch.Generator("cuda").manual_seed(n + D)
    f = torch.rand((Hkv, n, D), generator=g, device="cuda")
    u = (16 * f).floor() if codes == "even" else (-3 * torch.log(f.clamp_min(1e-9))).floor()
    u = u.clamp(0, 15)
    u = (15 - u if codes == "high" else u).to(torch.uint8)
    scale = worst_scale(power)
    one = torch.ones((Hkv, n), device="cuda")
    v = pack(u, scale * one, -scale * u.float().mean() * one)
    low = torch.arange(n, device="cuda") % 2 == 1
    k = pack(torch.zeros_like(u), 0 * one, -LEVEL * low * one)  # q = 1: a score is the least value
    q = torch.ones(1, Hq, T, D, device="cuda", dtype=dtype)
    lens, err = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = M.masked_gqa_attn_decode_q4(q, k[None], v[None], lens, scale=1.0 / D, dev_error=err)[0].double()
    assert int(err) == 0
    val, mag = values(v)
    h, hr = 2.0 ** -22 if dtype == FP else 2.0 ** -11, torch.finfo(dtype).eps / 2
    s = torch.where(low, -LEVEL, 0.0).half().double().expand(T, n).masked_fill(~sees(n, T, 0, 0, "cuda"), -math.inf)
    p = torch.softmax(s, -1)
    parts = [torch.where(x, p, 0.0) @ val for x in (low, ~low)]  # [Hkv, T, D]
    ref = (parts[0] + parts[1]).repeat_interleave(Hq // Hkv, 0)
    A = (parts[0].abs() + parts[1].abs()).repeat_interleave(Hq // Hkv, 0)
    tol = (2 * h + 2.0 ** -20) * A + hr * ref.abs() + h * scale / 64 + 2.0 ** -20 * mag.amax()
    worst = ((out - ref).abs() / (1.01 * tol)).max().item()
    assert worst <= 1.0, f"error {worst:.3g} times the bound ({(out - ref).abs().max() / ref.abs().max():.3g} of the output)"


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D", [64, 128])
def test_features_of_a_query_far_apart(M, dtype, D):
    """One feature of a query is 1, the others 2^-16 to 2^-24 of it; the large one meets zeros, so the scores are
    the small ones'. A feature is held to 2^-27 of the largest of its row (scaled to [2^6, 2^7), where those of
    every second code, divided by 16, have steps of 2^-24; fp32: two terms, 2^-31), and meets scale u; the sums
    are off by (D + 8) 2^-24 of their terms, twice (see _q4_ref). fp32 calls multiply u - 8 and add 8 times the
    queries' sums, so their terms are of |q| scale (|u - 8| + 8), which is not 0 for a code of 0: the large
    feature's are 16 scale, and off by the queries' 2^-22 besides."""
    g = torch.Generator("cuda").manual_seed(D)
    n, H, scale = 300, 2, 16.0
    u = torch.randint(0, 16, (H, n, D), generator=g, device="cuda", dtype=torch.uint8)
    u[..., 0] = 0
    size = 64.0 * (1 + torch.rand((H, n), generator=g, device="cuda"))
    k = pack(u, size, 0 * size)
    v = pack(u, size / 64, 0 * size)
    q = torch.randn((1, H, 9, D), generator=g, device="cuda")
    q *= 2.0 ** -torch.arange(16, 25, device="cuda")[:, None].float()
    q[..., 0] = 1.0
    q = q.to(dtype)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    lse = [torch.empty(1, H, 1, device="cuda") for _ in range(9)]
    for t in range(9):  # (a query a call, so that each sees every key)
        M.masked_gqa_attn_decode_q4(q[:, :, t:t + 1], k[None], v[None], lens, scale=scale, lse=lse[t])
    lse = torch.cat(lse, 2)
    val, mag = values(k)
    s = scale * (q[0].double() @ val.transpose(1, 2))
    held = 2.0 ** (-31 if dtype == FP else -27)
    terms = size[..., None] * ((u.double() - 8).abs() + 8) if dtype == FP else mag
    delta = scale * (held * mag.sum(-1).amax(-1)[:, None]
                     + 2 * (D + 8) * 2.0 ** -24 * (q[0].double().abs() @ terms.transpose(1, 2)).amax(-1))
    want = torch.logsumexp(s, -1)
    tol = delta + n * 2.0 ** -24 + 2.0 ** -20 * (1 + want.abs())
    worst = ((lse[0].double() - want).abs() / tol).max().item()
    assert worst <= 1.0, f"log-sums off by {worst:.3g} times the bound"
