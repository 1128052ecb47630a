"""Prefill attention with a sliding window and sinks against 64 bits."""
import pytest
import torch

from _cache_ref import attention, check

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def M():
    import masked_gqa_attention_gb300 as M
    M.build_library()
    return M


def visible(Lq, Lk, window, sinks, causal, device="cuda"):
    i = torch.arange(Lq, device=device)[:, None] + (Lk - Lq)
    j = torch.arange(Lk, device=device)[None]
    vis = ((i - j < window) & (j - i < window)) | (j < sinks)
    return vis & (j <= i) if causal else vis


def rand(shape, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def run(M, B, Hq, Hkv, Lq, Lk, D, dtype, window, sinks, causal, kv_len=None, seed=1, scale=None, extra=None, **kw):
    q, k, v = rand((B, Hq, Lq, D), dtype, seed), rand((B, Hkv, Lk, D), dtype, seed + 1), rand((B, Hkv, Lk, D), dtype, seed + 2)
    scale = D ** -0.5 if scale is None else scale
    lse = torch.empty(B, Hq, Lq, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kl = None if kv_len is None else torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    out = M.masked_gqa_attn_prefill_window(q, k, v, window=window, sinks=sinks, causal=causal, scale=scale, lse=lse,
                                           kv_len=kl, dev_error=err, **kw)
    vis = visible(Lq, Lk, window, sinks, causal)
    for b in range(B):
        vb = vis if kl is None else vis & (torch.arange(Lk, device="cuda") < kv_len[b])
        vb = vb if extra is None else vb & extra[b]
        check(out[b], lse[b], attention(q[b], k[b], v[b], vb, scale), Lk, f"row {b}")
    assert int(err) == 0
    return q, k, v, out


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("L,window,sinks", [
    (1, 1, 0), (1, 5, 3), (127, 1, 0), (129, 128, 0), (300, 64, 4), (517, 129, 130), (640, 100, 0), (1000, 257, 1),
    (257, 1000, 4), (257, 2 ** 31 - 1, 2 ** 31 - 1)])
def test_square(M, L, window, sinks, dtype, causal):
    run(M, 1, 4, 2, L, L, 128 if L % 2 else 64, dtype, window, sinks, causal)


@pytest.mark.parametrize("dtype,D", [(BF, 128), (HF, 64), (FP, 128)])
@pytest.mark.parametrize("Lq,Lk", [(1, 700), (130, 900), (257, 258), (300, 200)])  # the last: rows in front of every key
@pytest.mark.parametrize("causal", [True, False])
def test_rectangular(M, Lq, Lk, dtype, D, causal):
    run(M, 2, 3, 1, Lq, Lk, D, dtype, 150, 2, causal)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_padded_rows_see_nothing_behind_their_length(M, dtype):
    # rows behind kv_len + window have no key left but the sinks; without sinks none at all
    run(M, 4, 4, 4, 500, 500, 64, dtype, 60, 3, True, kv_len=[500, 130, 1, 0])
    run(M, 3, 2, 1, 500, 500, 128, dtype, 60, 0, True, kv_len=[500, 130, 0])


def test_every_group_size(M):
    for Hq, Hkv in ((1, 1), (8, 1), (7, 1), (6, 2)):
        run(M, 1, Hq, Hkv, 200, 333, 64, BF, 77, 5, True)


def test_window_wider_than_the_sequence_is_the_causal_call(M):
    q, k, v, out = run(M, 2, 4, 2, 400, 400, 128, BF, 400, 0, True)
    assert torch.equal(out, M.masked_gqa_attn_prefill(q, k, v, causal=True))
    q, k, v, out = run(M, 1, 4, 2, 300, 300, 64, HF, 300, 0, False)
    assert torch.equal(out, M.masked_gqa_attn_prefill(q, k, v))


def test_with_segments_and_bits(M):
    from _cache_ref import see_words
    B, L = 2, 320
    seg = torch.zeros(B, L, dtype=torch.int32, device="cuda")
    seg[:, 200:] = 1
    seg[1, 310:] = -1
    same = (seg[:, :, None] == seg[:, None, :]) & (seg >= 0)[:, :, None]
    run(M, B, 4, 2, L, L, 128, BF, 50, 0, True, extra=same, seg_q=seg, seg_k=seg)
    g = torch.Generator().manual_seed(3)
    m = torch.rand(B, L, L, generator=g) < 0.3
    m[0, 17] = False  # a row left empty
    run(M, B, 4, 2, L, L, 64, BF, 90, 4, True, extra=m.cuda(), mask_bits=see_words(m).cuda())
    run(M, B, 2, 2, L, L, 64, FP, 90, 4, False, extra=m.cuda(), mask_bits=see_words(m).cuda())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_hidden_keys_may_hold_anything_outside_the_read_tiles(M, dtype):
    # key tiles that neither the window nor the sinks reach are not read
    q, k, v = (rand((1, 2, 1024, 64), dtype, s) for s in (5, 6, 7))
    k[:, :, 256:512] = float("nan")
    v[:, :, 256:512] = float("inf")
    out = M.masked_gqa_attn_prefill_window(q[:, :, 768:], k, v, window=200, sinks=4)
    vis = visible(256, 1024, 200, 4, True)
    check(out[0], None, attention(q[0, :, 768:], k[0], v[0], vis, 64 ** -0.5), 1024)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,D", [(BF, 128), (HF, 64), (FP, 64), (FP, 128)])
def test_rows_behind_their_length_may_hold_anything(M, dtype, D, causal):
    lens, L, bad = [400, 130, 1, 0, 256, 399, 17], 400, float("nan")
    B, H = len(lens), 2
    q, k, v = (rand((B, H, L, D), dtype, s) for s in (1, 2, 3))
    for b, n in enumerate(lens):
        k[b, :, n:], v[b, :, n:] = bad, bad
        bad = -bad if b % 2 else float("inf")
    lse = torch.empty(B, H, L, device="cuda")
    for window, sinks in ((70, 3), (400, 0)):
        out = M.masked_gqa_attn_prefill_window(q, k, v, window=window, sinks=sinks, causal=causal, lse=lse,
                                               kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        vis = visible(L, L, window, sinks, causal)
        for b, n in enumerate(lens):
            kb, vb = k[b].clone(), v[b].clone()
            kb[:, n:], vb[:, n:] = 0, 0
            check(out[b], lse[b], attention(q[b], kb, vb, vis & (torch.arange(L, device="cuda") < n), D ** -0.5), L, f"row {b}")


def test_negative_scale_and_strides(M):
    run(M, 1, 4, 2, 260, 260, 128, BF, 99, 4, True, scale=-0.3)
    # a [B, L, H, D] projection's views
    B, H, L, D = 2, 4, 333, 64
    q, k, v = (rand((B, L, H, D), BF, s).transpose(1, 2) for s in (1, 2, 3))
    out = torch.full((B, L, H, D), 7.0, dtype=BF, device="cuda")
    M.masked_gqa_attn_prefill_window(q, k, v, out.transpose(1, 2), window=40, sinks=2)
    for b in range(B):
        check(out[b].transpose(0, 1), None, attention(q[b], k[b], v[b], visible(L, L, 40, 2, True), D ** -0.5), L)


def test_long_sequence(M):
    # thousands of key tiles; a sample of the rows against 64 bits
    L, W, D = 60000, 700, 64
    q, k, v = (rand((1, 2, L, D), BF, s) for s in (1, 2, 3))
    lse = torch.empty(1, 2, L, device="cuda")
    out = M.masked_gqa_attn_prefill_window(q, k, v, window=W, sinks=3, lse=lse)
    rows = torch.tensor([0, 1, 699, 700, 701, 4095, 30000, 59998, 59999], device="cuda")
    j = torch.arange(L, device="cuda")
    vis = ((rows[:, None] - j < W) | (j < 3)) & (j <= rows[:, None])
    check(out[0][:, rows], lse[0][:, rows], attention(q[0][:, rows], k[0], v[0], vis, D ** -0.5), W + 3)


def test_captured_and_replayed(M):
    q, k, v = (rand((1, 4, 300, 128), BF, s) for s in (1, 2, 3))
    out = torch.empty_like(q)
    want = M.masked_gqa_attn_prefill_window(q, k, v, window=64, sinks=4).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.masked_gqa_attn_prefill_window(q, k, v, out, window=64, sinks=4)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
