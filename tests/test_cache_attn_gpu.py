"""One token with a window, and trees of drafted tokens, over a cache in slots
or pages, against 64 bits. Everything that no query may see is NaN or a page
index far outside the pool, so a result shows whether it was read."""
import random

import pytest
import torch

from _cache_ref import attention, check, see_words

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def M():
    import masked_gqa_attention_gb300 as M
    M.build_library()
    return M


def rand(shape, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def tree_of(rng, T):
    seen = torch.zeros(T, T, dtype=torch.bool)
    for t in range(T):
        parent = rng.randint(max(-1, t - 5), t - 1)
        if parent >= 0:
            seen[t] = seen[parent]
        seen[t, t] = True
    return seen


class Case:
    """Inputs of one call and the 64-bit answer. page 0: the static cache."""

    def __init__(self, lens, T, Hq, Hkv, D, dtype, *, page=0, cap=None, window=0, sinks=0, seen="tree", live=None,
                 seed=1, scale=None, tree=True):
        rng = random.Random(seed)
        B = len(lens)
        cap = max(lens) + 5 if cap is None else cap
        cap = max(cap, 1)
        self.window, self.sinks, self.T, self.tree = window, sinks, T, tree
        self.scale = D ** -0.5 if scale is None else scale
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.q = rand((B, Hq, T, D), dtype, seed)
        kn, vn = rand((B, T, Hkv, D), dtype, seed + 1), rand((B, T, Hkv, D), dtype, seed + 2)
        self.kn, self.vn = kn.transpose(1, 2), vn.transpose(1, 2)
        if seen == "tree":
            self.seen = torch.stack([tree_of(rng, T) for _ in range(B)])
        elif seen == "chain":
            self.seen = torch.ones(T, T, dtype=torch.bool).tril().expand(B, T, T)
        else:
            self.seen = seen
        self.bits = None if isinstance(seen, str) and seen == "chain" else see_words(self.seen).cuda()
        self.live = None if live is None else torch.tensor(live, dtype=torch.int32, device="cuda")
        self.want = []
        keys, values = [], []
        for b, n in enumerate(lens):
            m = T if live is None else live[b]
            s = self.seen[b].clone().cuda()
            s[m:] = False
            s[:, m:] = False
            eye = torch.eye(T, dtype=torch.bool, device="cuda")
            pos = n + (s & ~eye).sum(1) if tree else torch.tensor([n - 1], device="cuda")
            j = torch.arange(n, device="cuda")
            see = torch.ones(T, n, dtype=torch.bool, device="cuda")
            if window:
                see = (pos[:, None] - j < window) | (j < sinks)
                s = s & ((pos[:, None] - pos < window) | (pos < sinks))
            see[m:] = False
            k, v = rand((Hkv, n, D), dtype, seed + 10 + b), rand((Hkv, n, D), dtype, seed + 500 + b)
            hid = ~see.any(0)
            k[:, hid], v[:, hid] = float("nan"), float("nan")
            keys.append((k, hid))
            values.append(v)
            if tree:
                self.kn[b, :, m:], self.vn[b, :, m:] = float("nan"), float("nan")
                full = torch.cat([see, s], 1)
                self.want.append((attention(self.q[b], torch.cat([k, self.kn[b]], 1), torch.cat([v, self.vn[b]], 1),
                                            full, self.scale), n + T))
            else:
                self.want.append((attention(self.q[b], k, v, see, self.scale), n))
        if page:
            mp = -(-cap // page)
            need = [-(-n // page) for n in lens]
            order = list(range(sum(need) + 2))
            rng.shuffle(order)
            self.k = torch.full((len(order), Hkv, page, D), float("nan"), dtype=dtype, device="cuda")
            self.v = self.k.clone()
            table = torch.full((B, mp), 2 ** 30, dtype=torch.int32)
            at = 0
            for b, n in enumerate(lens):
                k, hid = keys[b]
                for i in range(need[b]):
                    a, z = i * page, min(n, i * page + page)
                    if hid[a:z].all():
                        continue  # a page that nothing looks at: no entry
                    table[b, i] = order[at]
                    self.k[order[at], :, :z - a], self.v[order[at], :, :z - a] = k[:, a:z], values[b][:, a:z]
                    at += 1
            self.table = table.cuda()
        else:
            self.table = None
            self.k = torch.full((B, Hkv, cap, D), float("nan"), dtype=dtype, device="cuda")
            self.v = self.k.clone()
            for b, n in enumerate(lens):
                self.k[b, :, :n], self.v[b, :, :n] = keys[b][0], values[b]

    def call(self, M, **kw):
        B, Hq, T, _ = self.q.shape
        self.lse = torch.empty(B, Hq, T, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw = dict(dict(page_table=self.table, scale=self.scale, lse=self.lse, dev_error=self.err), **kw)
        if not self.tree:
            return M.masked_gqa_attn_decode_window(self.q, self.k, self.v, self.kv_len, window=self.window,
                                                   sinks=self.sinks, **kw)
        return M.masked_gqa_attn_decode_tree(self.q, self.k, self.v, self.kn, self.vn, self.kv_len,
                                             tree_bits=self.bits, tree_len=self.live, window=self.window,
                                             sinks=self.sinks, **kw)

    def run(self, M, **kw):
        out = self.call(M, **kw)
        for b, (want, n) in enumerate(self.want):
            check(out[b], self.lse[b], want, n, f"request {b}")
        assert int(self.err) == 0
        return out


@pytest.mark.parametrize("page", [0, 1, 8, 24, 64, 128])
@pytest.mark.parametrize("dtype,D", [(BF, 128), (HF, 64), (FP, 64), (FP, 128), (BF, 64)])
def test_decode_window(M, page, dtype, D):
    Case([1, 0, 63, 64, 65, 700, 1023], 1, 8, 2, D, dtype, page=page, window=130, sinks=4, tree=False,
         seen="chain").run(M)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 0), (64, 64), (65, 63), (100, 130), (129, 200),
                                          (2 ** 31 - 1, 0), (300, 2 ** 31 - 1)])
def test_decode_window_edges(M, window, sinks):
    for page in (0, 16):
        Case([1, 64, 128, 129, 191, 192, 193, 500, 640], 1, 4, 4, 64, BF, page=page, window=window, sinks=sinks,
             tree=False, seen="chain").run(M)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 1), (8, 8), (56, 8), (16, 1), (40, 2), (64, 1)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_decode_groups(M, Hq, Hkv, dtype):
    Case([5, 333], 1, Hq, Hkv, 128, dtype, page=16, window=100, sinks=4, tree=False, seen="chain").run(M)


@pytest.mark.parametrize("T", [1, 2, 5, 8, 16, 31, 32, 33, 64])
@pytest.mark.parametrize("dtype,D", [(BF, 128), (HF, 64), (FP, 128), (FP, 64), (BF, 64), (HF, 128)])
def test_tree(M, T, dtype, D):
    Case([0, 1, 64, 130, 777], T, 8, 2, D, dtype, page=16).run(M)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T", [100, 129, 256])
def test_large_trees(M, T, dtype):
    Case([700, 3], T, 4, 2, 64, dtype, page=32).run(M)
    Case([300, 65], T, 3, 1, 128, dtype, page=0, window=90, sinks=4, live=[T, T // 2]).run(M)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 0), (40, 4), (64, 70), (1000, 0)])
def test_tree_with_a_window(M, window, sinks, dtype):
    Case([0, 2, 63, 200, 515], 24, 4, 2, 64, dtype, page=8, window=window, sinks=sinks).run(M)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_ragged_trees(M, dtype):
    Case([0, 100, 64, 0, 300], 20, 8, 2, 128, dtype, page=16, live=[0, 0, 1, 20, 7]).run(M)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_chain_of_drafts(M, dtype):
    Case([0, 100, 513], 33, 6, 2, 64, dtype, page=16, seen="chain").run(M)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_masks_that_are_no_tree(M, dtype):
    g = torch.Generator().manual_seed(2)
    seen = torch.rand(3, 40, 40, generator=g) < 0.4  # rows without themselves, drafts behind them
    seen[:, 5] = False
    Case([0, 10, 200], 40, 2, 1, 64, dtype, page=16, seen=seen).run(M)  # row 5 of request 0 sees nothing
    Case([0, 10, 200], 40, 2, 1, 64, dtype, page=16, seen=seen, window=12, sinks=1).run(M)


@pytest.mark.parametrize("dtype,T,page", [(BF, 1, 16), (BF, 8, 16), (BF, 61, 64), (HF, 16, 0), (FP, 4, 32), (BF, 33, 0)])
def test_long_rows_are_split(M, dtype, T, page):
    # few requests: every unit is cut into many runs and joined
    Case([20011], T, 8, 2, 128, dtype, page=page, cap=20200).run(M)
    Case([9000, 1, 0, 4097], T, 4, 1, 64, dtype, page=page, cap=9300, window=5000, sinks=100).run(M)


def test_many_requests(M):
    rng = random.Random(4)
    lens = [rng.randint(0, 300) for _ in range(300)]
    Case(lens, 3, 4, 2, 64, BF, page=16, cap=310).run(M)
    Case(lens, 1, 4, 2, 64, FP, page=16, cap=310, window=100, sinks=2, tree=False, seen="chain").run(M)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_scales(M, dtype):
    for scale in (0.0, -0.4, 2.0):
        Case([130, 5], 6, 4, 2, 64, dtype, page=16, scale=scale).run(M)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_many_rows(M, dtype):
    # past one block of 128 rows, two of 128, and a group that no block holds
    Case([700, 0, 129], 64, 8, 2, 128, dtype, page=16).run(M)
    Case([300, 65], 40, 28, 4, 64, dtype, page=64, window=100, sinks=3).run(M)
    Case([130], 3, 200, 1, 64, dtype, page=16).run(M)
    Case([9000, 20], 70, 24, 8, 128, dtype, page=0).run(M)
    for T in (10, 12, 24, 26):  # 40, 48, 96 and 104 rows, short calls and long ones
        Case([333, 64, 0], T, 8, 2, 64, dtype, page=16).run(M)
        Case([20000, 17], T, 32, 8, 128, dtype, page=32, cap=40000, live=[T, 3]).run(M)


@pytest.mark.parametrize("dtype,D", [(BF, 128), (HF, 64), (FP, 64), (FP, 128)])
@pytest.mark.parametrize("page", [1, 3, 20])
def test_odd_pages(M, page, dtype, D):
    # rows fetched one by one: few and many rows, short calls and long ones, windows, live drafts, scales
    Case([5, 0, 333, 64], 3, 8, 2, D, dtype, page=page).run(M)
    Case([700, 129], 40, 8, 2, D, dtype, page=page, live=[40, 9]).run(M)
    Case([200, 1], 130, 4, 2, D, dtype, page=page, window=70, sinks=3).run(M)
    Case([900, 333], 20, 8, 2, D, dtype, page=page, scale=-0.2).run(M)
    Case([30000, 700], 8, 16, 2, D, dtype, page=page, cap=60000 // page * page).run(M)


def test_odd_pages_long(M):
    Case([40000, 39000, 33, 40001], 64, 32, 8, 128, BF, page=5, cap=200000).run(M)
    Case([300, 100], 100, 8, 2, 64, FP, page=1, cap=300000, window=50).run(M)


def test_large_trees_over_long_rows(M):
    # reads past the size where two row blocks share the key tiles
    Case([40000, 39000, 33, 40001], 64, 64, 16, 128, BF, page=64, cap=40100).run(M)
    Case([70000, 12], 61, 24, 8, 64, HF, page=0, cap=100000, window=30000, sinks=4, live=[61, 3]).run(M)
    Case([33000, 31000, 100], 44, 48, 16, 128, BF, page=16, cap=33100).run(M)  # groups of three heads


@pytest.mark.parametrize("dtype", [BF, FP])
def test_scales_of_many_rows(M, dtype):
    for scale in (0.0, -0.4, 3.0):
        Case([300, 5], 50, 8, 2, 64, dtype, page=16, scale=scale).run(M)


def test_rising_scores_rescale(M):
    # keys whose scores climb by more than 2^8 from tile to tile: the running
    # maximum moves at every one and the outputs so far are rescaled
    for T, Hq, window in ((1, 4, 0), (24, 8, 0), (64, 8, 0), (24, 8, 900)):
        c = Case([1500, 700], T, Hq, 2, 128, BF, page=64, window=window)
        g = torch.linspace(1, 40, c.k.shape[0], device="cuda").to(BF)  # by page: any order of tiles
        q = c.q[:, :, :, :1].sign() * torch.ones_like(c.q)
        kk = torch.full_like(c.k, 0.05) * g[:, None, None, None]
        c.k = torch.where(torch.isnan(c.k), c.k, kk)
        c.q = q
        want = []
        for b, n in enumerate((1500, 700)):
            rows = c.table[b].long()
            rows = torch.where((rows >= 0) & (rows < c.k.shape[0]), rows, 0)
            k = c.k[rows].transpose(0, 1).reshape(2, -1, 128)[:, :n]
            v = c.v[rows].transpose(0, 1).reshape(2, -1, 128)[:, :n]
            seen = c.seen[b].cuda()
            pos = n + seen.sum(1) - 1
            see = torch.ones(T, n, dtype=torch.bool, device="cuda")
            if window:
                see = pos[:, None] - torch.arange(n, device="cuda") < window
                seen = seen & (pos[:, None] - pos < window)
            want.append((attention(q[b], torch.cat([k, c.kn[b]], 1), torch.cat([v, c.vn[b]], 1),
                                   torch.cat([see, seen], 1), c.scale), n + T))
        c.want = want
        c.run(M)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_other_layouts(M, dtype):
    for T in (1, 6, 40):
        c = Case([100, 300], T, 8, 2, 64, dtype, page=16)
        want = c.run(M).clone()
        # pools stored slot by slot, [pages, page, Hkv, D], and a table inside a wider one
        k, v, table = c.k, c.v, c.table
        c.k, c.v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
        wide = torch.full((2, table.shape[1] + 7), -5, dtype=torch.int32, device="cuda")
        wide[:, 3:3 + table.shape[1]] = table
        c.table = wide[:, 3:3 + table.shape[1]]
        assert torch.equal(c.run(M), want)
        # K and V in one tensor, q as a projection leaves it
        c.k, c.v = torch.stack([k, v], 2).unbind(2)
        c.q = c.q.transpose(1, 2).contiguous().transpose(1, 2)
        assert torch.equal(c.run(M), want)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_broadcast_tensors(M, dtype):
    # one row of drafts for the whole batch, one mask for every request
    for T, names in ((5, ("kn", "vn", "q")), (40, ("kn", "vn", "q")), (70, ("kn", "vn"))):
        c = Case([100, 300], T, 4, 2, 64, dtype, page=16)
        d = Case([100, 300], T, 4, 2, 64, dtype, page=16)
        for name in names:
            x = getattr(c, name)[:1]
            setattr(c, name, x.expand(2, -1, -1, -1))
            setattr(d, name, x.expand(2, -1, -1, -1).contiguous())
        c.bits, d.bits = c.bits[:1], c.bits[:1].expand(2, -1, -1).contiguous()
        a, b = c.call(M), d.call(M)
        assert int(c.err) == 0 and (a.float() - b.float()).abs().max() <= 2e-2 and torch.isfinite(a).all()


def test_sizes_past_32_bits_in_counts(M):
    c = Case([100], 4, 4, 2, 64, BF, page=16)
    want = c.run(M).clone()
    c.window, c.sinks = 2 ** 40, 2 ** 33 + 1  # wider than anything: no window
    assert torch.equal(c.call(M), want)


def test_largest_slots(M):
    # past 2^31 elements of one cache: 64-bit offsets (bf16, 2 x 4.4 GB)
    n, Hkv, D = 2_200_000, 8, 128
    k = torch.empty(1, Hkv, n, D, dtype=BF, device="cuda").normal_()
    v = torch.empty(1, Hkv, n, D, dtype=BF, device="cuda").normal_()
    q = rand((1, 8, 1, D), BF, 1)
    kl = torch.tensor([n - 3], dtype=torch.int32, device="cuda")
    out = M.masked_gqa_attn_decode_window(q, k, v, kl, window=1000, sinks=4)
    sel = torch.cat([torch.arange(4), torch.arange(n - 1003, n - 3)]).cuda()
    vis = torch.ones(1, sel.numel(), dtype=torch.bool, device="cuda")
    check(out[0], None, attention(q[0], k[0][:, sel], v[0][:, sel], vis, D ** -0.5), 1004)


def test_one_token_tree_is_the_plain_decode(M):
    # the same mathematics as the static decode over n + 1 slots
    lens = [100, 515]
    c = Case(lens, 1, 8, 2, 128, BF, page=0)
    out = c.run(M)
    k, v = torch.nan_to_num(c.k.clone()), torch.nan_to_num(c.v.clone())
    for b, n in enumerate(lens):
        k[b, :, n], v[b, :, n] = c.kn[b, :, 0], c.vn[b, :, 0]
    ref = M.masked_gqa_attn_decode(c.q, k, v, scale=c.scale, kv_len=c.kv_len + 1)
    assert (out.float() - ref.float()).abs().max() <= 2e-2


def test_repeats_bit_for_bit(M):
    c = Case([5000, 7, 300], 8, 8, 2, 128, BF, page=16)
    a = c.run(M).clone()
    ws = torch.full((M.masked_gqa_attn_cache_workspace_size(),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(c.call(M, workspace=ws), a)  # whatever the workspace held


def test_captured_replayed_and_other_stream(M):
    a, b = Case([3000, 10], 8, 4, 2, 64, BF, page=16), Case([1, 2000], 20, 4, 2, 128, HF, page=0, window=500, sinks=3)
    wa, wb = M.new_cache_attn_workspace(), M.new_cache_attn_workspace()
    ra, rb = a.run(M).clone(), b.run(M).clone()
    oa, ob = torch.empty_like(ra), torch.empty_like(rb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.call(M, out=oa, workspace=wa, lse=None, dev_error=None)
        b.call(M, out=ob, workspace=wa, lse=None, dev_error=None)  # one after the other: one workspace
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        oa.zero_(), ob.zero_()
        graph.replay()
        with torch.cuda.stream(s):
            o2 = b.call(M, workspace=wb)
        o3 = a.call(M, stream=s, workspace=wb, out=torch.empty_like(ra))
        torch.cuda.synchronize()
        assert torch.equal(oa, ra) and torch.equal(ob, rb) and torch.equal(o2, rb) and torch.equal(o3, ra)
    # the lengths are read by the kernels: a replay follows them
    a.kv_len.copy_(torch.tensor([64, 0], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    want = a.call(M)
    assert torch.equal(oa, want)


@pytest.mark.parametrize("plain", [True, False])
def test_own_workspace_on_another_stream(M, plain):
    # a workspace that the call allocates is not given out again before the call is done
    c = Case([3000, 1500], 8, 8, 2, 64, BF, page=5)  # (the general form: partial results in the workspace)
    want = c.run(M).clone()
    s, out = torch.cuda.Stream(), torch.empty_like(want)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    c.call(M, out=out, stream=s if plain else s.cuda_stream, workspace=None)
    junk = [torch.full((M.masked_gqa_attn_cache_workspace_size(),), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and len(junk) == 3


@pytest.mark.parametrize("dtype", [BF, FP])
def test_bad_lengths_and_pages_are_reported(M, dtype):
    c = Case([100, 50], 4, 4, 2, 64, dtype, page=16, cap=128)
    good = c.run(M).clone()
    c.table[1, 1] = -1  # a page that request 1 needs
    out = c.call(M)
    assert int(c.err) == M.MGQA_ERR_INVALID_ARG
    assert torch.equal(out[0], good[0]) and torch.isfinite(out).all()
    k, v = c.k, c.v  # its slots count as masked
    sel = torch.tensor([*range(16), *range(32, 50)], device="cuda")
    kk = torch.cat([k[c.table[1, [0, 2, 3]].long()].transpose(0, 1).reshape(2, 48, 64)[:, [*range(16), *range(16, 34)]],
                    c.kn[1]], 1)
    vv = torch.cat([v[c.table[1, [0, 2, 3]].long()].transpose(0, 1).reshape(2, 48, 64)[:, [*range(16), *range(16, 34)]],
                    c.vn[1]], 1)
    vis = torch.cat([torch.ones(4, sel.numel(), dtype=torch.bool), c.seen[1]], 1).cuda()
    check(out[1], c.lse[1], attention(c.q[1], kk, vv, vis, c.scale), 50)
    c = Case([100, 50], 4, 4, 2, 64, dtype, page=0, cap=100)
    c.kv_len[1] = -7
    out = c.call(M)
    assert int(c.err) == M.MGQA_ERR_INVALID_ARG and torch.isfinite(out).all()
    c = Case([100, 30], 4, 4, 2, 64, dtype, page=0, cap=100, live=[4, 4])
    good = c.run(M).clone()
    c.kv_len[0], c.live[1] = 101, 9  # clamped
    out = c.call(M)
    assert int(c.err) == M.MGQA_ERR_INVALID_ARG and torch.equal(out, good)


def test_rows_behind_are_left_alone(M):
    # outputs in a larger buffer: only [B, Hq, T] rows are written, nothing of the caches
    c = Case([70, 9], 5, 4, 2, 64, BF, page=16)
    want = c.run(M)
    big = torch.full((2, 4, 9, 64), 3.0, dtype=BF, device="cuda")
    k0, v0 = c.k.clone(), c.v.clone()
    c.call(M, out=big[:, :, 2:7])
    assert torch.equal(big[:, :, 2:7], want)
    assert (big[:, :, :2] == 3).all() and (big[:, :, 7:] == 3).all()
    assert torch.equal(c.k.view(torch.int16), k0.view(torch.int16)) and torch.equal(c.v.view(torch.int16), v0.view(torch.int16))
