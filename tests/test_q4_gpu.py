"""A cache held in 4 bits: rows quantised as they are appended, bit for bit, and
attention of the last tokens over it against 64 bits. Everything that no query may
see is NaN or a page index far outside the pool."""
import random

import pytest
import torch

from _q4_ref import check_attention, records, sees, values

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
INVALID = 1


@pytest.fixture(scope="module")
def M():
    import masked_gqa_attention_gb300 as M
    M.build_library()
    return M


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rand(shape, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


class Case:
    """A cache of records, its requests and queries. page 0: the static cache."""

    def __init__(self, lens, T, Hq, Hkv, D, dtype, *, page=0, cap=None, window=0, sinks=0, seed=1, scale=None,
                 gain=None, slots_first=False):
        rng = random.Random(seed)
        self.lens, self.T, self.window, self.sinks, self.page = lens, T, window, sinks, page
        self.scale = D ** -0.5 if scale is None else scale
        self.kv_len = i32(lens)
        B, cap = len(lens), max([1, *lens]) + 5 if cap is None else cap
        self.q = rand((B, Hq, T, D), dtype, seed)
        gain = 1.0 if gain is None else gain
        self.rec = []  # [B][Hkv, n, rec] of K and V
        self.k = self.v = None
        R = D // 2 + 16
        if page:
            mp = -(-cap // page)
            need = [-(-n // page) for n in lens]
            pages = sum(need) + 4
            order = list(range(pages))
            rng.shuffle(order)
            table = torch.full((B, mp), 2 ** 30, dtype=torch.int32)
            at = 0
            for b, m in enumerate(need):
                table[b, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
                at += m
            self.table = table.cuda()
            shape = (pages, Hkv, page, R)
        else:
            self.table, shape = None, (B, Hkv, cap, R)
        if slots_first:  # the slots of a page apart: [.., slots, Hkv, rec]
            self.k, self.v = (torch.full((shape[0], shape[2], Hkv, R), 255, dtype=torch.uint8, device="cuda").transpose(1, 2)
                              for _ in range(2))
        else:
            self.k, self.v = (torch.full(shape, 255, dtype=torch.uint8, device="cuda") for _ in range(2))  # NaN scales
        seen = [sees(n, T, window, sinks, "cuda") for n in lens]
        for b, n in enumerate(lens):
            rows = [records(rand((Hkv, n, D), FP, seed * 100 + 2 * b + x) * gain) for x in range(2)]
            self.rec.append(rows)
            j = torch.nonzero(seen[b].any(0)).view(-1)
            if page:
                pg, sl = self.table[b].long()[j // page], j % page
                gone = sorted(set(range(need[b])) - set((j // page).tolist()))
                self.table[b, gone] = -2 ** 30  # pages without a visible slot are not looked at
            else:
                pg, sl = torch.full_like(j, b), j
            for x, r in ((self.k, rows[0]), (self.v, rows[1])):
                x[pg, :, sl] = r[:, j].transpose(0, 1)
        self.seen = seen
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.lse = torch.full((B, Hq, T), 777.0, device="cuda")

    def call(self, M, **kw):
        kw = {**dict(window=self.window, sinks=self.sinks, page_table=self.table, scale=self.scale, lse=self.lse,
                     dev_error=self.err), **kw}
        return M.masked_gqa_attn_decode_q4(self.q, self.k, self.v, self.kv_len, **kw)

    def check(self, out, lse=None):
        lse = self.lse if lse is None else lse
        for b in range(len(self.lens)):
            check_attention(out[b], lse[b], self.q[b], *self.rec[b], self.seen[b], self.scale, f"request {b}")

    def run(self, M, **kw):
        out = self.call(M, **kw)
        assert int(self.err) == 0
        self.check(out)
        again = self.call(M, **kw)
        assert torch.equal(out, again)
        return out


# ---- append ------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D", [64, 128])
def test_records_of_awkward_rows(M, D, dtype):
    """Every group with a trait of its own: constants, zeros of both signs, tiny and huge ranges, outliers, ties."""
    x = rand((1, 40, 3, D), FP, 7)
    x[0, 0] = 0.0
    x[0, 1] = -0.0
    x[0, 2] = 3.7
    x[0, 3] = -1e-9
    x[0, 4] *= 1e-6
    x[0, 5] *= 3e4 / 4
    x[0, 6, :, 5] = 1000.0
    x[0, 7] = x[0, 7].abs() + 500.0
    x[0, 8] = torch.arange(3 * D, device="cuda").view(3, D) % (D // 4)  # halves of a step and whole ones
    x[0, 9] = (torch.arange(3 * D, device="cuda").view(3, D) % 31 + 1) / 2 - 8
    if dtype != HF:
        x[0, 10] *= 1e7
        x[0, 11] = x[0, 11] * 1e5 + 3e5
        x[0, 12] = -1e30
        x[0, 13, :, 1::2] = 2e38
    x = x.transpose(1, 2).to(dtype)  # [1, 3, 40, D]
    k, v = (torch.zeros(1, 3, 64, D // 2 + 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    lens, new = i32([11]), i32([0])
    M.masked_gqa_cache_append_q4(k, v, x, -x, lens, new)
    assert int(new) == 51
    assert torch.equal(k[:, :, 11:51], records(x)) and torch.equal(v[:, :, 11:51], records(-x))
    assert (k[:, :, :11] == 0).all() and (k[:, :, 51:] == 0).all()
    got, _ = values(k[:, :, 11:51])
    near = (x.double().abs().amax(-1) < 6e4)  # within half a step, and the roundings of the step and the least value
    par = k[:, :, 11:51, D // 2:].contiguous().view(HF).double()
    step = par[..., :4].repeat_interleave(D // 4, -1)
    tol = (0.5 + 15 * 2.0 ** -11 + 2.0 ** -20) * step + 2.0 ** -11 * x.double().abs().amax(-1, keepdim=True) + 2.0 ** -20
    assert ((got - x.double()).abs() <= tol)[near].all()


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [0, 1, 5, 16, 64])
@pytest.mark.parametrize("layers,T,Hkv,chosen", [(1, 1, 3, False), (3, 1, 8, False), (2, 7, 3, True), (1, 150, 3, False),
                                                 (1, 40, 1, False), (2, 33, 40, False)])
def test_append_writes_what_it_should(M, dtype, D, page, layers, T, Hkv, chosen):
    rng = random.Random(page + T)
    B, cap = 4, 200
    lens = [0, 13, cap - T, 31]
    R = D // 2 + 16
    if page:
        mp = -(-cap // page)
        pages = B * mp
        table = torch.randperm(pages).int().view(B, mp).cuda()
        k, v = (torch.randint(0, 256, (layers, pages, Hkv, page, R), dtype=torch.uint8, device="cuda") for _ in range(2))
    else:
        table = None
        k, v = (torch.randint(0, 256, (layers, B, Hkv, cap, R), dtype=torch.uint8, device="cuda") for _ in range(2))
    kn, vn = (rand((layers, B, T, Hkv, D), dtype, 3 + x).transpose(2, 3) for x in range(2))
    index = count = None
    counts, paths = [T] * B, [list(range(T))] * B
    if chosen:
        counts = [0, 3, T, 1]
        paths = [rng.sample(range(T), c) for c in counts]
        index, count = i32([p + [-9] * (T - len(p)) for p in paths]), i32(counts)
    wk, wv = k.clone(), v.clone()
    rk, rv = records(kn), records(vn)
    for b in range(B):
        j = lens[b] + torch.arange(counts[b], device="cuda")
        row, slot = (table[b].long()[j // page], j % page) if page else (torch.full_like(j, b), j)
        for x, r in ((wk, rk), (wv, rv)):
            x[:, row, :, slot] = r[:, b][:, :, paths[b]].permute(2, 0, 1, 3)
    out, err = i32([-1] * B), i32([0])
    M.masked_gqa_cache_append_q4(k, v, kn, vn, i32(lens), out, index=index, count=count, page_table=table, dev_error=err)
    assert out.tolist() == [n + c for n, c in zip(lens, counts)] and int(err) == 0
    assert torch.equal(k, wk) and torch.equal(v, wv)


@pytest.mark.parametrize("page", [0, 16])
def test_append_takes_rows_and_caches_of_any_strides(M, page):
    """K and V, old rows and new ones, each with strides of its own; new rows expanded over the requests."""
    B, Hkv, D, T, R = 3, 2, 128, 5, 80
    table = torch.randperm(12).int().view(3, 4).cuda() if page else None
    n = 12 if page else B
    k = torch.zeros(n, 16 if page else 64, Hkv, R, dtype=torch.uint8, device="cuda").transpose(1, 2)
    v = torch.zeros(n, Hkv + 1, 16 if page else 64, R + 16, dtype=torch.uint8, device="cuda")[:, :Hkv, :, :R]
    kn = rand((1, T, Hkv, D), BF, 1).transpose(1, 2).expand(B, -1, -1, -1)
    vn = rand((B, Hkv, T + 2, D + 8), BF, 2)[:, :, :T, :D]
    lens, new = i32([3, 0, 14]), i32([0] * 3)
    M.masked_gqa_cache_append_q4(k, v, kn, vn, lens, new, page_table=table)
    assert new.tolist() == [8, 5, 19]
    for b in range(B):
        j = int(lens[b]) + torch.arange(T, device="cuda")
        pg, sl = (table[b].long()[j // 16], j % 16) if page else (torch.full_like(j, b), j)
        assert torch.equal(k[pg, :, sl].transpose(0, 1), records(kn[b])) and torch.equal(v[pg, :, sl].transpose(0, 1), records(vn[b]))


def test_append_reports_what_it_cannot_store(M):
    k, v = (torch.zeros(6, 2, 16, 48, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = i32([[0, 1], [2, 9], [3, -1]])
    x = rand((3, 2, 4, 64), BF, 1)
    for lens, index, count, want in (([29, 0, 0], None, None, [29, 4, 4]), ([0, 14, 0], None, None, [4, 18, 4]),
                                     ([0, 0, 0], [[0, 1, 2, 3], [0, 4, 1, 2], [3, 2, 1, 0]], None, [4, 4, 4]),
                                     ([0, 0, 0], None, [4, 5, -1], [4, 0, 0]), ([-1, 33, 0], None, None, [-1, 33, 4])):
        err, out = i32([0]), i32([0, 0, 0])
        M.masked_gqa_cache_append_q4(k, v, x, x, i32(lens), out, page_table=table, dev_error=err,
                                     index=None if index is None else i32(index), count=None if count is None else i32(count))
        assert int(err) == INVALID and out.tolist() == want, (lens, out.tolist())
    assert (k[4:] == 0).all()


def test_plain_append_refuses_records(M):
    k = torch.zeros(2, 2, 8, 48, dtype=torch.uint8, device="cuda")
    for D in (24, 48, 64):
        for kind in (torch.uint8, HF):
            x = torch.zeros(2, 2, 1, D, device="cuda").to(kind)
            with pytest.raises(ValueError):
                M.masked_gqa_cache_append(k, k, x, x, i32([0, 0]), i32([0, 0]))


def test_append_of_a_few_of_many_rows(M):
    """Counts far below T: the rows behind them are not looked at."""
    B, Hkv, D, T = 3, 2, 64, 500
    k, v = (torch.zeros(B, Hkv, 600, 48, dtype=torch.uint8, device="cuda") for _ in range(2))
    x = rand((B, Hkv, T, D), HF, 3)
    counts, new = [0, 5, 131], i32([0] * B)
    for b, n in enumerate(counts):
        x[b, :, n:] = float("nan")
    M.masked_gqa_cache_append_q4(k, v, x, -x, i32([7, 0, 90]), new, count=i32(counts))
    assert new.tolist() == [7, 5, 221]
    for b, (a, n) in enumerate(zip([7, 0, 90], counts)):
        assert torch.equal(k[b, :, a:a + n], records(x[b, :, :n])) and torch.equal(v[b, :, a:a + n], records(-x[b, :, :n]))
        assert (k[b, :, a + n:] == 0).all()


# ---- attention -----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (3, 3), (7, 1), (16, 2), (32, 2), (48, 2)])
def test_one_token(M, dtype, D, Hq, Hkv):
    Case([0, 1, 2, 31, 32, 33, 64, 100, 515, 1000], 1, Hq, Hkv, D, dtype, page=16).run(M)


@pytest.mark.parametrize("page", [0, 1, 2, 3, 8, 16, 24, 32, 40, 64, 100, 1024])
@pytest.mark.parametrize("D,dtype", [(64, BF), (128, HF), (128, FP)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5)])
def test_pages_of_any_size(M, page, D, dtype, window, sinks):
    Case([700, 1, 333, 0, 65], 3, 8, 2, D, dtype, page=page, window=window, sinks=sinks).run(M)


@pytest.mark.parametrize("T", [1, 2, 5, 8, 16, 33, 64, 256])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(4, 1, 128, BF), (10, 2, 64, HF), (2, 2, 128, FP)])
def test_the_last_tokens(M, T, Hq, Hkv, D, dtype):
    """More tokens than slots leave rows that see nothing."""
    Case([0, 1, T - 1, T, T + 1, 300, 77], T, Hq, Hkv, D, dtype, page=16).run(M)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (32, 0), (33, 4), (64, 40), (100, 300), (5, 0), (2 ** 31 - 1, 7),
                                          (0, 2 ** 31 - 1)])
@pytest.mark.parametrize("T,page,D", [(1, 16, 64), (6, 0, 128), (40, 8, 64)])
def test_windows(M, window, sinks, T, page, D):
    Case([400, 33, 7, 0, 129, 260], T, 6, 2, D, BF, page=page, window=window, sinks=sinks).run(M)


@pytest.mark.parametrize("lens,T,Hq,Hkv,D,dtype,page", [
    ([60000, 5, 31000], 1, 8, 2, 128, BF, 16),
    ([60000, 5, 31000], 4, 8, 2, 128, FP, 64),
    ([100003], 1, 32, 8, 64, HF, 0),
    ([100003], 8, 32, 8, 64, BF, 24),
    ([9000 + 61 * i for i in range(24)], 1, 32, 8, 128, BF, 16),
    ([1 + 997 * i % 7000 for i in range(70)], 2, 12, 4, 64, BF, 32),
    ([3000] * 300, 1, 4, 4, 128, HF, 16),
    ([50000, 3, 20011], 5, 16, 4, 128, BF, 16),   # blocks of 32 rows: one in part,
    ([50000, 30, 20011], 7, 40, 4, 128, HF, 40),  # three with the last in part,
    ([50000, 0, 44000], 16, 8, 4, 64, HF, 0),     # one whole
])
@pytest.mark.parametrize("window,sinks", [(0, 0), (9000, 70)])
def test_long_calls_are_cut_and_joined(M, lens, T, Hq, Hkv, D, dtype, page, window, sinks):
    c = Case(lens, T, Hq, Hkv, D, dtype, page=page, window=window, sinks=sinks)
    ws = M.new_cache_attn_workspace()
    ws.fill_(255)
    c.run(M, workspace=ws)


def test_a_wide_table_of_short_requests(M):
    Case([40, 3, 0, 900], 2, 8, 2, 128, BF, page=16, cap=200000).run(M)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
def test_scales(M, dtype, scale):
    Case([300, 40], 4, 8, 2, 64, dtype, page=16, scale=scale).run(M)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("gain", [1e-4, 100.0, 5000.0])
def test_small_and_large_values(M, dtype, gain):
    c = Case([300, 40], 2, 8, 2, 128, dtype, page=16, gain=gain, scale=1.0 / gain)
    if dtype == HF and gain > 4000:
        pytest.skip("the outputs pass fp16")
    c.run(M)


@pytest.mark.parametrize("dtype,power", [(BF, -90), (BF, 90), (FP, -100), (FP, 100), (HF, -18), (HF, 13)])
def test_queries_of_any_size(M, dtype, power):
    """Each row is scaled by itself: rows of very different size beside one another."""
    c = Case([300, 40], 2, 8, 2, 128, dtype, page=16)
    c.q[:, ::2] *= 2.0 ** power
    c.run(M)


def test_features_and_values_of_very_different_size(M):
    g = torch.exp(2 * rand((128,), FP, 3))
    Case([700, 65], 3, 8, 2, 128, BF, page=16, gain=g, scale=0.01).run(M)
    c = Case([700], 1, 8, 2, 128, FP, page=16)
    rows = torch.exp(3 * rand((1, 2, 700, 1), FP, 5)).expand(1, 2, 700, 128) * rand((1, 2, 700, 128), FP, 6)
    c.rec[0][1] = records(rows[0].clamp(-6e4, 6e4))  # later values larger than earlier ones, and back
    j = torch.arange(700, device="cuda")
    c.v[c.table[0].long()[j // 16], :, j % 16] = c.rec[0][1].transpose(0, 1)
    c.run(M)


@pytest.mark.parametrize("page", [0, 16])
def test_slots_apart(M, page):
    Case([300, 45, 0], 2, 8, 2, 128, BF, page=page, slots_first=True).run(M)


@pytest.mark.parametrize("page", [0, 16])
def test_keys_and_values_with_strides_of_their_own(M, page):
    c = Case([300, 45, 0], 2, 8, 2, 64, HF, page=page)
    wide = torch.full((*c.v.shape[:3], 80), 255, dtype=torch.uint8, device="cuda")
    wide[..., 16:64] = c.v
    c.v = wide[..., 16:64]
    c.run(M)
    c.k = c.k.transpose(1, 2).contiguous().transpose(1, 2)
    c.run(M)


def test_queries_and_outputs_with_strides(M):
    c = Case([300, 45], 3, 8, 2, 64, BF, page=16)
    c.q = c.q.transpose(1, 2).contiguous().transpose(1, 2)
    out = torch.zeros(2, 3, 8, 64, dtype=BF, device="cuda").transpose(1, 2)
    c.call(M, out=out)
    c.check(out)


def test_one_cache_for_every_request(M):
    """Records expanded over the requests (a stride of 0)."""
    c = Case([300], 2, 8, 2, 128, BF)
    q = rand((5, 8, 2, 128), BF, 9)
    lse = torch.empty(5, 8, 2, device="cuda")
    out = M.masked_gqa_attn_decode_q4(q, c.k.expand(5, -1, -1, -1), c.v.expand(5, -1, -1, -1), i32([300] * 5), lse=lse)
    for b in range(5):
        check_attention(out[b], lse[b], q[b], *c.rec[0], c.seen[0], c.scale)


@pytest.mark.parametrize("page", [0, 16])
def test_bad_lengths_and_pages(M, page):
    c = Case([100, 100, 100], 2, 8, 2, 128, BF, page=page, cap=112)
    c.kv_len = i32([-3, 100, 500])
    out = c.call(M)
    assert int(c.err) == INVALID
    assert (out[0] == 0).all() and (c.lse[0] == -float("inf")).all()
    check_attention(out[1], c.lse[1], c.q[1], *c.rec[1], c.seen[1], c.scale)
    if page:
        c = Case([100, 100], 2, 8, 2, 128, BF, page=page)
        c.table[0, 2] = 10 ** 6
        c.table[1, 0] = -1
        out = c.call(M)
        assert int(c.err) == INVALID
        for b, hole in ((0, slice(32, 48)), (1, slice(0, 16))):
            vis = c.seen[b].clone()
            vis[:, hole] = False  # the slots of a missing page count as masked
            check_attention(out[b], c.lse[b], c.q[b], *c.rec[b], vis, c.scale)


def test_offsets_past_32_bits(M):
    pages, page, Hkv, D = 430000, 16, 8, 128  # 4.4 GB a tensor
    k, v = (torch.empty(pages, Hkv, page, 80, dtype=torch.uint8, device="cuda") for _ in range(2))
    c = Case([90, 40], 2, 8, Hkv, D, BF, page=page)
    table = c.table.clone()
    for b, n in enumerate(c.lens):
        for i in range(-(-n // page)):
            to = pages - 1 - 7 * i - b
            k[to], v[to] = c.k[c.table[b, i]], c.v[c.table[b, i]]
            table[b, i] = to
    c.k, c.v, c.table = k, v, table
    c.run(M)
    x = rand((2, Hkv, 3, D), BF, 4)
    out = i32([0, 0])
    M.masked_gqa_cache_append_q4(k, v, x, x, i32([40, 32]), out, page_table=table)
    at = int(table[0, 2])
    assert torch.equal(k[at, :, 8:11], records(x[0])) and torch.equal(v[at, :, 8:11], records(x[0]))


def test_captured_and_replayed_with_new_lengths(M):
    c = Case([3000, 200, 1], 1, 8, 2, 128, BF, page=16, cap=40000)
    ws, out = M.new_cache_attn_workspace(), torch.empty_like(c.q)
    c.call(M, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(M, out=out, workspace=ws)
    for lens in ([3000, 200, 1], [1500, 0, 1], [77, 199, 1]):
        c.kv_len.copy_(i32(lens))
        out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        for b, n in enumerate(lens):
            check_attention(out[b], c.lse[b], c.q[b], c.rec[b][0][:, :n], c.rec[b][1][:, :n],
                            sees(n, 1, 0, 0, "cuda"), c.scale)


def test_calls_at_the_same_time(M):
    cases = [Case([20000 + 31 * i, 700], 1, 16, 4, 128, BF, page=16, seed=i) for i in range(2)]
    outs = [torch.empty_like(c.q) for c in cases]
    wss = [M.new_cache_attn_workspace() for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, o, w, s in zip(cases, outs, wss, streams):
            c.call(M, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check(o)


def test_on_another_stream_with_its_own_memory(M):
    c = Case([9000, 700], 1, 16, 4, 128, BF, page=16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [c.call(M, stream=s) for _ in range(4)]
    torch.cuda.synchronize()
    for o in outs:
        c.check(o)


def test_a_step_reads_what_was_just_appended(M):
    """Append and attention in turn, lengths between two buffers, with nothing between them."""
    B, Hkv, D, page, steps = 3, 2, 128, 16, 40
    lens = [0, 17, 100]
    mp = 10
    table = torch.randperm(B * mp).int().view(B, mp).cuda()
    k, v = (torch.full((B * mp, Hkv, page, 80), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    bufs = [i32(lens), i32([0] * B)]
    first = [rand((B, Hkv, max(lens), D), BF, 1 + x) for x in range(2)]
    M.masked_gqa_cache_append_q4(k, v, *first, i32([0] * B), bufs[0], count=i32(lens), page_table=table)
    new = [rand((steps, B, Hkv, 1, D), BF, 3 + x) for x in range(2)]
    q = rand((steps, B, 8, 1, D), BF, 5)
    outs, lses = [], []
    ws = M.new_cache_attn_workspace()
    for t in range(steps):
        a, z = bufs[t % 2], bufs[(t + 1) % 2]
        M.masked_gqa_cache_append_q4(k, v, new[0][t], new[1][t], a, z, page_table=table)
        lses.append(torch.empty(B, 8, 1, device="cuda"))
        outs.append(M.masked_gqa_attn_decode_q4(q[t], k, v, z, page_table=table, workspace=ws, lse=lses[-1]))
    torch.cuda.synchronize()
    for t in (0, 1, 7, steps - 1):
        for b, n in enumerate(lens):
            rec = [records(torch.cat([first[x][b, :, :n], new[x][:t + 1, b, :, 0].transpose(0, 1)], 1)) for x in range(2)]
            check_attention(outs[t][b], lses[t][b], q[t, b], *rec, sees(n + t + 1, 1, 0, 0, "cuda"), D ** -0.5, f"step {t}")


def test_requests_of_records_fork_and_pack(M):
    """fork and compact take a cache of records as it is."""
    c = Case([50, 33, 0, 0], 1, 8, 2, 64, BF, page=16, cap=96)
    table = torch.where((c.table < 0) | (c.table >= c.k.shape[0]), -1, c.table)
    k, v = (torch.cat([x, torch.zeros(12, *x.shape[1:], dtype=torch.uint8, device="cuda")]) for x in (c.k, c.v))
    ref = torch.zeros(k.shape[0], dtype=torch.int32, device="cuda")
    ref[table[table >= 0].long()] = 1
    M.masked_gqa_cache_fork(k, v, table, c.kv_len, ref, i32([0, 1]), i32([2, 3]), extra=4)
    M.masked_gqa_cache_fork(k, v, table, c.kv_len, ref, i32([-1]), i32([1]))
    M.masked_gqa_cache_compact(k, v, table, ref)
    assert c.kv_len.tolist() == [50, 0, 50, 33]
    out = M.masked_gqa_attn_decode_q4(c.q, k, v, c.kv_len, page_table=table, lse=c.lse)
    for b, src in ((0, 0), (2, 0), (3, 1)):
        check_attention(out[b], c.lse[b], c.q[b], *c.rec[src], c.seen[src], c.scale)
    assert (out[1] == 0).all()
