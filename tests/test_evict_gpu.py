"""What attention looks at, summed up against 64 bits, and the eviction of the slots
with the least, exactly."""
import math
import random

import pytest
import torch

from _q4_ref import check_weights, kept_slots, records, scores, sees, values

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


# ---- accumulated weights -----------------------------------------------------------------

class Weights:
    def __init__(self, lens, T, Hq, Hkv, D, dtype, *, q4=False, page=0, cap=None, window=0, sinks=0, seed=1, extra=3):
        rng = random.Random(seed)
        B, cap = len(lens), max([1, *lens]) + 5 if cap is None else cap
        self.lens, self.window, self.sinks, self.scale, self.q4 = lens, window, sinks, D ** -0.5, q4
        self.kv_len, self.q = i32(lens), rand((B, Hq, T, D), dtype, seed)
        self.seen = [sees(n, T, window, sinks, "cuda") for n in lens]
        row = D // 2 + 16 if q4 else D
        if page:
            need = [-(-n // page) for n in lens]
            pages = sum(need) + 3
            order = list(range(pages))
            rng.shuffle(order)
            table = torch.full((B, -(-cap // page)), 2 ** 30, dtype=torch.int32)
            at = 0
            for b, m in enumerate(need):
                table[b, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
                at += m
            self.table, shape = table.cuda(), (pages, Hkv, page, row)
        else:
            self.table, shape = None, (B, Hkv, cap, row)
        if q4:
            self.k = torch.full(shape, 255, dtype=torch.uint8, device="cuda")
        else:
            self.k = torch.full(shape, float("nan"), device="cuda").to(dtype)
        self.keys, lse = [], []
        for b, n in enumerate(lens):
            x = rand((Hkv, n, D), FP if q4 else dtype, seed * 50 + b)
            x = records(x) if q4 else x
            self.keys.append(values(x) if q4 else (x.double(), x.double().abs()))
            j = torch.nonzero(self.seen[b].any(0)).view(-1)
            pg, sl = (self.table[b].long()[j // page], j % page) if page else (torch.full_like(j, b), j)
            self.k[pg, :, sl] = x[:, j].transpose(0, 1)
            if page:
                self.table[b, sorted(set(range(need[b])) - set((j // page).tolist()))] = -5
            s, _ = scores(self.q[b], *self.keys[b], self.seen[b], self.scale)
            lse.append(torch.logsumexp(s, -1) if n else torch.full((Hq, T), -math.inf, dtype=torch.float64, device="cuda"))
        self.lse = torch.stack(lse).float()
        self.before = torch.rand((B, Hkv, (self.table.shape[1] * page if page else cap) + extra), device="cuda")
        self.err = i32([0])

    def call(self, M, weight, **kw):
        return M.masked_gqa_attn_cache_weights(self.q, self.k, self.kv_len, self.lse, weight, **{
            **dict(window=self.window, sinks=self.sinks, page_table=self.table, dev_error=self.err), **kw})

    def run(self, M):
        got = self.call(M, self.before.clone())
        assert int(self.err) == 0
        for b in range(len(self.lens)):
            check_weights(got[b], self.before[b], self.q[b], *self.keys[b], self.seen[b], self.lse[b], self.scale,
                          f"request {b}")
        assert torch.equal(got, self.call(M, self.before.clone()))
        return got


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (8, 2, 128), (9, 3, 64), (32, 2, 128), (7, 1, 128)])
def test_weights_of_one_token(M, dtype, q4, Hq, Hkv, D):
    Weights([0, 1, 15, 16, 17, 100, 515], 1, Hq, Hkv, D, dtype, q4=q4, page=16).run(M)


@pytest.mark.parametrize("T", [1, 3, 8, 40, 256])
@pytest.mark.parametrize("dtype,q4,D", [(BF, False, 128), (HF, False, 64), (FP, False, 64), (FP, False, 128), (BF, True, 64),
                                        (FP, True, 128)])
def test_weights_of_the_last_tokens(M, T, dtype, q4, D):
    Weights([0, 1, T, 300, 77], T, 8, 2, D, dtype, q4=q4, page=8).run(M)


@pytest.mark.parametrize("page", [0, 1, 3, 16, 24, 64])
@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 5), (64, 200), (2 ** 31 - 1, 0)])
def test_weights_under_a_window(M, page, q4, window, sinks):
    Weights([333, 0, 12, 70], 5, 4, 2, 64, BF, q4=q4, page=page, window=window, sinks=sinks).run(M)


@pytest.mark.parametrize("dtype,q4", [(BF, False), (BF, True), (FP, False)])
def test_weights_of_long_requests(M, dtype, q4):
    Weights([40000, 3, 9001], 2, 8, 4, 128, dtype, q4=q4, page=16).run(M)


def test_weights_of_rows_without_any(M):
    """A log-sum of -inf gives nothing, whatever the row would see."""
    w = Weights([100, 40], 4, 8, 2, 64, BF, page=16)
    w.lse[0, 3] = -math.inf
    w.lse[1, :, 2] = -math.inf
    w.run(M)


def test_weights_of_bad_lengths_and_pages(M):
    w = Weights([100, 100, 60], 2, 8, 2, 64, BF, page=16, cap=112)
    w.kv_len = i32([-1, 100, 60])
    w.table[2, 1] = 10 ** 6
    got = w.call(M, w.before.clone())
    assert int(w.err) == INVALID
    assert torch.equal(got[0], w.before[0]) and torch.equal(got[2][:, 16:32], w.before[2][:, 16:32])
    check_weights(got[1], w.before[1], w.q[1], *w.keys[1], w.seen[1], w.lse[1], w.scale)


def test_weights_with_strides_and_an_expanded_cache(M):
    w = Weights([200], 2, 8, 2, 64, BF)
    k = w.k[0].transpose(0, 1).contiguous().transpose(0, 1)[None].expand(3, -1, -1, -1)
    q, lse, wide = w.q.expand(3, -1, -1, -1), w.lse.expand(3, -1, -1).contiguous(), torch.zeros(2, 3, 400, device="cuda")
    weight = wide.transpose(0, 1)[..., :210]
    M.masked_gqa_attn_cache_weights(q, k, i32([200] * 3), lse, weight)
    for b in range(3):
        check_weights(weight[b], torch.zeros_like(weight[b]), w.q[0], *w.keys[0], w.seen[0], w.lse[0], w.scale)
    assert (wide[..., 210:] == 0).all()


# ---- eviction ------------------------------------------------------------------------------

class Evict:
    def __init__(self, lens, budget, sinks, recent, *, layers=1, Hkv=2, D=64, dtype=BF, page=0, cap=None, seed=1,
                 weights="some", flat=False):
        self.lens, self.budget, self.sinks, self.recent, self.page, self.flat = lens, budget, sinks, recent, page, flat
        rng = random.Random(seed)
        g = torch.Generator("cuda").manual_seed(seed)
        B, cap = len(lens), max([1, *lens]) + 3 if cap is None else cap
        if page:
            need = [-(-n // page) for n in lens]
            held = [m + rng.randint(0, 2) for m in need]
            mp = max(-(-cap // page), *held)
            pages = sum(held) + 5
            order = list(range(pages))
            rng.shuffle(order)
            table = torch.full((B, mp), -1, dtype=torch.int32)
            at = 0
            for b, m in enumerate(held):
                table[b, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
                at += m
            self.table, self.ref = table.cuda(), torch.zeros(pages, dtype=torch.int32, device="cuda")
            self.ref[self.table[self.table >= 0].long()] = 1
            shape, cap = (layers, pages, Hkv, page), mp * page
        else:
            self.table, self.ref, shape = None, None, (layers, B, Hkv, cap)
        if dtype == torch.uint8:
            self.k, self.v = (torch.randint(0, 256, (*shape, D // 2 + 16), generator=g, device="cuda", dtype=torch.uint8)
                              for _ in range(2))
        else:
            self.k, self.v = (torch.randn((*shape, D), generator=g, device="cuda").to(dtype) for _ in range(2))
        w = torch.exp(2 * torch.randn((layers, B, Hkv, cap), generator=g, device="cuda"))
        if weights == "ties":
            w = torch.randint(0, 3, w.shape, generator=g, device="cuda").float()
        elif weights == "equal":
            w = torch.full_like(w, 0.25)
        elif weights == "odd":  # signs, infinities, NaN, zeros of both signs, subnormals
            odd = torch.tensor([0.0, -0.0, -1.0, 1.0, math.inf, -math.inf, math.nan, 1e-42, -1e-42, 3e38, 1e-3],
                               device="cuda")
            w = odd[torch.randint(0, len(odd), w.shape, generator=g, device="cuda")]
        self.w, self.host, self.kv_len, self.err = w, w.cpu(), i32(lens), i32([0])

    def want(self, layer, b, g):
        return kept_slots(self.host[layer, b, g], self.lens[b], self.budget, self.sinks, self.recent)

    def place(self, table, b, j):
        j = torch.as_tensor(j, device="cuda", dtype=torch.long)
        return (table[b].long()[j // self.page], j % self.page) if self.page else (torch.full_like(j, b), j)

    def run(self, M, *, in_place=True, with_ref=False, **kw):
        k, v, w, lens = self.k.clone(), self.v.clone(), self.w.clone(), self.kv_len.clone()
        table = None if self.table is None else self.table.clone()
        ref = self.ref.clone() if with_ref else None
        w_out = w if in_place else torch.full_like(w, 9.0)
        len_out = lens if in_place else torch.full_like(lens, -7)
        pick = (lambda x: x[0]) if self.flat else (lambda x: x)
        M.masked_gqa_cache_evict(pick(k), pick(v), pick(w), lens, budget=self.budget, sinks=self.sinks, recent=self.recent,
                                 page_table=table, ref=ref, weight_out=pick(w_out), kv_len_out=len_out,
                                 dev_error=self.err, **kw)
        assert int(self.err) == 0
        assert len_out.tolist() == [min(n, self.budget) for n in self.lens]
        wk, wv, ww = self.k.clone(), self.v.clone(), (self.w if in_place else torch.full_like(self.w, 9.0)).clone()
        for b, n in enumerate(self.lens):
            for layer in range(self.w.shape[0]):
                for g in range(self.w.shape[2]):
                    keep = self.want(layer, b, g)
                    ww[layer, b, g, :n] = 0.0
                    ww[layer, b, g, :len(keep)] = self.w[layer, b, g, keep]
                    if n <= self.budget:
                        continue
                    (pa, sa), (pb, sb) = self.place(self.table, b, keep), self.place(self.table, b, range(len(keep)))
                    wk[layer, pb, g, sb], wv[layer, pb, g, sb] = self.k[layer, pa, g, sa], self.v[layer, pa, g, sa]
        assert torch.equal(k, wk) and torch.equal(v, wv)
        assert torch.equal(w_out.view(torch.int32), ww.view(torch.int32))
        if with_ref:
            wt, wr = self.table.clone(), self.ref.clone()
            for b, n in enumerate(self.lens):
                if n > self.budget:
                    gone = wt[b, -(-self.budget // self.page):]
                    wr[gone[gone >= 0].long()] -= 1
                    gone.fill_(-1)
            assert torch.equal(table, wt) and torch.equal(ref, wr)
        elif table is not None:
            assert torch.equal(table, self.table)


@pytest.mark.parametrize("weights", ["some", "ties", "equal", "odd"])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (64, 4, 16), (64, 0, 0), (64, 30, 34),
                                                 (100, 0, 99), (300, 8, 0)])
@pytest.mark.parametrize("page", [0, 16])
def test_what_stays(M, weights, budget, sinks, recent, page):
    Evict([0, 1, 64, 65, 300, 301, 700, 2], budget, sinks, recent, page=page, weights=weights).run(M)


@pytest.mark.parametrize("dtype", [BF, HF, FP, torch.uint8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [0, 1, 5, 16, 64])
def test_rows_of_any_kind(M, dtype, D, page):
    c = Evict([200, 31, 129], 77, 4, 20, layers=3, Hkv=3, D=D, dtype=dtype, page=page)
    c.run(M)
    c.run(M, in_place=False)
    if page:
        c.run(M, with_ref=True)


@pytest.mark.parametrize("lens,budget,layers,Hkv,weights", [
    ([33000], 4096, 1, 2, "some"), ([70001], 30000, 1, 1, "some"), ([20000, 100, 5000], 4999, 1, 3, "ties"),
    ([9000] * 20, 2048, 1, 8, "some"), ([4096], 4095, 2, 8, "equal"), ([12289], 1, 1, 1, "some"),
    ([1030] * 5, 1024, 9, 4, "some"), ([330000], 5000, 1, 1, "some"), ([50000, 41000], 300, 1, 2, "ties")])
@pytest.mark.parametrize("page", [0, 64])
def test_long_requests(M, lens, budget, layers, Hkv, weights, page):
    Evict(lens, budget, min(4, budget - 1), min(256, budget // 2), layers=layers, Hkv=Hkv, D=128, page=page,
          weights=weights).run(M)


def test_four_dimensions(M):
    Evict([90, 20], 40, 2, 8, page=16, flat=True).run(M, with_ref=True)
    Evict([90, 20], 40, 2, 8, flat=True).run(M, in_place=False)


def test_trailing_pages_go_back_and_serve_again(M):
    c = Evict([100, 20], 40, 2, 8, page=16)
    k, v, w, lens, table, ref = (x.clone() for x in (c.k, c.v, c.w, c.kv_len, c.table, c.ref))
    free = int((ref == 0).sum())
    M.masked_gqa_cache_evict(k, v, w, lens, budget=40, sinks=2, recent=8, page_table=table, ref=ref)
    assert int((ref == 0).sum()) > free and (table[0, 3:] == -1).all()
    M.masked_gqa_cache_fork(k, v, table, lens, ref, i32([0]), i32([0]), extra=30, dev_error=c.err)
    assert int(c.err) == 0 and (table[0, :5] >= 0).all() and int(ref.sum()) == int((table >= 0).sum())


def test_shared_and_missing_pages_leave_a_request_alone(M):
    for fault in ("shared", "missing", "outside", "long", "negative"):
        c = Evict([100, 100], 40, 2, 8, page=16, cap=112)
        c.table[0, 7:] = -1
        k, v, w, lens, table, ref = (x.clone() for x in (c.k, c.v, c.w, c.kv_len, c.table, c.ref))
        if fault == "shared":
            ref[table[0, 1].long()] = 2
        elif fault == "missing":
            table[0, 5] = -1
        elif fault == "outside":
            table[0, 6] = 10 ** 6
        else:
            lens[0] = 10 ** 6 if fault == "long" else -1
        was = lens[0].item(), table[0].clone()
        err = i32([0])
        M.masked_gqa_cache_evict(k, v, w, lens, budget=40, sinks=2, recent=8, page_table=table, ref=ref, dev_error=err)
        assert int(err) == INVALID and lens.tolist() == [was[0], 40], fault
        assert torch.equal(table[0], was[1]) and torch.equal(w[0, 0], c.w[0, 0])
        mine = c.table[0][c.table[0] >= 0].long()
        assert torch.equal(k[:, mine], c.k[:, mine]) and torch.equal(v[:, mine], c.v[:, mine])
        keep = c.want(0, 1, 0)
        (pa, sa), (pb, sb) = c.place(c.table, 1, keep), c.place(c.table, 1, range(40))
        assert torch.equal(k[0, pb, 0, sb], c.k[0, pa, 0, sa])


def test_a_page_shared_behind_the_budget_is_read_only(M):
    """Pages that are only read may be shared; they are given back once."""
    c = Evict([100, 20], 40, 2, 8, page=16, cap=112)
    c.ref[c.table[0, 5].long()] = 2
    c.run(M, with_ref=True)


def test_on_another_stream_with_its_own_memory(M):
    c = Evict([500, 90], 128, 4, 32, layers=2, page=16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.run(M)
    torch.cuda.synchronize()
    k, v, w, lens = (x.clone() for x in (c.k, c.v, c.w, c.kv_len))
    torch.cuda.synchronize()
    M.masked_gqa_cache_evict(k, v, w, lens, budget=128, sinks=4, recent=32, page_table=c.table, stream=s)
    s.synchronize()
    assert lens.tolist() == [128, 90]
    for g in range(2):
        keep = c.want(1, 0, g)
        (pa, sa), (pb, sb) = c.place(c.table, 0, keep), c.place(c.table, 0, range(128))
        assert torch.equal(k[1, pb, g, sb], c.k[1, pa, g, sa]) and torch.equal(w[1, 0, g, :128], c.w[1, 0, g, keep])


def test_a_budget_past_every_length(M):
    Evict([50, 3], 1 << 20, 4, 32, page=16).run(M)
    Evict([50, 3], 1 << 24, 0, 1 << 24).run(M, in_place=False)


def test_weights_shorter_than_the_table(M):
    """Slots that have no weight: a longer request is left alone; shorter ones are cut."""
    c = Evict([100, 100], 40, 2, 8, page=16, cap=160)
    w = c.w[..., :100].contiguous()
    k, v, lens, err = c.k.clone(), c.v.clone(), i32([100, 101]), i32([0])
    M.masked_gqa_cache_evict(k, v, w, lens, budget=40, sinks=2, recent=8, page_table=c.table, dev_error=err)
    assert lens.tolist() == [40, 101] and int(err) == INVALID and torch.equal(w[0, 1], c.w[0, 1, :, :100])
    keep = c.want(0, 0, 1)
    (pa, sa), (pb, sb) = c.place(c.table, 0, keep), c.place(c.table, 0, range(40))
    assert torch.equal(k[0, pb, 1, sb], c.k[0, pa, 1, sa])


def test_weights_and_eviction_captured(M):
    c = Evict([500, 200, 90], 128, 4, 32, layers=2, page=16, cap=512)
    k, v, w, lens = (x.clone() for x in (c.k, c.v, c.w, c.kv_len))
    ws = torch.empty(M.masked_gqa_cache_evict_workspace_size(k, v, 128, page_table=c.table), dtype=torch.uint8, device="cuda")
    kw = dict(budget=128, sinks=4, recent=32, page_table=c.table, workspace=ws)
    M.masked_gqa_cache_evict(k, v, w, lens, **kw)
    torch.cuda.synchronize()
    want = [x.clone() for x in (k, v, w, lens)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.masked_gqa_cache_evict(k, v, w, lens, **kw)
    for _ in range(3):
        for x, y in zip((k, v, w, lens), (c.k, c.v, c.w, c.kv_len)):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip((k, v, w, lens), want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("q4", [False, True])
def test_a_serving_loop(M, q4):
    """Prompt, weights of its last tokens, eviction, then steps that append, attend, sum up and evict again,
    all queued without a look at the results; against the same loop in 64 bits."""
    B, Hq, Hkv, D, page, cap, budget, T, steps = 2, 8, 2, 64, 16, 160, 48, 8, 6
    n0 = [130, 70]
    mp = cap // page
    table = torch.randperm(B * mp).int().view(B, mp).cuda()
    ref = torch.ones(B * mp, dtype=torch.int32, device="cuda")
    row, kind = (D // 2 + 16, torch.uint8) if q4 else (D, BF)
    k, v = (torch.zeros(B * mp, Hkv, page, row, dtype=kind, device="cuda") for _ in range(2))
    append = M.masked_gqa_cache_append_q4 if q4 else M.masked_gqa_cache_append
    prompt = [rand((B, Hkv, max(n0), D), BF, 1 + x) for x in range(2)]
    new = [rand((steps, B, Hkv, 1, D), BF, 3 + x) for x in range(2)]
    q0, qs = 2 * rand((B, Hq, T, D), BF, 5), 2 * rand((steps, B, Hq, 1, D), BF, 6)
    lens, nxt = i32([0] * B), i32([0] * B)
    weight = torch.zeros(B, Hkv, cap, device="cuda")
    ws = M.new_cache_attn_workspace()

    def attend(q, n):
        lse = torch.empty(q.shape[:3], device="cuda")
        if q4:
            out = M.masked_gqa_attn_decode_q4(q, k, v, n, page_table=table, workspace=ws, lse=lse)
        else:
            out = torch.empty_like(q)
            for t in range(q.shape[2]):  # one query at a time, each the last of its own length
                one = torch.empty(B, Hq, 1, device="cuda")
                out[:, :, t:t + 1] = M.masked_gqa_attn_decode_window(
                    q[:, :, t:t + 1].contiguous(), k, v, n - (q.shape[2] - 1 - t), window=1 << 20, page_table=table,
                    workspace=ws, lse=one)
                lse[:, :, t:t + 1] = one
        M.masked_gqa_attn_cache_weights(q, k, n, lse, weight, page_table=table)
        return out

    err, rows = i32([0]), i32([0, 1])

    def trim():  # the pages behind the budget go back, and those for the next steps are taken
        M.masked_gqa_cache_evict(k, v, weight, nxt, budget=budget, sinks=2, recent=8, page_table=table, ref=ref,
                                 dev_error=err)
        M.masked_gqa_cache_fork(k, v, table, nxt, ref, rows, rows, extra=steps, dev_error=err)

    append(k, v, *prompt, lens, nxt, count=i32(n0), page_table=table, dev_error=err)
    outs = [attend(q0, nxt)]
    trim()
    for t in range(steps):
        lens, nxt = nxt, lens
        append(k, v, new[0][t], new[1][t], lens, nxt, page_table=table, dev_error=err)
        outs.append(attend(qs[t], nxt))
        if t % 3 == 2:
            trim()
    torch.cuda.synchronize()
    assert int(err) == 0

    held = (lambda x: values(records(x))[0]) if q4 else (lambda x: x.double())
    for b in range(B):
        kk, vv = (held(p[b, :, :n0[b]]) for p in prompt)
        w = torch.zeros(Hkv, n0[b], dtype=torch.float64, device="cuda")

        def step(q, kk, vv, w):
            n = kk.shape[1]
            s, _ = scores(q, kk, kk.abs(), sees(n, q.shape[1], 0, 0, "cuda"), D ** -0.5)
            p = torch.softmax(s, -1)
            return p @ vv.repeat_interleave(Hq // Hkv, 0), w + p.reshape(Hkv, -1, n).sum(1)

        def cut(kk, vv, w):
            if kk.shape[1] <= budget:
                return kk, vv, w
            keep = torch.tensor([kept_slots(w[g].cpu(), kk.shape[1], budget, 2, 8) for g in range(Hkv)], device="cuda")
            pick = lambda x: torch.gather(x, 1, keep[..., None].expand(-1, -1, D))  # noqa: E731
            return pick(kk), pick(vv), torch.gather(w, 1, keep)

        # (outputs of order 1: 2^-8 for their rounding and the weights', 2^-7 with the sums)
        want, w = step(q0[b], kk, vv, w)
        assert (outs[0][b].double() - want).abs().max() < 2.0 ** -6
        kk, vv, w = cut(kk, vv, w)
        for t in range(steps):
            kk, vv = (torch.cat([x, held(y[t, b])], 1) for x, y in ((kk, new[0]), (vv, new[1])))
            w = torch.cat([w, torch.zeros(Hkv, 1, dtype=torch.float64, device="cuda")], 1)
            want, w = step(qs[t, b], kk, vv, w)
            assert (outs[1 + t][b].double() - want).abs().max() < 2.0 ** -6, (b, t)
            if t % 3 == 2:
                kk, vv, w = cut(kk, vv, w)
        n = kk.shape[1]
        assert int(nxt[b]) == n
        assert (weight[b, :, :n].double() - w).abs().max() < 1e-4
