"""Appending, forking, freeing and packing a cache against a sequential model:
everything is moved as it is, so every comparison is exact."""
import random

import pytest
import torch

from _cache_ref import compact_model, fork_model

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def M():
    import masked_gqa_attention_gb300 as M
    M.build_library()
    return M


def pools(shape, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(2)]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_table(rng, lens, page, mp, spare):
    need = [-(-n // page) for n in lens]
    order = list(range(sum(need) + spare))
    rng.shuffle(order)
    table, at = [], 0
    for m in need:
        table.append(order[at:at + m] + [-1] * (mp - m))
        at += m
    ref = [0] * len(order)
    for row in table:
        for e in row:
            if e >= 0:
                ref[e] += 1
    return table, ref


# ---- append -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("layers,Hkv,D,T,page", [(1, 1, 8, 1, 0), (3, 2, 64, 5, 16), (1, 8, 128, 300, 24), (2, 3, 128, 17, 1),
                                                 (2, 2, 64, 33, 0)])
def test_append(M, dtype, layers, Hkv, D, T, page):
    rng = random.Random(T)
    lens = [0, 7, 31, 100]
    B, cap = 4, 100 + T
    if page:
        table, _ = make_table(rng, [n + T for n in lens], page, -(-cap // page) + 1, 2)
        shape = (layers, sum(-(-(n + T) // page) for n in lens) + 2, Hkv, page, D)
    else:
        table, shape = None, (layers, B, Hkv, cap, D)
    k, v = pools(shape, dtype, 1)
    kn, vn = (x.transpose(2, 3) for x in pools((layers, B, T, Hkv, D), dtype, 2))
    for chosen in (False, True):
        index = [[rng.randrange(T) for _ in range(T)] for _ in range(B)] if chosen else None  # repeats among them
        count = [0, 1, T // 2, T] if chosen else None
        k1, v1 = k.clone(), v.clone()
        for b, n in enumerate(lens):
            for i in range(count[b] if chosen else T):
                f = index[b][i] if chosen else i
                p, s = (table[b][(n + i) // page], (n + i) % page) if page else (b, n + i)
                k1[:, p, :, s], v1[:, p, :, s] = kn[:, b, :, f], vn[:, b, :, f]
        out, err = i32([9] * B), i32([0])
        kk, vv = k.clone(), v.clone()
        M.masked_gqa_cache_append(kk, vv, kn, vn, i32(lens), out, index=None if index is None else i32(index),
                                  count=None if count is None else i32(count),
                                  page_table=None if table is None else i32(table), dev_error=err)
        assert torch.equal(kk, k1) and torch.equal(vv, v1) and int(err) == 0
        assert out.tolist() == [n + (count[b] if chosen else T) for b, n in enumerate(lens)]


def test_append_4d_and_refused_rows(M):
    # one layer without the layer dimension; a full request, a bad count, a bad index and a missing page
    lens, page, T = [14, 0, 30, 0, 5], 16, 4
    table = [[0, 1], [2, 3], [4, 5], [-1, 6], [7, 8]]
    k, v = pools((9, 2, page, 64), BF, 3)
    kn, vn = pools((5, 2, T, 64), BF, 4)
    count = [4, 5, 4, 2, 3]
    index = [[0, 1, 2, 3]] * 4 + [[2, -1, 1, 0]]
    k1, v1, out, err = k.clone(), v.clone(), i32([0] * 5), i32([0])
    M.masked_gqa_cache_append(k, v, kn, vn, i32(lens), out, index=i32(index), count=i32(count), page_table=i32(table),
                              dev_error=err)
    for b, i, f in [(0, 0, 0), (0, 1, 1), (0, 2, 2), (0, 3, 3), (4, 0, 2), (4, 2, 1)]:
        p, s = table[b][(lens[b] + i) // page], (lens[b] + i) % page
        k1[p, :, s], v1[p, :, s] = kn[b, :, f], vn[b, :, f]
    assert torch.equal(k, k1) and torch.equal(v, v1)
    assert int(err) == M.MGQA_ERR_INVALID_ARG and out.tolist() == [18, 0, 30, 2, 8]


# ---- fork ---------------------------------------------------------------------

def run_fork(M, table, lens, ref, src, dst, extra, page, layers=2, Hkv=2, D=64, dtype=BF, slot_major=False, **kw):
    npages = len(ref)
    if slot_major:  # [layers, pages, page, Hkv, D] storage
        k, v = (x.transpose(2, 3) for x in pools((layers, npages, page, Hkv, D), dtype, 5))
    else:
        k, v = pools((layers, npages, Hkv, page, D), dtype, 5)
    t, n, r, err = i32(table), i32(lens), i32(ref), i32([0])
    k1, v1 = k.clone(), v.clone()
    M.masked_gqa_cache_fork(k, v, t, n, r, i32(src), i32(dst), extra=extra, dev_error=err, **kw)
    table, lens, ref = [list(x) for x in table], list(lens), list(ref)
    copies, bad = fork_model(table, lens, ref, src, dst, extra, page)
    for a, b, s in copies:
        k1[:, b, :, :s], v1[:, b, :, :s] = k1[:, a, :, :s], v1[:, a, :, :s]
    assert t.tolist() == table and n.tolist() == lens and r.tolist() == ref
    assert torch.equal(k, k1) and torch.equal(v, v1)
    assert int(err) == (M.MGQA_ERR_INVALID_ARG if bad else 0)
    return table, lens, ref


@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("seed", range(4))
def test_fork_random_sequences(M, page, seed):
    rng = random.Random(seed * 100 + page)
    rows, cap = 24, 150
    mp = -(-cap // page) + 2
    lens = [rng.randint(0, cap) for _ in range(rows)]
    table, ref = make_table(rng, lens, page, mp, 4 * rows + 200 // page)
    for step in range(6):  # the state goes from call to call
        n = rng.randint(1, rows)
        dst = rng.sample(range(rows), n)
        src = [rng.choice([-1, d, rng.randrange(rows)]) for d in dst]  # sources that are destinations too
        table, lens, ref = run_fork(M, table, lens, ref, src, dst, rng.choice([0, 1, page, 2 * page + 1]), page,
                                    slot_major=step % 2 == 1, dtype=[BF, FP, HF][step % 3])
        held = [0] * len(ref)
        for row in table:
            for e in row:
                if e >= 0:
                    held[e] += 1
        assert held == ref


def test_fork_swap_reorder_and_free(M):
    table, ref = make_table(random.Random(1), [20, 40, 17, 16], 16, 4, 12)
    run_fork(M, table, [20, 40, 17, 16], ref, [1, 0], [0, 1], 0, 16)  # two rows change places
    run_fork(M, table, [20, 40, 17, 16], ref, [3, 3, 3], [0, 1, 2], 8, 16)  # full pages only, and one to write
    run_fork(M, table, [20, 40, 17, 16], ref, [-1, -1, -1, -1], [0, 1, 2, 3], 8, 16)


def test_fork_own_page_before_writing(M):
    # rows 0 and 1 share a partly filled page (as after a rollback): each reserving row gets its own
    table = [[0, 1, -1], [0, 1, 2], [3, -1, -1]]
    ref = [2, 2, 1, 1, 0, 0, 0, 0]
    run_fork(M, table, [20, 20, 3], ref, [0], [0], 1, 16)
    run_fork(M, table, [20, 20, 3], ref, [0, 1], [0, 1], 1, 16)
    run_fork(M, table, [20, 20, 3], ref, [2, 1], [2, 1], 20, 16)


def test_fork_without_enough_pages(M):
    table = [[0, 1, 2, -1], [3, -1, -1, -1], [4, -1, -1, -1], [-1] * 4]
    ref = [1, 1, 1, 1, 1, 0]
    run_fork(M, table, [40, 3, 7, 0], ref, [0, 1], [3, 2], 0, 16)  # one page is free, two are wanted (row 2's counts)
    run_fork(M, table, [40, 3, 7, 0], ref, [0, 1], [3, 1], 30, 16)  # the first asks for two: nothing for either
    run_fork(M, table, [40, 3, 7, 0], ref, [0], [0], 100, 16)  # past the row
    run_fork(M, table, [40, 3, 7, 0], ref, [1, -1], [1, 0], 20, 16)


def test_fork_bad_pairs_are_skipped(M):
    table, ref = make_table(random.Random(2), [20, 40, 17], 16, 4, 12)
    run_fork(M, table, [20, 40, 17], ref, [0, 5, -2, 1, 2], [1, 0, 2, 1, 7], 0, 16)
    table[0][1] = 10 ** 6  # an entry that is no page
    run_fork(M, table, [16, 40, 17], ref, [0], [2], 0, 16)


def test_fork_many_pages_and_pairs(M):
    rng = random.Random(7)
    rows, page = 1000, 16
    lens = [rng.randint(0, 400) for _ in range(rows)]
    table, ref = make_table(rng, lens, page, 40, 70000 - sum(-(-n // page) for n in lens))
    dst = rng.sample(range(rows), 900)
    run_fork(M, table, lens, ref, [rng.randrange(-1, rows) for _ in dst], dst, 100, page, layers=1, Hkv=1, D=8)


# ---- compact --------------------------------------------------------------------

@pytest.mark.parametrize("npages", [1, 2, 31, 33, 1000, 40000])
@pytest.mark.parametrize("share", [0.0, 0.03, 0.5, 0.97, 1.0])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact(M, npages, share, in_place):
    rng = random.Random(npages)
    held = rng.sample(range(npages), round(share * npages))
    rows = 5
    mp = -(-len(held) // rows) + 1
    table = [[-1] * mp for _ in range(rows)]
    for i, p in enumerate(held):
        table[i % rows][i // rows] = p
    if held:
        table[rows - 1] = list(table[0])
    ref = [0] * npages
    for row in table:
        for e in row:
            if e >= 0:
                ref[e] += 1
    page, Hkv, layers, D, dtype = rng.choice([(4, 2, 2, 64, BF), (1, 1, 3, 8, HF), (16, 2, 1, 128, FP)])
    if npages > 10000:
        page, Hkv, layers, D = 1, 1, 1, 8
    k, v = pools((layers, npages, Hkv, page, D), dtype, 6)
    t, r, used, err = i32(table), i32(ref), i32([-1]), i32([0])
    k1, v1 = k.clone(), v.clone()
    to_t, to_r = (t, r) if in_place else (torch.zeros_like(t), torch.zeros_like(r))
    got = M.masked_gqa_cache_compact(k, v, t, r, *(() if in_place else (to_t, to_r)), used_out=used, dev_error=err)
    table1, ref1, to, n = compact_model(table, ref)
    for a, b in to.items() if npages <= 1000 else ():
        k1[:, b], v1[:, b] = k1[:, a], v1[:, a]
    if npages > 1000 and to:
        a, b = torch.tensor(list(to)).cuda(), torch.tensor(list(to.values())).cuda()
        k1[:, b], v1[:, b] = k1[:, a], v1[:, a]
    assert got[0] is to_t and got[1] is to_r
    assert to_t.tolist() == table1 and to_r.tolist() == ref1 and int(used) == n and int(err) == 0
    assert torch.equal(k, k1) and torch.equal(v, v1)
    if not in_place:
        assert t.tolist() == table and r.tolist() == ref


def test_compact_large_offsets(M):
    # a pool past 2^31 elements
    npages, page, Hkv, D = 70000, 32, 8, 128
    k = torch.zeros(1, npages, Hkv, page, D, dtype=BF, device="cuda")
    k[0, :, 0, 0, 0] = (torch.arange(npages, device="cuda") % 251).to(BF)
    k[0, :, -1, -1, -1] = (torch.arange(npages, device="cuda") % 241).to(BF)
    v = k.clone()
    ref = torch.zeros(npages, dtype=torch.int32, device="cuda")
    ref[5], ref[npages - 1] = 1, 2
    table = i32([[5, npages - 1], [npages - 1, -1]])
    M.masked_gqa_cache_compact(k, v, table, ref)
    # two pages in use: pages 0 and 1 are free and take them
    assert table.tolist() == [[0, 1], [1, -1]] and ref[:2].tolist() == [1, 2] and int(ref.sum()) == 3
    for x in (k, v):
        assert x[0, 0, 0, 0, 0] == 5 and x[0, 1, 0, 0, 0] == (npages - 1) % 251
        assert x[0, 1, -1, -1, -1] == (npages - 1) % 241


def test_the_largest_pool(M):
    # 2^20 pages, the most that are planned: fork's free pages and compact's moves at both ends
    n = 1 << 20
    k = torch.zeros(1, n, 1, 1, 8, dtype=BF, device="cuda")
    k[0, :, 0, 0, 0] = (torch.arange(n, device="cuda") % 127).to(BF)
    v = k.clone()
    ref = torch.ones(n, dtype=torch.int32, device="cuda")
    ref[[7, n - 1]] = 0
    table, lens = i32([[n - 2, n - 3, -1], [-1, -1, -1]]), i32([2, 0])
    M.masked_gqa_cache_fork(k, v, table, lens, ref, i32([0, 0]), i32([0, 1]), extra=1)
    assert table.tolist() == [[n - 2, n - 3, 7], [n - 2, n - 3, n - 1]] and lens.tolist() == [2, 2]
    assert ref[[7, n - 1, n - 2]].tolist() == [1, 1, 2]
    ref.zero_()
    ref[table[0].long()], ref[n - 1] = 1, 1
    M.masked_gqa_cache_compact(k, v, table, ref)
    assert table.tolist() == [[2, 1, 0], [2, 1, 3]] or sorted(table.flatten().tolist()) == [0, 1, 1, 2, 2, 3]
    assert int(ref[:4].sum()) == 4 and int(ref.sum()) == 4


def test_lengths_side_by_side(M):
    # old and new lengths in the same 32 bytes, each step reading what the one before wrote
    B, cap, D, steps = 4, 700, 64, 300
    k = torch.zeros(B, 1, cap, D, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    new = torch.randn(steps, B, 1, 1, D, device="cuda").to(BF)
    lens = torch.zeros(2, B, dtype=torch.int32, device="cuda")
    q, ws = torch.randn(B, 1, 1, D, device="cuda").to(BF), M.new_cache_attn_workspace()
    outs = torch.empty(steps, B, 1, 1, D, dtype=BF, device="cuda")
    for i in range(steps):
        M.masked_gqa_cache_append(k, v, new[i], new[i], lens[i % 2], lens[1 - i % 2])
        M.masked_gqa_attn_decode_window(q, k, v, lens[1 - i % 2], outs[i], window=1, workspace=ws)
    assert lens.tolist() == [[steps] * B, [steps - 1] * B]
    assert torch.equal(outs, new)  # a window of one: the token just appended


# ---- together -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, FP])
def test_a_serving_loop(M, dtype):
    """Prompts, forks, speculative steps with acceptance, a finished request and
    a packed pool; the paged results against a plain copy of every sequence."""
    from _cache_ref import attention, check, see_words
    rng = random.Random(3)
    layers, Hq, Hkv, D, page, rows, mp, npages, W, S = 2, 4, 2, 64, 16, 6, 12, 80, 70, 4
    k, v = pools((layers, npages, Hkv, page, D), dtype, 1)
    table, kv_len, ref, err = i32([[-1] * mp] * rows), i32([0] * rows), i32([0] * npages), i32([0])
    ws = M.new_cache_attn_workspace()
    plain = [[torch.zeros(layers, Hkv, 0, D, dtype=dtype, device="cuda") for _ in range(2)] for _ in range(rows)]

    def new(T, seed):
        return pools((layers, rows, Hkv, T, D), dtype, seed)

    def append(kn, vn, index, count):
        out = torch.empty_like(kv_len)
        M.masked_gqa_cache_append(k, v, kn, vn, kv_len, out, index=i32(index), count=i32(count), page_table=table,
                                  dev_error=err)
        kv_len.copy_(out)
        for b in range(rows):
            for c, x in enumerate((kn, vn)):
                plain[b][c] = torch.cat([plain[b][c], x[:, b, :, index[b][:count[b]]]], 2)

    def fork(src, dst, extra):
        M.masked_gqa_cache_fork(k, v, table, kv_len, ref, i32(src), i32(dst), extra=extra, dev_error=err)
        old = [list(x) for x in plain]
        for s, d in zip(src, dst):
            plain[d] = list(old[s]) if s >= 0 else [x[:, :, :0] for x in old[d]]

    lens = [40, 33, 0, 16, 1, 0]
    fork(range(rows), range(rows), 48)  # room for the prompts
    append(*new(40, 2), [list(range(40))] * rows, lens)
    for step in range(5):
        if step == 1:
            fork([0, 0, 1], [2, 5, 4], 0)  # samples of request 0, and request 1 in the place of 4
        if step == 3:
            fork([-1], [3], 0)
            M.masked_gqa_cache_compact(k, v, table, ref, dev_error=err)
            assert table.max() + 1 == (ref > 0).sum()
        T = [1, 7, 12, 3, 20][step]
        fork(range(rows), range(rows), T)  # every row owns what this step may write
        kn, vn = new(T, 50 + step)
        seen = torch.zeros(rows, T, T, dtype=torch.bool)
        for b in range(rows):
            for t in range(T):
                parent = rng.randint(max(-1, t - 4), t - 1)
                if parent >= 0:
                    seen[b, t] = seen[b, parent]
                seen[b, t, t] = True
        for layer in range(layers):
            q = pools((rows, Hq, T, D), dtype, 90 + step + 7 * layer)[0]
            for window in (0, W):
                out = M.masked_gqa_attn_decode_tree(q, k[layer], v[layer], kn[layer], vn[layer], kv_len,
                                                    tree_bits=see_words(seen).cuda(), window=window, sinks=S,
                                                    page_table=table, workspace=ws, dev_error=err)
                for b in range(rows):
                    kb, vb = (torch.cat([plain[b][c][layer], x[layer, b]], 1) for c, x in enumerate((kn, vn)))
                    n = kb.shape[1] - T
                    s = seen[b].cuda()
                    pos = n + s.sum(1) - 1
                    see, j = torch.ones(T, n, dtype=torch.bool, device="cuda"), torch.arange(n, device="cuda")
                    if window:
                        see = (pos[:, None] - j < W) | (j < S)
                        s = s & ((pos[:, None] - pos < W) | (pos < S))
                    check(out[b], None, attention(q[b], kb, vb, torch.cat([see, s], 1), D ** -0.5), n + T)
        # accept the path to one draft of each tree
        index, count = [], []
        for b in range(rows):
            path = [i for i, x in enumerate(seen[b, rng.randrange(T)].tolist()) if x]
            index.append(path + [0] * (T - len(path)))
            count.append(len(path))
        append(kn, vn, index, count)
        q1 = pools((rows, Hq, 1, D), dtype, 300 + step)[0]
        out = M.masked_gqa_attn_decode_window(q1, k[0], v[0], kv_len, window=W, sinks=S, page_table=table, workspace=ws,
                                              dev_error=err)
        for b in range(rows):
            kb, vb = (plain[b][c][0] for c in range(2))
            j = torch.arange(kb.shape[1], device="cuda")
            vis = ((kb.shape[1] - 1 - j < W) | (j < S))[None]
            check(out[b], None, attention(q1[b], kb, vb, vis, D ** -0.5), kb.shape[1])
        assert kv_len.tolist() == [plain[b][0].shape[2] for b in range(rows)]
    assert int(err) == 0
