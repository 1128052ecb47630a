"""The cache's steps at the ends of their ranges."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def M():
    import masked_gqa_attention_gb300 as M
    M.build_library()
    return M


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_fork_requests_that_add_up_past_32_bits(M):
    # 139 pairs ask for 2^24 - 1 pages each: together more than 2^31, of which none is served
    rows, mp, pages = 141, 1 << 24, 64
    k = torch.arange(pages * 8, device="cuda").to(BF).view(1, pages, 1, 1, 8)
    v = -k
    k1, v1 = k.clone(), v.clone()
    table = torch.full((rows, mp), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[140, 0] = 5, 6
    lens, ref, err = i32([1] + [0] * 139 + [1]), torch.zeros(pages, dtype=torch.int32, device="cuda"), i32([0])
    ref[5], ref[6] = 1, 1
    M.masked_gqa_cache_fork(k, v, table, lens, ref, i32([0] * 139 + [-1]), i32(list(range(1, 141))), extra=mp - 1,
                            dev_error=err)
    assert int(err) == M.MGQA_ERR_INVALID_ARG
    assert lens.tolist() == [1] + [0] * 140  # the last pair frees its request
    assert ref.nonzero().flatten().tolist() == [5] and int(ref[5]) == 1
    assert int(table[0, 0]) == 5 and int((table != -1).sum()) == 1
    assert torch.equal(k, k1) and torch.equal(v, v1)


@pytest.mark.parametrize("paged", [False, True])
def test_counts_and_tables_beside_the_lengths(M, paged):
    # the step's small integers in one buffer, so in one line of 128 bytes: each step reads what the one before wrote
    B, cap, D, steps = 4, 700, 64, 300
    k = torch.zeros(B, 1, cap, D, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    new = torch.randn(steps, B, 1, 1, D, device="cuda").to(BF)
    ints = torch.zeros(32, dtype=torch.int32, device="cuda")
    lens, count, index, table = ints[:8].view(2, B), ints[8:12], ints[12:16].view(B, 1), None
    count.fill_(1)
    if paged:
        table = ints[16:20].view(B, 1)
        table.copy_(torch.tensor([[2], [0], [3], [1]], dtype=torch.int32))
    q, ws = torch.randn(B, 1, 1, D, device="cuda").to(BF), M.new_cache_attn_workspace()
    outs = torch.empty(steps, B, 1, 1, D, dtype=BF, device="cuda")
    for i in range(steps):
        old, now = lens[i % 2], lens[1 - i % 2]
        M.masked_gqa_cache_append(k, v, new[i], new[i], old, now, index=index, count=count, page_table=table)
        M.masked_gqa_attn_decode_window(q, k, v, now, outs[i], window=1, page_table=table, workspace=ws)
    assert lens.tolist() == [[steps] * B, [steps - 1] * B]
    assert torch.equal(outs, new)  # a window of one: the token just appended


def test_the_largest_pool_is_packed_in_order(M):
    # 2^20 pages: which page moves where is fixed, for the tables, the counts and the contents
    n = 1 << 20
    mark = (torch.arange(n, device="cuda") % 127).to(BF)
    k = torch.zeros(1, n, 1, 1, 8, dtype=BF, device="cuda")
    k[0, :, 0, 0, 0] = mark
    v = k * 2
    used = [5, n - 1 - 1000, n - 3, n - 2, n - 1]  # five pages: 5 stays behind the holes 0 .. 4 and moves, as the others do
    ref = torch.zeros(n, dtype=torch.int32, device="cuda")
    ref[torch.tensor(used, device="cuda")] = i32([3, 1, 4, 1, 5])
    table, n_used, err = i32([[n - 1, 5, n - 3, -1], [n - 2, n - 1001, 5, n - 1]]), i32([-1]), i32([0])
    M.masked_gqa_cache_compact(k, v, table, ref, used_out=n_used, dev_error=err)
    assert table.tolist() == [[4, 0, 2, -1], [3, 1, 0, 4]] and int(n_used) == 5 and int(err) == 0
    assert ref[:5].tolist() == [3, 1, 4, 1, 5] and int(ref.sum()) == 14
    want = mark.clone()
    want[:5] = mark[torch.tensor(used, device="cuda")]
    assert torch.equal(k[0, :, 0, 0, 0], want) and torch.equal(v[0, :, 0, 0, 0], 2 * want)
    assert not k[..., 1:].any() and not v[..., 1:].any()


def test_the_largest_pool_is_forked_in_order(M):
    # the fresh pages are the lowest free ones in the order of the pairs, over the whole pool
    n = 1 << 20
    k = torch.zeros(1, n, 1, 2, 8, dtype=BF, device="cuda")
    k[0, :, 0, :, 0] = (torch.arange(n, device="cuda") % 127).to(BF)[:, None]
    v = k * 2
    ref = torch.ones(n, dtype=torch.int32, device="cuda")
    free = [7, 32767, 500000, n - 1]
    ref[torch.tensor(free, device="cuda")] = 0
    table = i32([[n - 2, n - 5, -1], [-1] * 3, [-1] * 3, [n - 3, -1, -1]])
    lens, err = i32([3, 0, 0, 2]), i32([0])
    M.masked_gqa_cache_fork(k, v, table, lens, ref, i32([0, 3, 0]), i32([1, 2, 3]), extra=1, dev_error=err)
    # request 1: a shared page and a copy of the half one; request 2: a shared page and a new one; request 3 as 1
    assert table.tolist() == [[n - 2, n - 5, -1], [n - 2, 7, -1], [n - 3, 32767, -1], [n - 2, 500000, -1]]
    assert lens.tolist() == [3, 3, 2, 3] and int(err) == 0
    assert ref[torch.tensor([n - 2, n - 5, n - 3, *free], device="cuda")].tolist() == [3, 1, 1, 1, 1, 1, 0]
    for x, f in ((k, 1), (v, 2)):
        for page, src in ((7, n - 5), (500000, n - 5)):
            assert x[0, page, 0, 0, 0] == f * (src % 127) and x[0, page, 0, 1, 0] == f * (page % 127)
        assert x[0, 32767, 0, :, 0].tolist() == [f * (32767 % 127)] * 2
