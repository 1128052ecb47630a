"""Calls on a stream that is not the current one: what they allocate may not be
memory that work queued on the current stream still uses."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
DELAY = 40_000_000  # cycles: some 20 ms, in which the call on the other stream runs


@pytest.fixture(scope="module")
def M():
    import masked_gqa_attention_gb300 as M
    M.build_library()
    return M


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(*shape):
    return torch.randn(shape, device="cuda").to(BF)


def tree_call(M, seed):
    """A call whose units are cut (partial results in the workspace), as a function of its keywords."""
    torch.manual_seed(seed)
    pages = 1300
    q, k, v = randn(1, 8, 8, 128), randn(pages, 2, 16, 128), randn(pages, 2, 16, 128)
    kn, vn = randn(1, 2, 8, 128), randn(1, 2, 8, 128)
    table = torch.full((1, 12500), -1, dtype=torch.int32, device="cuda")
    table[0, :1260] = torch.randperm(pages, device="cuda")[:1260].int()
    lens = i32([20011])
    return lambda **kw: M.masked_gqa_attn_decode_tree(q, k, v, kn, vn, lens, page_table=table, **kw)


def pool(M, rows=40, page=16, mp=30):
    """A pool whose requests fork; returns (arguments, workspace bytes of a fork and of a compaction)."""
    torch.manual_seed(3)
    pages = rows * mp
    k, v = randn(2, pages, 2, page, 64), randn(2, pages, 2, page, 64)
    table = torch.randperm(pages, device="cuda").int().view(rows, mp)
    lens = i32([(mp - 3) * page + r % page for r in range(rows)])
    table[:, mp - 2:] = -1
    ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
    ref[table[table >= 0].long()] = 1
    n = rows // 2
    sizes = [M.masked_gqa_cache_workspace_size(k, v, table, ref, x) for x in (n, 0)]
    return [k, v, table, lens, ref, i32(list(range(n))), i32(list(range(n, rows)))], sizes


def sum_in_flight(size):
    """A freed tensor of `size` bytes whose sum is still queued on the current stream; returns the sum."""
    x = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(DELAY)
    total = x.sum(dtype=torch.int64)
    return total  # (x goes: the allocator may hand its block out to this stream at once)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("op", ["tree", "fork", "compact"])
def test_own_workspace_spares_memory_in_use(M, op, handle):
    s = torch.cuda.Stream()
    on = s.cuda_stream if handle else s
    if op == "tree":
        call, size = tree_call(M, 1), M.masked_gqa_attn_cache_workspace_size()
        want = call().clone()
        out = torch.empty_like(want)
        total = sum_in_flight(size)
        call(out=out, stream=on)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    else:
        (k, v, table, lens, ref, src, dst), sizes = pool(M)
        k1, v1, table1, lens1, ref1 = (x.clone() for x in (k, v, table, lens, ref))

        def step(stream, k, v, table, lens, ref):
            if op == "fork":
                M.masked_gqa_cache_fork(k, v, table, lens, ref, src, dst, extra=5, stream=stream)
            else:
                M.masked_gqa_cache_compact(k, v, table, ref, stream=stream)

        step(None, k1, v1, table1, lens1, ref1)
        size = sizes[0 if op == "fork" else 1]
        total = sum_in_flight(size)
        step(on, k, v, table, lens, ref)
        torch.cuda.synchronize()
        for a, b in ((k, k1), (v, v1), (table, table1), (lens, lens1), (ref, ref1)):
            assert torch.equal(a, b)
    assert int(total) == 7 * size


def test_own_workspaces_of_two_streams_are_apart(M):
    # one call is queued on the current stream, its workspace freed again; the other runs meanwhile
    a, b = tree_call(M, 1), tree_call(M, 2)
    wa, wb = a().clone(), b().clone()
    oa, ob = torch.empty_like(wa), torch.empty_like(wb)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        torch.cuda._sleep(200_000)
        a(out=oa)
        b(out=ob, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)
