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


def outputs():
    """Calls that allocate their output, by name: a function of the module that gives (a call of a stream, the shape
    of its output)."""
    def attn(Lq, Lk=256):
        return randn(2, 4, Lq, 64), randn(2, 2, Lk, 64), randn(2, 2, Lk, 64)

    def plain(name, Lq, **kw):
        def make(M):
            q, k, v = attn(Lq)
            more = {x: y() for x, y in kw.items()}
            return lambda s: getattr(M, name)(q, k, v, stream=s, **more)
        return make

    def append(M):
        q, k, v = attn(1)
        new, lens = randn(2, 2, 1, 64), i32([100, 7])
        return lambda s: M.masked_gqa_attn_decode_append(q, k, v, new, new, lens, stream=s)

    def append_rope(M):
        q, k, v = attn(1)
        new, lens, f = randn(2, 2, 1, 64), i32([100, 7]), torch.rand(32, device="cuda")
        return lambda s: M.masked_gqa_attn_decode_append_rope(q, k, v, new, new, lens, inv_freq=f, stream=s)

    def window(M):
        q, k, v = attn(1)
        lens, ws = i32([200, 7]), M.new_cache_attn_workspace()
        return lambda s: M.masked_gqa_attn_decode_window(q, k, v, lens, window=64, workspace=ws, stream=s)

    def tree(M):
        q, k, v = attn(3)
        new, lens, ws = randn(2, 2, 3, 64), i32([200, 7]), M.new_cache_attn_workspace()
        return lambda s: M.masked_gqa_attn_decode_tree(q, k, v, new, new, lens, workspace=ws, stream=s)

    def pack(M):
        a = randn(2, 4, 100, 64)
        return lambda s: M.masked_gqa_pack_pair(a, a, stream=s)[0]

    def unpack(M):
        a = randn(2, 4, 200, 64)
        return lambda s: M.masked_gqa_unpack_pair(a, 90, stream=s)[0]

    rope = dict(inv_freq=lambda: torch.rand(32, device="cuda"))
    return dict(prefill=plain("masked_gqa_attn_prefill", 256), prefill_rope=plain("masked_gqa_attn_prefill_rope", 256, **rope),
                prefill_window=plain("masked_gqa_attn_prefill_window", 256, window=lambda: 32),
                decode=plain("masked_gqa_attn_decode", 1), decode_static=plain("masked_gqa_attn_decode_static", 1),
                append=append, append_rope=append_rope, decode_window=window, decode_tree=tree, pack=pack, unpack=unpack)


@pytest.mark.parametrize("name", list(outputs()))
def test_own_output_spares_memory_in_use(M, name):
    call = outputs()[name](M)
    want = call(None).clone()
    s = torch.cuda.Stream()
    for on in (s, s.cuda_stream):
        total = sum_in_flight(want.numel() * want.element_size())
        out = call(on)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert int(total) == 7 * want.numel() * want.element_size()


def test_output_lives_while_the_current_stream_reads_it(M):
    call = outputs()["prefill"](M)
    want = call(None).float().sum()
    s = torch.cuda.Stream()
    out = call(s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(DELAY)
    total, shape = out.float().sum(), out.shape
    del out
    with torch.cuda.stream(s):  # s may not get the block again before that sum is done
        junk = [torch.full(shape, 1e4, dtype=BF, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert float(total) == float(want) and len(junk) == 4
