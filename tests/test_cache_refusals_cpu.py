"""Calls of the cache's steps that are refused before anything is launched."""

import pytest

import masked_gqa_attention_gb300 as M
from test_cache_abi_cpu import BASE, CUDA, INVALID, UNSUPPORTED, append, cache, compact, fork, no_gpu, ref


@pytest.fixture(scope="module")
def L():
    M.build_library()
    return M.lib()


def overlapping(c, T):
    """(what kv_len_out lies in, its first and last element's address, the arguments of append)."""
    index, count = BASE * 9, BASE * 10
    kw = dict(index=index, count=count, T=T)
    table = ((c.rows - 1) * c.table_stride + c.max_pages) * 4
    return [("kv_len", c.kv_len, 4 * c.rows, kw), ("count", count, 4 * c.rows, kw),
            ("index", index, 4 * c.rows * T, kw), ("table", c.page_table, table, kw)]


@pytest.mark.parametrize("what", range(4))
@pytest.mark.parametrize("T", [1, 3])
def test_new_lengths_that_overlap_an_input_are_refused(L, what, T):
    c = cache()
    name, at, size, kw = overlapping(c, T)[what]
    for out in (at, at + 4, at - 4, at + size - 4, at - 4 * (c.rows - 1)):
        assert append(L, c, out=out, **kw) == INVALID, (name, out - at)
        assert b"overlap" in L.mgqa_last_error_detail()


@no_gpu
@pytest.mark.parametrize("what", range(4))
def test_new_lengths_beside_an_input_are_taken(L, what):
    c = cache()
    name, at, size, kw = overlapping(c, 3)[what]
    for out in (at - 4 * c.rows, at + size):
        assert append(L, c, out=out, **kw) == CUDA, (name, out - at)


@no_gpu
def test_new_lengths_of_the_static_cache(L):
    c = cache()
    c.page_table, c.max_pages, c.table_stride, c.num_pages = None, 0, 0, c.rows
    assert append(L, c, out=c.kv_len + 4 * c.rows) == CUDA
    assert append(L, c, out=c.kv_len + 4 * c.rows - 4) == INVALID


@pytest.mark.parametrize("page,D,dtype", [(1 << 24, 2048, M.MGQA_BF16), (1 << 24, 513 * 8, M.MGQA_FP16),
                                          (1 << 24, 260, M.MGQA_FP32), ((1 << 23) + 1, 1024, M.MGQA_BF16)])
def test_copied_pages_past_32_bits_are_refused(L, page, D, dtype):
    c = cache()
    c.page_size, c.max_pages, c.D, c.dtype = page, 1, D, dtype
    assert fork(L, c) == UNSUPPORTED and compact(L, c) == UNSUPPORTED
    assert L.masked_gqa_cache_workspace_size(ref(c), 3) == 0


@no_gpu
def test_the_largest_copied_pages_are_taken(L):
    c = cache()
    c.page_size, c.max_pages, c.D = 1 << 24, 1, 512
    assert fork(L, c) == CUDA and compact(L, c) == CUDA
    c.D = 2048  # (no page is copied)
    assert append(L, c) == CUDA
