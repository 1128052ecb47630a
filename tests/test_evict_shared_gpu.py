"""Eviction of requests that share the pages of a common beginning."""
import pytest
import torch

from test_evict_gpu import BF, INVALID, M, Evict, i32  # noqa: F401

pytestmark = pytest.mark.gpu


def beginning(c, pages):
    """Request 1 takes the first `pages` pages of request 0 for its own first ones."""
    for i in range(pages):
        c.ref[c.table[1, i].long()] -= 1
        c.table[1, i] = c.table[0, i]
        c.ref[c.table[0, i].long()] += 1


@pytest.mark.parametrize("dtype", [BF, torch.uint8])
@pytest.mark.parametrize("budget,sinks,recent,pages", [(48, 16, 8, 1), (48, 20, 8, 1), (100, 64, 36, 4), (64, 64, 0, 4),
                                                       (70, 64, 0, 4), (40, 37, 0, 2)])
def test_pages_inside_the_sinks_may_be_shared(M, dtype, budget, sinks, recent, pages):  # noqa: F811
    """They are not written to: their rows and counts stay, and both requests are cut."""
    c = Evict([150, 130], budget, sinks, recent, layers=2, dtype=dtype, page=16, cap=160)
    beginning(c, pages)
    c.run(M, with_ref=True)
    c.run(M, with_ref=True, in_place=False)


@pytest.mark.parametrize("budget,sinks,pages", [(48, 15, 1), (48, 16, 2), (64, 20, 2), (40, 40, 3), (48, 0, 1)])
def test_pages_past_the_sinks_may_not(M, budget, sinks, pages):  # noqa: F811
    """(The page of slot `sinks` is one of them.)"""
    c = Evict([150, 130, 90], budget, sinks, 0, page=16, cap=160)
    beginning(c, pages)
    k, v, w, lens, table, ref, err = (x.clone() for x in (c.k, c.v, c.w, c.kv_len, c.table, c.ref, c.err))
    M.masked_gqa_cache_evict(k, v, w, lens, budget=budget, sinks=sinks, page_table=table, ref=ref, dev_error=err)
    assert int(err) == INVALID and lens.tolist() == [150, 130, budget]
    assert torch.equal(table[:2], c.table[:2]) and torch.equal(w[:, :2], c.w[:, :2])
    held = torch.cat([c.table[b][c.table[b] >= 0] for b in range(2)]).long()
    assert torch.equal(k[:, held], c.k[:, held]) and torch.equal(v[:, held], c.v[:, held])
    assert torch.equal(ref[held], c.ref[held])


def test_forked_requests_are_cut(M):  # noqa: F811
    """Fork shares the full pages of a prompt; with them inside the sinks both are cut, apart from one another."""
    c = Evict([130, 0], 60, 48, 4, page=16, cap=160)
    k, v, w, lens, table, ref, err = (x.clone() for x in (c.k, c.v, c.w, c.kv_len, c.table, c.ref, c.err))
    table[1], ref[c.table[1][c.table[1] >= 0].long()] = -1, 0
    M.masked_gqa_cache_fork(k, v, table, lens, ref, i32([0]), i32([1]), extra=0, dev_error=err)
    assert int(err) == 0 and lens.tolist() == [130, 130] and torch.equal(table[0, :8], table[1, :8])
    M.masked_gqa_cache_evict(k, v, w, lens, budget=60, sinks=48, recent=4, page_table=table, ref=ref, dev_error=err)
    assert int(err) == INVALID and lens.tolist() == [130, 130]  # page 3 is shared and would be written to
    M.masked_gqa_cache_evict(k, v, w, lens, budget=128, sinks=128, page_table=table, ref=ref, dev_error=err.zero_())
    assert int(err) == 0 and lens.tolist() == [128, 128] and (ref[table[0, :8].long()] == 2).all()
    assert (table[:, 8:] == -1).all()
    kept = table[0, :8].long()
    assert torch.equal(k[:, kept], c.k[:, kept]) and torch.equal(v[:, kept], c.v[:, kept])
