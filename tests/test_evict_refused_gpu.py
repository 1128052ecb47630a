"""What eviction leaves of a request that it refuses, in buffers of its own as in place."""
import pytest
import torch

from test_evict_gpu import INVALID, M, Evict, i32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fault", ["shared", "missing", "outside", "long", "negative"])
@pytest.mark.parametrize("n,budget", [(100, 40), (20000, 300), (330000, 5000)])
def test_refused_requests_keep_their_weights(M, fault, n, budget):  # noqa: F811
    """weight_out gets the weights as they are, as long as the length is one (else nothing), and the length goes on."""
    c = Evict([n, n - 7], budget, 2, 8, layers=2, page=16, cap=n + 12)
    k, v, lens, table, ref = (x.clone() for x in (c.k, c.v, c.kv_len, c.table, c.ref))
    if fault == "shared":
        ref[table[0, 1].long()] = 2
    elif fault == "missing":
        table[0, 5] = -1
    elif fault == "outside":
        table[0, (n - 1) // 16] = 10 ** 6
    else:
        lens[0] = 10 ** 6 if fault == "long" else -1
    out, len_out, err = torch.full_like(c.w, 9.0), i32([-7, -7]), i32([0])
    was = lens[0].item(), table[0].clone()
    M.masked_gqa_cache_evict(k, v, c.w, lens, budget=budget, sinks=2, recent=8, page_table=table, ref=ref,
                             weight_out=out, kv_len_out=len_out, dev_error=err)
    assert int(err) == INVALID and len_out.tolist() == [was[0], budget] and torch.equal(table[0], was[1])
    want = torch.full_like(c.w, 9.0)
    if fault not in ("long", "negative"):
        want[:, 0, :, :n] = c.w[:, 0, :, :n]
    assert torch.equal(out[:, 0], want[:, 0])
    mine = c.table[0][c.table[0] >= 0].long()
    assert torch.equal(k[:, mine], c.k[:, mine]) and torch.equal(v[:, mine], c.v[:, mine])
    keep = c.want(1, 1, 0)
    assert torch.equal(out[1, 1, 0, :budget], c.w[1, 1, 0, keep]) and (out[1, 1, 0, budget:n - 7] == 0).all()
