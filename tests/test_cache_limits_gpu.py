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
