"""What the windowed prefill refuses of its tensors, whichever mask forms they come with."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import masked_gqa_attention_gb300 as M
    M.build_library()
    return M


def forms(B, L):
    """Mask forms that allow every key, by name."""
    one = torch.ones(B, L, dtype=torch.int32, device="cuda")
    return {"plain": {}, "bits": dict(mask_bits=torch.full((1, 1, 4), -1, dtype=torch.int32, device="cuda")),
            "segments": dict(seg_q=one, seg_k=one)}


@pytest.mark.parametrize("form", ["plain", "bits", "segments"])
def test_lengths_and_error_words_of_other_shapes_are_refused(M, form):
    B, L = 3, 100
    q = torch.randn(B, 2, L, 64, device="cuda").bfloat16()
    masks = forms(B, L)[form]
    i32 = lambda *n: torch.full(n, 50, dtype=torch.int32, device="cuda")  # noqa: E731
    call = lambda **kw: M.masked_gqa_attn_prefill_window(q, q, q, window=9, **masks, **kw)  # noqa: E731
    for bad in (i32(1), i32(2), i32(4), i32(3, 1), i32(6)[::2], i32(0)):
        with pytest.raises(ValueError, match="kv_len"):
            call(kv_len=bad)
    for bad in (i32(0), i32(2), i32(1, 1)):
        with pytest.raises(ValueError, match="dev_error"):
            call(dev_error=bad)
    with pytest.raises(ValueError, match="kv_len"):
        call(kv_len=i32(3).long())
    err = i32(1).zero_()
    assert torch.isfinite(call(kv_len=i32(3), dev_error=err)).all() and int(err) == 0


def test_forms_agree(M):
    B, L = 3, 100
    q, k, v = (torch.randn(B, 2, L, 64, device="cuda").bfloat16() for _ in range(3))
    n = torch.tensor([100, 31, 0], dtype=torch.int32, device="cuda")
    a, b, c = (M.masked_gqa_attn_prefill_window(q, k, v, window=20, sinks=2, kv_len=n, **m) for m in forms(B, L).values())
    assert torch.equal(a, b) and torch.equal(a, c)
