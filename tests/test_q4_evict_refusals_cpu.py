"""Calls over a cache in 4 bits, of the accumulated weights and of the eviction that
are refused before anything is launched, and the binding's own checks."""
import ctypes

import pytest
import torch

import masked_gqa_attention_gb300 as M
from test_cache_abi_cpu import BASE, CUDA, INVALID, UNSUPPORTED, args, cache, no_gpu, pages, ref


@pytest.fixture(scope="module")
def L():
    M.build_library()
    return M.lib()


def q4_args(T=1, cap=1024):
    a = args(T, cap)
    a.k_stride[:] = a.v_stride[:] = [2 * cap * 48, cap * 48, 48]
    a.lse = BASE * 12
    return a


def decode(L, a, p=None, window=0, sinks=0, ws=BASE * 10, n=None):
    n = L.masked_gqa_attn_cache_workspace_size() if n is None else n
    return L.masked_gqa_attn_decode_q4(ref(a), ref(p), window, sinks, ws, n, None)


def weights(L, a, p=None, window=0, sinks=0, q4=1, w=BASE * 11, st=(2048, 1024), slots=1024):
    s = None if st is None else (ctypes.c_int64 * 2)(*st)
    return L.masked_gqa_attn_cache_weights(ref(a), ref(p), window, sinks, q4, w, s and ctypes.addressof(s), slots, None)


@no_gpu
def test_good_arguments_reach_the_launch(L):
    for T in (1, 2, 256):
        for dt in (M.MGQA_BF16, M.MGQA_FP16, M.MGQA_FP32):
            a = q4_args(T)
            a.dtype = dt
            assert decode(L, a) == CUDA and decode(L, a, pages(), 5, 3) == CUDA
            assert weights(L, a) == CUDA and weights(L, a, pages(), 5, 3) == CUDA
            b = args(T)
            b.dtype, b.lse, b.v, b.out = dt, BASE * 12, None, None  # not looked at
            assert weights(L, b, q4=0) == CUDA
    assert weights(L, q4_args(), slots=3, st=(6, 3)) == CUDA
    assert weights(L, q4_args(), st=(1024, 2048)) == CUDA  # heads outside requests
    assert evict(L, cache()) == CUDA and evict(L, cache(), out=BASE * 40) == CUDA
    c = cache()
    c.ref = None
    assert evict(L, c) == CUDA
    c.page_table, c.num_pages = None, c.rows
    assert evict(L, c) == CUDA and append(L, q4_cache()) == CUDA


@pytest.mark.parametrize("change,code", [
    (lambda a, p: setattr(a, "Lq", 257), UNSUPPORTED), (lambda a, p: setattr(a, "Lq", 0), INVALID),
    (lambda a, p: setattr(a, "kv_len", None), INVALID), (lambda a, p: setattr(a, "mask_bits", BASE), INVALID),
    (lambda a, p: setattr(a, "causal", 1), INVALID), (lambda a, p: setattr(a, "D", 96), UNSUPPORTED),
    (lambda a, p: setattr(a, "D", 256), UNSUPPORTED), (lambda a, p: setattr(a, "Hq", 7), INVALID),
    (lambda a, p: setattr(a, "scale", float("nan")), INVALID), (lambda a, p: a.k_stride.__setitem__(2, 40), INVALID),
    (lambda a, p: a.k_stride.__setitem__(0, -48), INVALID), (lambda a, p: setattr(a, "k", BASE + 8), INVALID),
    (lambda a, p: setattr(a, "k", None), INVALID), (lambda a, p: setattr(a, "q", BASE + 2), INVALID),
    (lambda a, p: setattr(p, "table", None), INVALID), (lambda a, p: setattr(p, "page_size", 8), INVALID),
    (lambda a, p: setattr(p, "table_stride", 63), INVALID), (lambda a, p: setattr(a, "Lk", 1 << 25), UNSUPPORTED)])
def test_the_last_tokens_refuse(L, change, code):
    a, p = q4_args(), pages()
    change(a, p)
    assert decode(L, a, p) == code and L.mgqa_last_error_detail() != b""
    assert weights(L, a, p) == code and L.mgqa_last_error_detail() != b""


def test_windows_workspaces_and_weights_refuse(L):
    n = L.masked_gqa_attn_cache_workspace_size()
    assert decode(L, None) == INVALID and weights(L, None) == INVALID
    for w, s in ((-1, 0), (0, -1)):
        assert decode(L, q4_args(), None, w, s) == INVALID and weights(L, q4_args(), None, w, s) == INVALID
    for ws, size in ((None, n), (BASE + 8, n), (BASE, n - 1)):
        assert decode(L, q4_args(), ws=ws, n=size) == INVALID
    a = q4_args()
    a.v = None
    assert decode(L, a) == INVALID
    a.lse = None
    assert weights(L, a) == INVALID
    a = q4_args()
    for kw in (dict(w=None), dict(w=BASE + 2), dict(st=None), dict(slots=0), dict(st=(2048, 1023)), dict(st=(1024, 1024)),
               dict(st=(0, 1024)), dict(st=(-2048, 1024)), dict(st=(1 << 62, 1024))):
        assert weights(L, a, **kw) == INVALID, kw


def q4_cache():
    c = cache()
    c.k_stride[:] = c.v_stride[:] = [100 * 2 * 16 * 48, 2 * 16 * 48, 16 * 48, 48]
    return c


def append(L, c, T=3, out=BASE * 8, index=None, count=None, k=BASE * 6, stride=64):
    s = (ctypes.c_int64 * 4)(0, 2 * T * 64, T * 64, stride)
    return L.masked_gqa_cache_append_q4(ref(c), k, BASE * 7, ctypes.addressof(s), ctypes.addressof(s), T, index, count, out,
                                        None)


@pytest.mark.parametrize("change,code", [
    (lambda c: setattr(c, "dtype", 9), INVALID), (lambda c: setattr(c, "D", 96), UNSUPPORTED),
    (lambda c: setattr(c, "k", BASE + 8), INVALID), (lambda c: c.k_stride.__setitem__(3, 40), INVALID),
    (lambda c: c.v_stride.__setitem__(0, -48), INVALID), (lambda c: setattr(c, "kv_len", None), INVALID),
    (lambda c: setattr(c, "max_pages", 0), INVALID), (lambda c: setattr(c, "page_table", None), INVALID)])
def test_appending_records_refuses(L, change, code):
    c = q4_cache()
    change(c)
    assert append(L, c) == code and L.mgqa_last_error_detail() != b""
    c = q4_cache()
    assert append(L, None) == INVALID and append(L, c, T=0) == INVALID and append(L, c, out=c.kv_len) == INVALID
    assert append(L, c, k=BASE + 8) == INVALID and append(L, c, stride=4) == INVALID and append(L, c, index=BASE + 1) == INVALID


def evict(L, c, w=BASE * 30, out=BASE * 30, st=(8 * 2 * 160, 2 * 160, 160), so=None, slots=160, budget=32, sinks=2, recent=8,
          to=BASE * 4, ws=BASE * 50, size=1 << 30):
    st = None if st is None else (ctypes.c_int64 * 3)(*st)
    so = st if so is None else (ctypes.c_int64 * 3)(*so)
    at = lambda x: None if x is None else ctypes.addressof(x)  # noqa: E731
    return L.masked_gqa_cache_evict(ref(c), w, at(st), out, at(so), slots, budget, sinks, recent, to, ws, size, None)


@pytest.mark.parametrize("kw", [
    dict(budget=0), dict(budget=-1), dict(budget=(1 << 24) + 1), dict(sinks=-1), dict(recent=-1), dict(sinks=20, recent=13),
    dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), dict(w=None), dict(out=None), dict(w=BASE * 30 + 2), dict(st=None),
    dict(slots=0), dict(st=(8 * 2 * 160, 2 * 160, 159)), dict(st=(8 * 2 * 160 - 1, 2 * 160, 160)),
    dict(so=(16 * 2 * 160, 2 * 160, 160)), dict(out=BASE * 30 + 4 * 160), dict(out=BASE * 30 + 4 * (2 * 8 * 2 * 160 - 1)),
    dict(to=None), dict(to=BASE * 4 + 2), dict(to=BASE * 4 + 4), dict(to=BASE * 3 + 8), dict(to=BASE * 30 + 64),
    dict(ws=None), dict(ws=BASE * 50 + 8), dict(size=64)])
def test_evictions_refuse(L, kw):
    assert evict(L, cache(), **kw) == INVALID and L.mgqa_last_error_detail() != b""


def test_evictions_refuse_caches(L):
    assert evict(L, None) == INVALID
    for change, code in ((lambda c: setattr(c, "kv_len", None), INVALID), (lambda c: setattr(c, "ref", BASE + 1), INVALID),
                         (lambda c: setattr(c, "D", 4), UNSUPPORTED), (lambda c: setattr(c, "layers", 0), INVALID),
                         (lambda c: setattr(c, "rows", 1 << 25), UNSUPPORTED)):
        c = cache()
        change(c)
        assert evict(L, c) == code, L.mgqa_last_error_detail()
    c = cache()
    c.page_table, c.num_pages = None, c.rows  # counts without a table
    assert evict(L, c) == INVALID
    need = L.masked_gqa_cache_evict_workspace_size(ref(cache()), 32)
    assert need > 0 and evict(L, cache(), size=need - 1) == INVALID
    for budget in (0, -5, (1 << 24) + 1):
        assert L.masked_gqa_cache_evict_workspace_size(ref(cache()), budget) == 0


def test_binding_takes_all_arguments_or_none():
    calls = M._calls()
    for f in (calls.cache_append_q4, calls.decode_q4, calls.cache_weights, calls.cache_evict,
              calls.cache_evict_workspace_size):
        with pytest.raises(TypeError, match="wanted"):
            f(1, 2)
    k = torch.zeros(3, 2, 4, 48, dtype=torch.uint8)
    table, count = torch.zeros(5, 7, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    assert M.masked_gqa_cache_evict_workspace_size(k, k, 9, page_table=table) > 0
    assert M.masked_gqa_cache_workspace_size(k, k, table, count) > 0  # (fork and compact of records)
    odd = torch.zeros(3, 2, 4, 40, dtype=torch.uint8)
    with pytest.raises(ValueError, match="16 bytes"):
        M.masked_gqa_cache_evict_workspace_size(odd, odd, 9)
    with pytest.raises(ValueError, match="16 bytes"):
        apart = torch.zeros(3, 2, 4, 50, dtype=torch.uint8)[..., :48]
        M.masked_gqa_cache_evict_workspace_size(apart, apart, 9)
    with pytest.raises(M.MgqaError, match="budget"):
        M.masked_gqa_cache_evict_workspace_size(k, k, 0)


def test_no_workspace_for_a_budget_that_nobody_exceeds(L):
    c = cache()
    least = L.masked_gqa_cache_evict_workspace_size(ref(c), c.max_pages * c.page_size)
    assert 0 < least <= 64 and L.masked_gqa_cache_evict_workspace_size(ref(c), 1 << 24) == least
    assert L.masked_gqa_cache_evict_workspace_size(ref(c), c.max_pages * c.page_size - 1) > 1000


def test_binding_refuses_tensors_off_the_gpu():
    q, rec = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 4, 48, dtype=torch.uint8)
    n, lse, w = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, 1), torch.zeros(1, 2, 4)
    for call in (lambda: M.masked_gqa_attn_decode_q4(q, rec, rec, n),
                 lambda: M.masked_gqa_cache_append_q4(rec, rec, q, q, n, n.clone()),
                 lambda: M.masked_gqa_attn_cache_weights(q, rec, n, lse, w),
                 lambda: M.masked_gqa_cache_evict(rec, rec, w, n, budget=2)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
