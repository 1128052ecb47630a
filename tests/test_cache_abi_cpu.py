"""Host-side checks of the windowed, tree and cache calls that need no GPU: the
struct mirrors, and that bad arguments are refused before anything is launched."""
import ctypes
import os
import subprocess

import pytest
import torch

import masked_gqa_attention_gb300 as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, CUDA = M.MGQA_ERR_INVALID_ARG, M.MGQA_ERR_UNSUPPORTED, M.MGQA_ERR_CUDA
BASE = 1 << 20  # fake pointers, never dereferenced: validation fails, or there is no GPU to launch on
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="on a GPU machine the call would run on fake pointers")


@pytest.fixture(scope="module")
def L():
    M.build_library()
    return M.lib()


@pytest.mark.parametrize("cname,py", [("mgqa_pages", M.MgqaPages), ("mgqa_tree", M.MgqaTree), ("mgqa_cache", M.MgqaCache)])
def test_struct_layout_matches_header(tmp_path, cname, py):
    fields = [f for f, _ in py._fields_]
    body = "\n".join(f'printf("{f} %zu\\n", offsetof({cname}, {f}));' for f in fields)
    src, exe = tmp_path / "off.c", tmp_path / "off"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "masked_gqa_attn.h"\n'
                   f'int main(void){{ {body} printf("size %zu\\n", sizeof({cname})); return 0; }}\n')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include", str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    got = dict(line.split() for line in out if line)
    for f in fields:
        assert int(got[f]) == getattr(py, f).offset, f
    assert int(got["size"]) == ctypes.sizeof(py)


def args(Lq=1, cap=1024, B=2):
    a = M.MgqaArgs()
    a.dtype = M.MGQA_BF16
    a.B, a.Hq, a.Hkv, a.Lq, a.Lk, a.D = B, 8, 2, Lq, cap, 64
    a.q, a.k, a.v, a.out = BASE, BASE * 2, BASE * 3, BASE * 4
    a.q_stride[:] = a.o_stride[:] = [8 * Lq * 64, Lq * 64, 64]
    a.k_stride[:] = a.v_stride[:] = [2 * cap * 64, cap * 64, 64]
    a.scale, a.kv_len = 0.125, BASE * 5
    return a


def pages():
    return M.MgqaPages(BASE * 6, 64, 500, 16, 64)


def tree(T):
    t = M.MgqaTree()
    t.k_new, t.v_new, t.bits = BASE * 7, BASE * 8, BASE * 9
    t.k_stride[:] = t.v_stride[:] = [2 * T * 64, T * 64, 64]
    t.bits_stride_b, t.bits_stride_t = T * ((T + 31) // 32), (T + 31) // 32
    return t


def ref(x):
    return None if x is None else ctypes.byref(x)


def window_call(L, a, p, window=100, sinks=4, ws=BASE * 10, n=None):
    n = L.masked_gqa_attn_cache_workspace_size() if n is None else n
    return L.masked_gqa_attn_decode_window(ref(a), ref(p), window, sinks, ws, n, None)


def tree_call(L, a, p, t, window=0, sinks=0, ws=BASE * 10, n=None):
    n = L.masked_gqa_attn_cache_workspace_size() if n is None else n
    return L.masked_gqa_attn_decode_tree(ref(a), ref(p), ref(t), window, sinks, ws, n, None)


@no_gpu
def test_good_arguments_reach_the_launch(L):
    assert window_call(L, args(), None) == CUDA
    assert window_call(L, args(), pages()) == CUDA
    for T in (1, 7, 256):
        assert tree_call(L, args(T), None, tree(T)) == CUDA
        assert tree_call(L, args(T), pages(), tree(T), 50, 4) == CUDA
    a = args(40)
    for dt in (M.MGQA_FP16, M.MGQA_FP32):
        a.dtype = dt
        assert tree_call(L, a, pages(), tree(40)) == CUDA
    a = args(300, 300)
    assert L.masked_gqa_attn_prefill_window(ref(a), 10, 0, None) == CUDA


@pytest.mark.parametrize("change,code", [
    (lambda a, p: setattr(a, "Lq", 2), INVALID),
    (lambda a, p: setattr(a, "kv_len", None), INVALID),
    (lambda a, p: setattr(a, "kv_len", BASE + 2), INVALID),
    (lambda a, p: setattr(a, "mask_bits", BASE), INVALID),
    (lambda a, p: (setattr(a, "seg_q", BASE), setattr(a, "seg_k", BASE)), INVALID),
    (lambda a, p: setattr(a, "causal", 1), INVALID),
    (lambda a, p: setattr(a, "D", 96), UNSUPPORTED),
    (lambda a, p: setattr(a, "Lk", (1 << 24) + 16), UNSUPPORTED),
    (lambda a, p: setattr(a, "scale", float("inf")), INVALID),
    (lambda a, p: a.k_stride.__setitem__(0, 12), INVALID),
    (lambda a, p: setattr(a, "v", BASE + 8), INVALID),
    (lambda a, p: setattr(p, "table", None), INVALID),
    (lambda a, p: setattr(p, "table", BASE + 2), INVALID),
    (lambda a, p: setattr(p, "num_pages", 0), INVALID),
    (lambda a, p: setattr(p, "page_size", 0), INVALID),
    (lambda a, p: setattr(p, "page_size", 8), INVALID),  # max_pages * page_size is not Lk
    (lambda a, p: setattr(p, "table_stride", 63), INVALID),
])
def test_cached_calls_refuse(L, change, code):
    a, p = args(), pages()
    change(a, p)
    assert window_call(L, a, p) == code
    assert L.mgqa_last_error_detail() != b""
    if a.Lq == 1:
        assert tree_call(L, a, p, tree(1)) == code


def test_windows_and_workspaces_refuse(L):
    n = L.masked_gqa_attn_cache_workspace_size()
    assert n > 0
    for w, s in ((0, 0), (-1, 0), (5, -1)):
        assert window_call(L, args(), None, w, s) == INVALID
        assert L.masked_gqa_attn_prefill_window(ref(args(9)), w, s, None) == INVALID
    assert tree_call(L, args(3), None, tree(3), -1, 0) == INVALID
    assert tree_call(L, args(3), None, tree(3), 0, -1) == INVALID
    for ws, size in ((None, n), (BASE + 8, n), (BASE, n - 1), (BASE, 0)):
        assert window_call(L, args(), None, ws=ws, n=size) == INVALID
        assert tree_call(L, args(3), None, tree(3), ws=ws, n=size) == INVALID
    assert window_call(L, None, None) == INVALID
    assert L.masked_gqa_attn_prefill_window(None, 4, 0, None) == INVALID


@pytest.mark.parametrize("change", [
    lambda t: setattr(t, "k_new", None), lambda t: setattr(t, "v_new", BASE + 4),
    lambda t: t.k_stride.__setitem__(1, -64), lambda t: t.v_stride.__setitem__(2, 60),
    lambda t: setattr(t, "bits", BASE + 1), lambda t: setattr(t, "bits_stride_t", 1),
    lambda t: setattr(t, "bits_stride_b", -2), lambda t: setattr(t, "len", BASE + 3)])
def test_trees_refuse(L, change):
    t = tree(40)
    change(t)
    assert tree_call(L, args(40), None, t) == INVALID
    assert tree_call(L, args(40), None, None) == INVALID
    assert tree_call(L, args(257), None, tree(257)) == UNSUPPORTED


def cache():
    c = M.MgqaCache()
    c.dtype, c.layers, c.num_pages, c.Hkv, c.page_size, c.D = M.MGQA_BF16, 2, 100, 2, 16, 64
    c.k, c.v = BASE, BASE * 2
    c.k_stride[:] = c.v_stride[:] = [100 * 2 * 16 * 64, 2 * 16 * 64, 16 * 64, 64]
    c.rows, c.max_pages, c.page_table, c.table_stride = 8, 10, BASE * 3, 10
    c.kv_len, c.ref = BASE * 4, BASE * 5
    return c


def append(L, c, T=3, out=BASE * 8, index=None, count=None, k=BASE * 6, stride=64):
    s = (ctypes.c_int64 * 4)(0, 2 * T * 64, T * 64, stride)
    return L.masked_gqa_cache_append(ref(c), k, BASE * 7, ctypes.addressof(s), ctypes.addressof(s), T, index, count, out, None)


def fork(L, c, n=3, src=BASE * 6, dst=BASE * 7, extra=0, ws=BASE * 8, size=None):
    size = 1 << 30 if size is None else size
    return L.masked_gqa_cache_fork(ref(c), n, src, dst, extra, ws, size, None)


def compact(L, c, to=BASE * 6, stride=10, r=BASE * 7, used=None, ws=BASE * 8, size=1 << 30):
    return L.masked_gqa_cache_compact(ref(c), to, stride, r, used, ws, size, None)


@no_gpu
def test_good_caches_reach_the_launch(L):
    c = cache()
    assert append(L, c) == CUDA and fork(L, c) == CUDA and compact(L, c) == CUDA
    assert fork(L, c, n=0, src=None, dst=None) == M.MGQA_OK  # nothing to do
    c.page_table, c.ref, c.num_pages = None, None, c.rows
    assert append(L, c) == CUDA  # the static cache


@pytest.mark.parametrize("change,code", [
    (lambda c: setattr(c, "dtype", 9), INVALID), (lambda c: setattr(c, "layers", 0), INVALID),
    (lambda c: setattr(c, "page_size", 0), INVALID), (lambda c: setattr(c, "rows", 0), INVALID),
    (lambda c: setattr(c, "D", 4), UNSUPPORTED), (lambda c: setattr(c, "k", None), INVALID),
    (lambda c: setattr(c, "v", BASE + 8), INVALID), (lambda c: c.k_stride.__setitem__(3, 4), INVALID),
    (lambda c: c.v_stride.__setitem__(0, -64), INVALID), (lambda c: setattr(c, "kv_len", BASE + 1), INVALID),
    (lambda c: setattr(c, "dev_error", BASE + 1), INVALID), (lambda c: setattr(c, "page_table", BASE + 1), INVALID),
    (lambda c: setattr(c, "max_pages", 0), INVALID), (lambda c: setattr(c, "table_stride", 9), INVALID),
    (lambda c: setattr(c, "max_pages", 1 << 21), INVALID), (lambda c: setattr(c, "page_table", None), INVALID)])
def test_caches_refuse(L, change, code):
    c = cache()
    change(c)
    assert append(L, c) == code, L.mgqa_last_error_detail()
    assert fork(L, c) == code and compact(L, c) == code
    assert L.masked_gqa_cache_workspace_size(ref(c), 3) == 0


def test_cache_steps_refuse(L):
    for call in (append, fork, compact):
        assert call(L, None) == INVALID
    c = cache()
    assert append(L, c, T=0) == INVALID and append(L, c, out=None) == INVALID and append(L, c, out=c.kv_len) == INVALID
    assert append(L, c, index=BASE + 1) == INVALID and append(L, c, count=BASE + 2) == INVALID
    assert append(L, c, k=None) == INVALID and append(L, c, k=BASE + 8) == INVALID and append(L, c, stride=4) == INVALID
    assert fork(L, c, n=-1) == INVALID and fork(L, c, n=1025) == INVALID and fork(L, c, extra=-1) == INVALID
    assert fork(L, c, src=None) == INVALID and fork(L, c, dst=BASE + 1) == INVALID
    need = L.masked_gqa_cache_workspace_size(ref(c), 3)
    assert need > 0 and fork(L, c, size=need - 1) == INVALID and fork(L, c, ws=None) == INVALID
    assert fork(L, c, ws=BASE + 8) == INVALID
    assert L.masked_gqa_cache_workspace_size(ref(c), 1025) == 0
    need = L.masked_gqa_cache_workspace_size(ref(c), 0)
    assert need > 0 and compact(L, c, size=need - 1) == INVALID and compact(L, c, ws=None) == INVALID
    assert compact(L, c, to=None) == INVALID and compact(L, c, r=None) == INVALID and compact(L, c, used=BASE + 1) == INVALID
    assert compact(L, c, stride=9) == INVALID
    assert compact(L, c, to=c.page_table, stride=12) == INVALID  # in place, with another stride
    c.num_pages = (1 << 20) + 1
    assert fork(L, c) == UNSUPPORTED and compact(L, c) == UNSUPPORTED
    c = cache()
    c.ref = None
    assert fork(L, c) == INVALID and compact(L, c) == INVALID
    c = cache()
    c.kv_len = None
    assert fork(L, c) == INVALID and append(L, c) == INVALID


def test_windowed_prefill_refuses_expanded_tensors(L):
    for field, dtypes in (("k_stride", (M.MGQA_BF16, M.MGQA_FP32)), ("v_stride", (M.MGQA_FP16, M.MGQA_FP32)),
                          ("q_stride", (M.MGQA_BF16, M.MGQA_FP16))):
        for dt in dtypes:
            for i in range(3):
                a = args(9)
                a.dtype = dt
                getattr(a, field)[i] = 0
                assert L.masked_gqa_attn_prefill_window(ctypes.byref(a), 4, 0, None) == UNSUPPORTED
    a = args(1, B=1)  # one element: the stride says nothing
    a.q_stride[0] = a.k_stride[0] = a.q_stride[2] = 0
    if not torch.cuda.is_available():
        assert L.masked_gqa_attn_prefill_window(ctypes.byref(a), 4, 0, None) == CUDA


def test_binding_takes_all_arguments_or_none():
    calls = M._calls()
    for f in (calls.prefill_window, calls.decode_window, calls.decode_tree, calls.cache_append, calls.cache_fork,
              calls.cache_compact, calls.cache_workspace_size):
        with pytest.raises(TypeError, match="wanted"):
            f(1, 2, 3)
    with pytest.raises(ValueError, match="tensor"):
        calls.cache_workspace_size(1, 2, None, None, 0)
    k = torch.zeros(3, 2, 4, 64, dtype=torch.bfloat16)
    assert M.masked_gqa_cache_workspace_size(k, k, torch.zeros(5, 7, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)) > 0
    for bad in (torch.zeros(4, dtype=torch.int32), torch.zeros(3)):
        with pytest.raises(ValueError, match="ref"):
            M.masked_gqa_cache_workspace_size(k, k, torch.zeros(5, 7, dtype=torch.int32), bad)


def test_binding_refuses_tensors_off_the_gpu():
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    n = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: M.masked_gqa_attn_prefill_window(q, q, q, window=3),
                 lambda: M.masked_gqa_attn_decode_window(q, q, q, n, window=3),
                 lambda: M.masked_gqa_attn_decode_tree(q, q, q, q, q, n),
                 lambda: M.masked_gqa_cache_append(q, q, q, q, n, n.clone()),
                 lambda: M.masked_gqa_cache_fork(q, q, n[None], n, n, n, n),
                 lambda: M.masked_gqa_cache_compact(q, q, n[None], n)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
