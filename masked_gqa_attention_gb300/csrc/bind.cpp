// The Python side of the calls that a serving loop makes once per layer and token
// (sliding windows, drafted tokens, the cache's own steps): tensors checked and
// passed to the C ABI in one native call. (Marshalled in Python, a call of drafted
// tokens took 13.0 us of the host's time and an append 9.6; here 4.1 and 2.5,
// nearly all of it the launch.)
//
// Every function takes its arguments by position, as the wrappers in __init__.py
// pass them, raises ValueError for tensors that do not fit together, and returns
// the C function's status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/masked_gqa_attn.h"

namespace {

using at::Tensor;

struct PythonError {};  // a Python exception is set

[[noreturn]] void bad(const std::string &what) { throw std::invalid_argument(what); }

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
const Tensor *optional_tensor(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }

int device_of(const Tensor &first) {
  if (!first.is_cuda()) bad("tensors must be CUDA tensors");
  return first.get_device();
}
struct Named {
  const Tensor *t;
  const char *name;
};
void together(int dev, std::initializer_list<Named> others) {
  for (const Named &o : others)
    if (o.t && (!o.t->is_cuda() || o.t->get_device() != dev))
      bad(std::string(o.name) + " is on " + o.t->device().str() + ", not on cuda:" + std::to_string(dev));
}

mgqa_dtype dtype_of(const Tensor &t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MGQA_BF16;
    case at::kHalf: return MGQA_FP16;
    case at::kFloat: return MGQA_FP32;
    default: bad("tensors must be bfloat16, float16 or float32");
  }
}

// Address of an int32 tensor of the given shape (null: absent).
int32_t *ints(const Tensor *t, const char *name, std::initializer_list<int64_t> shape) {
  if (!t) return nullptr;
  if (t->scalar_type() != at::kInt || t->sizes() != at::IntArrayRef(shape) || !t->is_contiguous()) {
    std::string s;
    for (int64_t n : shape) s += (s.empty() ? "" : ", ") + std::to_string(n);
    bad(std::string(name) + " must be contiguous int32 [" + s + "]");
  }
  return static_cast<int32_t *>(t->data_ptr());
}
int32_t small(int64_t n, const char *what) {
  if (n > 0x7fffffff) bad(std::string(what) + " past 2^31");
  return (int32_t)n;
}

// A Python integer as a 32-bit count: what lies past the range stays past every size.
int32_t count(PyObject *o) {
  PyObject *i = PyNumber_Index(o);
  if (!i) throw PythonError();
  int over = 0;
  const long long x = PyLong_AsLongLongAndOverflow(i, &over);
  Py_DECREF(i);
  if (over) return over < 0 ? -1 : 0x7fffffff;
  if (x == -1 && PyErr_Occurred()) throw PythonError();
  return x < -1 ? -1 : x > 0x7fffffff ? 0x7fffffff : (int32_t)x;
}

// Device `dev` made current for a call, and the call's stream: the device's
// current one unless one is given (an object with `cuda_stream`, or a handle).
struct Launch {
  std::optional<c10::cuda::CUDAGuard> guard;
  cudaStream_t stream;

  Launch(int dev, PyObject *o) {
    if (c10::cuda::current_device() != dev) guard.emplace((c10::DeviceIndex)dev);
    if (o == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
      return;
    }
    PyObject *h = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
    if (!h) throw PythonError();
    void *p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!p && PyErr_Occurred()) throw PythonError();
    stream = static_cast<cudaStream_t>(p);
  }
};

// The attention arguments for k / v [B, Hkv, slots, D] or, with a page table,
// [pages, Hkv, page_size, D].
struct Attention {
  mgqa_args a{};
  mgqa_pages pages{};
  const mgqa_pages *paged = nullptr;

  Attention(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &out, const Tensor *kv_len, PyObject *scale,
            const Tensor *lse, const Tensor *err, const Tensor *table) {
    if (q.dim() != 4 || k.dim() != 4 || v.sizes() != k.sizes() || out.sizes() != q.sizes())
      bad("q, out must be [B, Hq, L, D] and k, v [B or pages, Hkv, slots, D]");
    a.dtype = dtype_of(q);
    if (k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type() || out.scalar_type() != q.scalar_type())
      bad("q, out, k and v must share one dtype of bfloat16, float16, float32");
    if (k.size(3) != q.size(3) || q.stride(3) != 1 || k.stride(3) != 1 || v.stride(3) != 1 || out.stride(3) != 1)
      bad("the head dims must agree and have unit stride");
    a.B = small(q.size(0), "B");
    a.Hq = small(q.size(1), "Hq");
    a.Hkv = small(k.size(1), "Hkv");
    a.Lq = small(q.size(2), "L");
    a.D = small(q.size(3), "D");
    int64_t cap = k.size(2);
    if (table) {
      if (table->scalar_type() != at::kInt || table->dim() != 2 || table->size(0) != q.size(0) || table->stride(1) != 1)
        bad("page_table must be int32 [B, max_pages] with unit-stride rows");
      pages.table = static_cast<const int32_t *>(table->data_ptr());
      pages.table_stride = table->stride(0);
      pages.num_pages = small(k.size(0), "pages");
      pages.page_size = small(k.size(2), "page_size");
      pages.max_pages = small(table->size(1), "max_pages");
      paged = &pages;
      cap *= table->size(1);
    } else if (k.size(0) != q.size(0)) {
      bad("k and v without a page table must be [B, Hkv, slots, D]");
    }
    a.Lk = small(cap, "slots of a request");
    a.q = q.data_ptr();
    a.k = k.data_ptr();
    a.v = v.data_ptr();
    a.out = out.data_ptr();
    for (int t = 0; t < 3; ++t) {
      a.q_stride[t] = q.stride(t);
      a.k_stride[t] = k.stride(t);
      a.v_stride[t] = v.stride(t);
      a.o_stride[t] = out.stride(t);
    }
    a.kv_len = ints(kv_len, "kv_len", {q.size(0)});
    if (scale == Py_None) {
      a.scale = (float)(1.0 / std::sqrt((double)q.size(3)));
    } else {
      const double x = PyFloat_AsDouble(scale);
      if (x == -1.0 && PyErr_Occurred()) throw PythonError();
      a.scale = (float)x;
    }
    if (lse) {
      if (lse->scalar_type() != at::kFloat || lse->sizes() != q.sizes().slice(0, 3) || !lse->is_contiguous())
        bad("lse must be contiguous fp32 [B, Hq, L]");
      a.lse = static_cast<float *>(lse->data_ptr());
    }
    a.dev_error = ints(err, "dev_error", {1});
  }
};

// The cache of tensors [layers, pages, Hkv, page_size, D], or without the layers.
struct Cache {
  mgqa_cache c{};
  int64_t layers, rows, Hkv, D;

  Cache(const Tensor &k, const Tensor &v, const Tensor *table, const Tensor *kv_len, const Tensor *ref,
        const Tensor *err) {
    const int n = (int)k.dim(), x = n - 4;  // x: the page dimension
    if ((n != 4 && n != 5) || v.sizes() != k.sizes() || k.stride(n - 1) != 1 || v.stride(n - 1) != 1)
      bad("the caches must be [layers, pages, Hkv, page_size, D] (or 4-D, one layer) with a unit-stride head dim");
    if (v.scalar_type() != k.scalar_type()) bad("the caches must share one dtype of bfloat16, float16, float32");
    c.dtype = dtype_of(k);
    layers = x ? k.size(0) : 1;
    rows = k.size(x);
    Hkv = k.size(x + 1);
    D = k.size(x + 3);
    c.layers = small(layers, "layers");
    c.num_pages = small(rows, "pages");
    c.Hkv = small(Hkv, "Hkv");
    c.page_size = small(k.size(x + 2), "page_size");
    c.D = small(D, "D");
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    for (int t = 0; t < 4; ++t) {
      c.k_stride[t] = t || x ? k.stride(x - 1 + t) : 0;
      c.v_stride[t] = t || x ? v.stride(x - 1 + t) : 0;
    }
    if (table) {
      if (table->scalar_type() != at::kInt || table->dim() != 2 || table->stride(1) != 1)
        bad("page_table must be int32 [rows, max_pages] with unit-stride rows");
      rows = table->size(0);
      c.max_pages = small(table->size(1), "max_pages");
      c.page_table = static_cast<int32_t *>(table->data_ptr());
      c.table_stride = table->stride(0);
    }
    c.rows = small(rows, "rows");
    c.kv_len = ints(kv_len, "kv_len", {rows});
    c.ref = ints(ref, "ref", {k.size(x)});
    c.dev_error = ints(err, "dev_error", {1});
  }
};

// The status of a C call, made without the interpreter's lock: a launch may wait.
// (Nothing in it may throw: what PyTorch is asked for is asked before.)
template <typename F>
PyObject *status_of(F call) {
  mgqa_status st;
  Py_BEGIN_ALLOW_THREADS
  st = call();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// f(args) as a Python function of `want` positional arguments.
template <typename F>
PyObject *guarded(PyObject *const *, Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, want);
    return nullptr;
  }
  try {
    return f();
  } catch (const PythonError &) {
  } catch (const std::invalid_argument &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// q k v out kv_len scale lse dev_error causal window sinks stream
PyObject *prefill_window(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(o, n, 12, [&] {
    const Tensor &q = tensor(o[0], "q"), &k = tensor(o[1], "k"), &v = tensor(o[2], "v"), &out = tensor(o[3], "out");
    const Tensor *len = optional_tensor(o[4], "kv_len"), *lse = optional_tensor(o[6], "lse"),
                 *err = optional_tensor(o[7], "dev_error");
    const int dev = device_of(q);
    together(dev, {{&k, "k"}, {&v, "v"}, {&out, "out"}, {len, "kv_len"}, {lse, "lse"}, {err, "dev_error"}});
    Attention at(q, k, v, out, len, o[5], lse, err, nullptr);
    const int causal = PyObject_IsTrue(o[8]);
    if (causal < 0) throw PythonError();
    at.a.causal = causal;
    const int32_t window = count(o[9]), sinks = count(o[10]);
    const Launch l(dev, o[11]);
    return status_of([&] {
      return masked_gqa_attn_prefill_window(&at.a, window, sinks, l.stream);
    });
  });
}

// q k_cache v_cache kv_len out window sinks page_table workspace scale lse dev_error stream
PyObject *decode_window(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(o, n, 13, [&] {
    const Tensor &q = tensor(o[0], "q"), &k = tensor(o[1], "k_cache"), &v = tensor(o[2], "v_cache"),
                 &len = tensor(o[3], "kv_len"), &out = tensor(o[4], "out"), &ws = tensor(o[8], "workspace");
    const Tensor *table = optional_tensor(o[7], "page_table"), *lse = optional_tensor(o[10], "lse"),
                 *err = optional_tensor(o[11], "dev_error");
    const int dev = device_of(q);
    together(dev, {{&k, "k_cache"}, {&v, "v_cache"}, {&len, "kv_len"}, {&out, "out"}, {table, "page_table"},
                   {&ws, "workspace"}, {lse, "lse"}, {err, "dev_error"}});
    const Attention at(q, k, v, out, &len, o[9], lse, err, table);
    const int32_t window = count(o[5]), sinks = count(o[6]);
    void *wp = ws.data_ptr();
    const size_t wn = ws.nbytes();
    const Launch l(dev, o[12]);
    return status_of([&] {
      return masked_gqa_attn_decode_window(&at.a, at.paged, window, sinks, wp, wn, l.stream);
    });
  });
}

// q k_cache v_cache k_new v_new kv_len out tree_bits tree_len window sinks page_table workspace scale lse
// dev_error stream
PyObject *decode_tree(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(o, n, 17, [&] {
    const Tensor &q = tensor(o[0], "q"), &k = tensor(o[1], "k_cache"), &v = tensor(o[2], "v_cache"),
                 &kn = tensor(o[3], "k_new"), &vn = tensor(o[4], "v_new"), &len = tensor(o[5], "kv_len"),
                 &out = tensor(o[6], "out"), &ws = tensor(o[12], "workspace");
    const Tensor *bits = optional_tensor(o[7], "tree_bits"), *live = optional_tensor(o[8], "tree_len"),
                 *table = optional_tensor(o[11], "page_table"), *lse = optional_tensor(o[14], "lse"),
                 *err = optional_tensor(o[15], "dev_error");
    const int dev = device_of(q);
    together(dev, {{&k, "k_cache"}, {&v, "v_cache"}, {&kn, "k_new"}, {&vn, "v_new"}, {&len, "kv_len"}, {&out, "out"},
                   {bits, "tree_bits"}, {live, "tree_len"}, {table, "page_table"}, {&ws, "workspace"}, {lse, "lse"},
                   {err, "dev_error"}});
    const Attention at(q, k, v, out, &len, o[13], lse, err, table);
    const int64_t B = q.size(0), T = q.size(2), W = (T + 31) / 32, shape[4] = {B, k.size(1), T, q.size(3)};
    if (kn.sizes() != at::IntArrayRef(shape, 4) || vn.sizes() != kn.sizes() || kn.scalar_type() != q.scalar_type() ||
        vn.scalar_type() != q.scalar_type() || kn.stride(3) != 1 || vn.stride(3) != 1)
      bad("k_new and v_new must have q's dtype, [B, Hkv, T, D] and a unit-stride head dim");
    mgqa_tree tree{};
    tree.k_new = kn.data_ptr();
    tree.v_new = vn.data_ptr();
    for (int t = 0; t < 3; ++t) {
      tree.k_stride[t] = kn.stride(t);
      tree.v_stride[t] = vn.stride(t);
    }
    if (bits) {
      if ((bits->scalar_type() != at::kInt && bits->scalar_type() != at::kUInt32) || bits->dim() != 3 ||
          bits->stride(2) != 1)
        bad("tree_bits must be 3-D int32/uint32 words, contiguous along drafts");
      const int64_t b0 = bits->size(0), t0 = bits->size(1);
      if ((b0 != 1 && b0 != B) || (t0 != 1 && t0 != T) || bits->size(2) < W)
        bad("tree_bits must be [B or 1, T or 1, >= " + std::to_string(W) + "] words");
      tree.bits = static_cast<const uint32_t *>(bits->data_ptr());
      tree.bits_stride_b = b0 > 1 ? bits->stride(0) : 0;
      tree.bits_stride_t = t0 > 1 ? bits->stride(1) : 0;
    }
    tree.len = ints(live, "tree_len", {B});
    const int32_t window = count(o[9]), sinks = count(o[10]);
    void *wp = ws.data_ptr();
    const size_t wn = ws.nbytes();
    const Launch l(dev, o[16]);
    return status_of([&] {
      return masked_gqa_attn_decode_tree(&at.a, at.paged, &tree, window, sinks, wp, wn, l.stream);
    });
  });
}

// k_cache v_cache k_new v_new kv_len kv_len_out index count page_table dev_error stream
PyObject *cache_append(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(o, n, 11, [&] {
    const Tensor &k = tensor(o[0], "k_cache"), &v = tensor(o[1], "v_cache"), &kn = tensor(o[2], "k_new"),
                 &vn = tensor(o[3], "v_new"), &len = tensor(o[4], "kv_len"), &len_out = tensor(o[5], "kv_len_out");
    const Tensor *index = optional_tensor(o[6], "index"), *cnt = optional_tensor(o[7], "count"),
                 *table = optional_tensor(o[8], "page_table"), *err = optional_tensor(o[9], "dev_error");
    const int dev = device_of(k);
    together(dev, {{&v, "v_cache"}, {&kn, "k_new"}, {&vn, "v_new"}, {&len, "kv_len"}, {&len_out, "kv_len_out"},
                   {index, "index"}, {cnt, "count"}, {table, "page_table"}, {err, "dev_error"}});
    const Cache cache(k, v, table, &len, nullptr, err);
    const int x = (int)k.dim() - 4;
    bool fits = kn.dim() == k.dim() && vn.sizes() == kn.sizes() && kn.scalar_type() == k.scalar_type() &&
                vn.scalar_type() == k.scalar_type() && kn.stride(x + 3) == 1 && vn.stride(x + 3) == 1;
    fits = fits && (!x || kn.size(0) == cache.layers) && kn.size(x) == cache.rows && kn.size(x + 1) == cache.Hkv &&
           kn.size(x + 3) == cache.D;
    if (!fits)
      bad("k_new and v_new must have the caches' dtype, [layers, B, Hkv, T, D] (4-D with 4-D caches) and a "
          "unit-stride head dim");
    const int64_t T = kn.size(x + 2);
    int64_t ks[4] = {0}, vs[4] = {0};
    for (int t = x ? 0 : 1; t < 4; ++t) {
      ks[t] = kn.stride(x - 1 + t);
      vs[t] = vn.stride(x - 1 + t);
    }
    const int32_t *ip = ints(index, "index", {cache.rows, T}), *cp = ints(cnt, "count", {cache.rows});
    int32_t *lp = ints(&len_out, "kv_len_out", {cache.rows});
    const void *kp = kn.data_ptr(), *vp = vn.data_ptr();
    const int32_t rows = small(T, "T");
    const Launch l(dev, o[10]);
    return status_of([&] {
      return masked_gqa_cache_append(&cache.c, kp, vp, ks, vs, rows, ip, cp, lp, l.stream);
    });
  });
}

// k_cache v_cache page_table ref n
PyObject *cache_workspace_size(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(o, n, 5, [&] {
    const Cache cache(tensor(o[0], "k_cache"), tensor(o[1], "v_cache"), optional_tensor(o[2], "page_table"), nullptr,
                      optional_tensor(o[3], "ref"), nullptr);
    return PyLong_FromSize_t(masked_gqa_cache_workspace_size(&cache.c, count(o[4])));
  });
}

// k_cache v_cache page_table kv_len ref src dst extra workspace dev_error stream
PyObject *cache_fork(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(o, n, 11, [&] {
    const Tensor &k = tensor(o[0], "k_cache"), &v = tensor(o[1], "v_cache"), &table = tensor(o[2], "page_table"),
                 &len = tensor(o[3], "kv_len"), &ref = tensor(o[4], "ref"), &src = tensor(o[5], "src"),
                 &dst = tensor(o[6], "dst"), &ws = tensor(o[8], "workspace");
    const Tensor *err = optional_tensor(o[9], "dev_error");
    const int dev = device_of(k);
    together(dev, {{&v, "v_cache"}, {&table, "page_table"}, {&len, "kv_len"}, {&ref, "ref"}, {&src, "src"},
                   {&dst, "dst"}, {&ws, "workspace"}, {err, "dev_error"}});
    const int64_t pairs = src.numel();
    const int32_t *sp = ints(&src, "src", {pairs}), *dp = ints(&dst, "dst", {pairs});
    const Cache cache(k, v, &table, &len, &ref, err);
    const int32_t extra = count(o[7]);
    void *wp = ws.data_ptr();
    const size_t wn = ws.nbytes();
    const int32_t np = small(pairs, "pairs");
    const Launch l(dev, o[10]);
    return status_of([&] {
      return masked_gqa_cache_fork(&cache.c, np, sp, dp, extra, wp, wn, l.stream);
    });
  });
}

// k_cache v_cache page_table ref page_table_out ref_out used_out workspace dev_error stream
PyObject *cache_compact(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(o, n, 10, [&] {
    const Tensor &k = tensor(o[0], "k_cache"), &v = tensor(o[1], "v_cache"), &table = tensor(o[2], "page_table"),
                 &ref = tensor(o[3], "ref"), &to = tensor(o[4], "page_table_out"), &ref_out = tensor(o[5], "ref_out"),
                 &ws = tensor(o[7], "workspace");
    const Tensor *used = optional_tensor(o[6], "used_out"), *err = optional_tensor(o[8], "dev_error");
    const int dev = device_of(k);
    together(dev, {{&v, "v_cache"}, {&table, "page_table"}, {&ref, "ref"}, {&to, "page_table_out"},
                   {&ref_out, "ref_out"}, {used, "used_out"}, {&ws, "workspace"}, {err, "dev_error"}});
    const Cache cache(k, v, &table, nullptr, &ref, err);
    if (to.scalar_type() != at::kInt || to.sizes() != table.sizes() || to.stride(1) != 1)
      bad("page_table_out must be int32 of page_table's shape with unit-stride rows");
    int32_t *rp = ints(&ref_out, "ref_out", {ref.numel()}), *up = ints(used, "used_out", {1});
    int32_t *tp = static_cast<int32_t *>(to.data_ptr());
    const int64_t stride = to.stride(0);
    void *wp = ws.data_ptr();
    const size_t wn = ws.nbytes();
    const Launch l(dev, o[9]);
    return status_of([&] {
      return masked_gqa_cache_compact(&cache.c, tp, stride, rp, up, wp, wn, l.stream);
    });
  });
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(prefill_window), FAST(decode_window), FAST(decode_tree), FAST(cache_append),
                         FAST(cache_workspace_size), FAST(cache_fork), FAST(cache_compact),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mgqa_bind", nullptr, -1, methods};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__mgqa_bind() { return PyModule_Create(&module); }
