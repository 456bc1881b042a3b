// paged_binding.cpp -- argument checks of the paged cache's Python calls.
//
// A decode step makes these calls once per layer on tensors that a kernel is
// done with in a few microseconds, so the checks read the tensors' properties
// directly (about 0.3 us a call; through the interpreter they cost 4 us, more
// than the launch).  Like the ctypes part of the binding it marshals only:
// every call ends in the C ABI's function of the same name.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <new>
#include <string>

#include "wave_index.h"

namespace {

constexpr int64_t kD = 128;

// What the checks need to know of a handle.
struct Context {
  wi_paged* handle;
  int device;
  int64_t hq, hkv, page, n_pages, max_pages;
};

void drop(PyObject* capsule) { delete static_cast<Context*>(PyCapsule_GetPointer(capsule, "wi_paged")); }

enum Kind { kBf16, kInt32, kFp32 };
const char* const kKindName[] = {"torch.bfloat16 (or int16)", "torch.int32", "torch.float32"};

bool is_kind(const at::Tensor& t, Kind k) {
  const at::ScalarType s = t.scalar_type();
  return k == kBf16 ? s == at::kBFloat16 || s == at::kShort : s == (k == kInt32 ? at::kInt : at::kFloat);
}

std::string text(at::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + ")";
}

std::string text(const at::Tensor& t) {
  return std::string(c10::toString(t.scalar_type())) + " " + text(t.sizes()) + " on " + t.device().str() + ", strides " +
         text(t.strides());
}

// Reads one call's arguments; the first that is not what it has to be sets a ValueError and `ok` to false.
struct Reader {
  const Context* c;
  bool ok = true;

  void fail(const std::string& s) {
    if (ok) PyErr_SetString(PyExc_ValueError, s.c_str());
    ok = false;
  }
  const at::Tensor* tensor(const char* name, PyObject* o) {
    if (!ok) return nullptr;
    if (!THPVariable_Check(o)) {
      fail(std::string(name) + " must be a tensor");
      return nullptr;
    }
    return &THPVariable_Unpack(o);
  }
  int64_t size0(const char* name, PyObject* o) {
    const at::Tensor* t = tensor(name, o);
    if (!t) return 0;
    if (t->dim() < 1) fail(std::string(name) + " must have a dimension");
    return ok ? t->size(0) : 0;
  }
  // Data of a contiguous tensor of this device, type and shape; null for None where that is allowed.
  void* data(const char* name, PyObject* o, Kind k, at::IntArrayRef shape, bool may_be_none = false) {
    if (may_be_none && o == Py_None) return nullptr;
    const at::Tensor* t = tensor(name, o);
    if (!t) return nullptr;
    if (!is_kind(*t, k) || t->sizes() != shape || !t->is_contiguous() || !t->is_cuda() || t->get_device() != c->device) {
      fail(std::string(name) + " must be a contiguous " + kKindName[k] + " tensor of shape " + text(shape) + " on cuda:" +
           std::to_string(c->device) + " (got " + text(*t) + ")");
      return nullptr;
    }
    return t->data_ptr();
  }
  // ... of [n][heads][128] with contiguous heads, and the distance of its tokens.
  void* heads(const char* name, PyObject* o, int64_t n, int64_t heads, long long* stride) {
    const at::Tensor* t = tensor(name, o);
    *stride = 0;
    if (!t) return nullptr;
    if (!is_kind(*t, kBf16) || t->sizes() != at::IntArrayRef({n, heads, kD}) || t->stride(2) != 1 ||
        (heads > 1 && t->stride(1) != kD) || !t->is_cuda() || t->get_device() != c->device) {
      fail(std::string(name) + " must be a " + kKindName[kBf16] + " tensor " + text({n, heads, kD}) +
           " with contiguous heads on cuda:" + std::to_string(c->device) + " (got " + text(*t) + ")");
      return nullptr;
    }
    *stride = t->stride(0);
    return t->data_ptr();
  }
  int32_t* table(PyObject* o, int64_t batch) {
    const int64_t rows = size0("block_table", o);
    if (ok && rows < batch) fail("block_table must have a row for each of the " + std::to_string(batch) + " requests");
    return static_cast<int32_t*>(data("block_table", o, kInt32, {rows, c->max_pages}));
  }
  // Sizes that the C ABI takes as int.
  void fits(const char* what, int64_t n) {
    if (n > INT32_MAX) fail(std::string(what) + " must be below 2^31 (got " + std::to_string(n) + ")");
  }
  int32_t* ints(const char* name, PyObject* o, int64_t n) { return static_cast<int32_t*>(data(name, o, kInt32, {n})); }
};

void* stream_of(PyObject* o, Reader& r) {
  void* s = PyLong_AsVoidPtr(o);
  if (!s && PyErr_Occurred()) r.ok = false;
  return s;
}

// The call's context, or an exception for a wrong number of arguments or a handle that has been freed.
const Context* begin(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments wanted, %zd given", want, n);
    return nullptr;
  }
  if (!PyCapsule_IsValid(a[0], "wi_paged")) {
    PyErr_SetString(PyExc_ValueError, "the paged cache has been freed");
    return nullptr;
  }
  return static_cast<const Context*>(PyCapsule_GetPointer(a[0], "wi_paged"));
}

// Every entry: tensor accesses may throw (a tensor without storage, say), and nothing may leave through C.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

PyObject* context(PyObject*, PyObject* args) {
  unsigned long long handle;
  Context c{};
  long long hq, hkv, page, n_pages, max_pages;
  if (!PyArg_ParseTuple(args, "KiLLLLL", &handle, &c.device, &hq, &hkv, &page, &n_pages, &max_pages)) return nullptr;
  c.handle = reinterpret_cast<wi_paged*>(static_cast<uintptr_t>(handle));
  c.hq = hq, c.hkv = hkv, c.page = page, c.n_pages = n_pages, c.max_pages = max_pages;
  Context* p = new (std::nothrow) Context(c);
  if (!p) return PyErr_NoMemory();
  PyObject* o = PyCapsule_New(p, "wi_paged", drop);
  if (!o) delete p;
  return o;
}

// (ctx, ctx_len, new_len, free_pages, n_free, block_table, kv_len, q_start, slots, positions, n_free_out, stream)
PyObject* tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Context* c = begin(a, n, 12);
    if (!c) return nullptr;
    Reader r{c};
    const int64_t b = r.size0("ctx_len", a[1]), cap = r.size0("free_pages", a[3]), t = r.size0("slots", a[8]);
    const int32_t *ctx = r.ints("ctx_len", a[1], b), *fresh = r.ints("new_len", a[2], b),
                  *pages = r.ints("free_pages", a[3], cap), *left = r.ints("n_free", a[4], 1);
    int32_t *table = r.table(a[5], b), *kv = r.ints("kv_len", a[6], b), *start = r.ints("q_start", a[7], b + 1),
            *slots = r.ints("slots", a[8], t), *pos = r.ints("positions", a[9], t), *out = r.ints("n_free_out", a[10], 1);
    void* stream = stream_of(a[11], r);
    r.fits("the requests", b), r.fits("the free pages", cap), r.fits("the tokens", t);
    if (!r.ok) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS rc = wi_paged_tables(c->handle, (int)b, ctx, fresh, pages, left, (int)cap, table, kv, start,
                                                slots, pos, (int)t, out, stream);
    Py_END_ALLOW_THREADS return PyLong_FromLong(rc);
  });
}

// (ctx, q, k, v, positions, slots, k_pages, v_pages, q_out, q_weight, k_weight, stream)
PyObject* write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Context* c = begin(a, n, 12);
    if (!c) return nullptr;
    Reader r{c};
    const int64_t t = r.size0("q", a[1]);
    long long qs, ks, vs;
    const void *q = r.heads("q", a[1], t, c->hq, &qs), *k = r.heads("k", a[2], t, c->hkv, &ks),
               *v = r.heads("v", a[3], t, c->hkv, &vs);
    const int32_t* pos = r.ints("positions", a[4], t);
    const bool pool = a[5] != Py_None;
    const int32_t* slots = pool ? r.ints("slots", a[5], t) : nullptr;
    const int64_t p4[] = {c->n_pages, c->hkv, c->page, kD}, p3[] = {t, c->hkv, kD};
    const at::IntArrayRef shape = pool ? at::IntArrayRef(p4, 4) : at::IntArrayRef(p3, 3);
    void *kp = r.data("k_pages", a[6], kBf16, shape), *vp = r.data("v_pages", a[7], kBf16, shape),
         *qo = r.data("q_out", a[8], kBf16, {t, c->hq, kD});
    const void *wq = r.data("q_weight", a[9], kBf16, {kD}, true), *wk = r.data("k_weight", a[10], kBf16, {kD}, true);
    void* stream = stream_of(a[11], r);
    r.fits("the tokens", t);
    if (!r.ok) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS rc =
        wi_paged_write(c->handle, (int)t, q, qs, k, ks, v, vs, wq, wk, pos, slots, qo, kp, vp, stream);
    Py_END_ALLOW_THREADS return PyLong_FromLong(rc);
  });
}

// (ctx, q, k_pages, v_pages, block_table, q_start, kv_len, out, lse, stream)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Context* c = begin(a, n, 10);
    if (!c) return nullptr;
    Reader r{c};
    const int64_t t = r.size0("q", a[1]), b = r.size0("kv_len", a[6]);
    const void *q = r.data("q", a[1], kBf16, {t, c->hq, kD}),
               *kp = r.data("k_pages", a[2], kBf16, {c->n_pages, c->hkv, c->page, kD}),
               *vp = r.data("v_pages", a[3], kBf16, {c->n_pages, c->hkv, c->page, kD});
    const int32_t *table = r.table(a[4], b), *start = r.ints("q_start", a[5], b + 1), *kv = r.ints("kv_len", a[6], b);
    void* out = r.data("out", a[7], kBf16, {t, c->hq, kD});
    float* lse = static_cast<float*>(r.data("lse", a[8], kFp32, {t, c->hq}, true));
    void* stream = stream_of(a[9], r);
    r.fits("the tokens", t), r.fits("the requests", b);
    if (!r.ok) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS rc =
        wi_paged_attention(c->handle, (int)b, (int)t, q, kp, vp, table, start, kv, out, lse, stream);
    Py_END_ALLOW_THREADS return PyLong_FromLong(rc);
  });
}

// (ctx, k_pages, v_pages, block_table, kv_len, pos0, k_out, v_out, stream)
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Context* c = begin(a, n, 9);
    if (!c) return nullptr;
    Reader r{c};
    const int64_t b = r.size0("kv_len", a[4]);
    const at::Tensor* o = r.tensor("k_out", a[6]);
    if (r.ok && o->dim() != 5) r.fail("k_out must have shape [batch][layers][n_kv_heads][n][128]");
    if (!r.ok) return nullptr;
    const int64_t layers = o->size(1), rows = o->size(3);
    const at::Tensor* pk = r.tensor("k_pages", a[1]);
    const int64_t p5[] = {layers, c->n_pages, c->hkv, c->page, kD};
    // one pool may come without the layers' dimension
    const at::IntArrayRef pool = r.ok && layers == 1 && pk->dim() == 4 ? at::IntArrayRef(p5 + 1, 4) : at::IntArrayRef(p5, 5);
    const void *kp = r.data("k_pages", a[1], kBf16, pool), *vp = r.data("v_pages", a[2], kBf16, pool);
    const int32_t *table = r.table(a[3], b), *kv = r.ints("kv_len", a[4], b);
    const long long pos0 = r.ok ? PyLong_AsLongLong(a[5]) : 0;
    if (r.ok && pos0 == -1 && PyErr_Occurred()) r.ok = false;
    void *ko = r.data("k_out", a[6], kBf16, {b, layers, c->hkv, rows, kD}),
         *vo = r.data("v_out", a[7], kBf16, {b, layers, c->hkv, rows, kD});
    void* stream = stream_of(a[8], r);
    r.fits("the requests", b), r.fits("the layers", layers);
    if (!r.ok) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS rc =
        wi_paged_gather(c->handle, (int)b, (int)layers, kp, vp, table, kv, pos0, rows, ko, vo, stream);
    Py_END_ALLOW_THREADS return PyLong_FromLong(rc);
  });
}

#define WI_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f))
PyMethodDef kMethods[] = {
    {"context", context, METH_VARARGS, "(handle, device, n_q_heads, n_kv_heads, page_size, n_pages, max_pages)"},
    {"tables", WI_FAST(tables), METH_FASTCALL, "wi_paged_tables; returns its status"},
    {"write", WI_FAST(write), METH_FASTCALL, "wi_paged_write; returns its status"},
    {"attention", WI_FAST(attention), METH_FASTCALL, "wi_paged_attention; returns its status"},
    {"gather", WI_FAST(gather), METH_FASTCALL, "wi_paged_gather; returns its status"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_paged", "Argument checks of the paged cache's calls.", -1, kMethods,
                       nullptr,               nullptr,  nullptr,                                        nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged(void) { return PyModule_Create(&kModule); }
