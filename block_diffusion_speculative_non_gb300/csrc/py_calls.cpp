// py_calls.cpp — Python calls of the operators on a context store, as a module of CPython's own C interface.
//
// These operators take 3 to 10 us on the GPU for short contexts, and ctypes with the checks of ten tensors in Python took 6 to
// 8 us of the host for each call, more than its launches (3 to 4 us).  Here the arguments go straight from the tensors to
// the library's entry points.  The entry points are handed in by address, so that the module serves either build of the library.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <exception>
#include <initializer_list>

#include "fpd.h"

namespace {

struct Entries {
  decltype(&fpd_shared_attention) shared_attention;
  decltype(&fpd_context_weights) context_weights;
  decltype(&fpd_evict_context) evict_context;
} g_entries;

int64_t product(std::initializer_list<int64_t> f) {   // as large as it gets where 64 bits do not hold it
  int64_t r = 1;
  for (int64_t v : f)
    if (__builtin_mul_overflow(r, v, &r)) return INT64_MAX;
  return r;
}

// Device address of a tensor that must be contiguous, of the given type, on device `dev` and hold at least n elements; an int
// address or None is passed on.  False with the Python error set.
bool address(PyObject* o, at::ScalarType type, int64_t n, const char* what, int dev, void** out) {
  *out = nullptr;
  if (o == Py_None) return true;
  if (PyLong_CheckExact(o)) {
    *out = reinterpret_cast<void*>(static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(o)));
    return !PyErr_Occurred();
  }
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor, an address or None, got %s", what, Py_TYPE(o)->tp_name);
    return false;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != type) {
    PyObject* got = PyObject_GetAttrString(o, "dtype");
    if (got) PyErr_Format(PyExc_ValueError, "%s must be %S, got %S", what, (PyObject*)torch::getTHPDtype(type), got);
    Py_XDECREF(got);
  } else if (!t.is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous (row-major)", what);
  } else if (t.numel() < n) {
    PyErr_Format(PyExc_ValueError, "%s holds %lld elements, the call needs %lld", what, (long long)t.numel(), (long long)n);
  } else if (dev < 0 || t.get_device() != dev) {
    PyErr_Format(PyExc_ValueError, "%s is on %s, the current device is cuda:%d", what, t.device().str().c_str(), dev);
  } else {
    *out = const_cast<void*>(t.const_data_ptr());
    return true;
  }
  return false;
}

// The arguments of a call, read in turn; after a failure the rest reads as zero and the Python error stands.
struct Reader {
  PyObject* const* a;
  Py_ssize_t n, k = 0;
  int dev = 0;
  bool ok = true;
  Reader(PyObject* const* args, Py_ssize_t nargs, Py_ssize_t want) : a(args), n(nargs) {
    if (nargs != want) {
      PyErr_Format(PyExc_TypeError, "%zd arguments, the call takes %zd", nargs, want);
      ok = false;
    } else if (!g_entries.shared_attention) {
      PyErr_SetString(PyExc_RuntimeError, "the library's entry points are not bound");
      ok = false;
    } else {
      k = want - 1;   // the current device comes last
      dev = i();
      k = 0;
    }
  }
  int i() {
    if (!ok) return 0;
    const long v = PyLong_AsLong(a[k++]);
    if (v == -1 && PyErr_Occurred()) ok = false;
    else if (v < INT_MIN || v > INT_MAX) {
      PyErr_Format(PyExc_OverflowError, "argument %zd does not fit 32 bits", k);
      ok = false;
    }
    return ok ? (int)v : 0;
  }
  size_t size() {
    if (!ok) return 0;
    const size_t v = PyLong_AsSize_t(a[k++]);
    if (PyErr_Occurred()) ok = false;
    return ok ? v : 0;
  }
  void* stream() {
    if (!ok) return nullptr;
    void* v = a[k] == Py_None ? nullptr : PyLong_AsVoidPtr(a[k]);
    k++;
    if (PyErr_Occurred()) ok = false;
    return v;
  }
  void* at(at::ScalarType type, std::initializer_list<int64_t> n, const char* what) {
    void* v = nullptr;
    if (ok) ok = address(a[k++], type, product(n), what, dev, &v);
    return v;
  }
};

constexpr auto kBf16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt, kU8 = at::kByte;

// f's status as a Python int; no C++ exception leaves the module.
template <class F>
PyObject* call(F f) {
  try {
    return f();
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}
template <class F>
PyObject* run(const Reader& r, F f) {
  if (!r.ok) return nullptr;
  int s;
  Py_BEGIN_ALLOW_THREADS   // as ctypes does
  s = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(s);
}

PyObject* shared_attention(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return call([&]() -> PyObject* {
    Reader r(args, nargs, 21);
    const int batch = r.i(), L = r.i(), nq = r.i(), nkv = r.i(), h = r.i(), layer = r.i();
    const int64_t layers = (int64_t)layer + 1;
    const void* q = r.at(kBf16, {batch, L, nq, h}, "q");
    const void* k_blk = r.at(kBf16, {batch, nkv, L, h}, "k_blk");
    const void* v_blk = r.at(kBf16, {batch, nkv, L, h}, "v_blk");
    PyObject* prefix = r.ok ? args[r.k++] : nullptr;   // its size follows it
    const int p_cap = r.i();
    void* prefix_store = nullptr;
    if (r.ok) r.ok = address(prefix, kBf16, product({layers, p_cap, 2, nkv, h}), "prefix_store", r.dev, &prefix_store);
    const int32_t* prefix_len = (const int32_t*)r.at(kI32, {1}, "prefix_len");
    PyObject* store = r.ok ? args[r.k++] : nullptr;
    const int t_cap = r.i();
    void* kv_store = nullptr;
    if (r.ok) r.ok = address(store, kBf16, product({layers, batch, t_cap, 2, nkv, h}), "kv_store", r.dev, &kv_store);
    const int32_t* ctx_len = (const int32_t*)r.at(kI32, {batch}, "ctx_len");
    void* out = r.at(kBf16, {batch, L, nq, h}, "out");
    float* lse = (float*)r.at(kF32, {batch, L, nq}, "lse");
    PyObject* work = r.ok ? args[r.k++] : nullptr;
    const size_t bytes = r.size();
    void* ws = nullptr;
    if (r.ok) r.ok = address(work, kU8, (int64_t)std::min<size_t>(bytes, INT64_MAX), "workspace", r.dev, &ws);
    void* st = r.stream();
    return run(r, [&] {
      return (int)g_entries.shared_attention(batch, L, nq, nkv, h, layer, q, k_blk, v_blk, prefix_store, p_cap, prefix_len,
                                             kv_store, t_cap, ctx_len, out, lse, ws, bytes, st);
    });
  });
}

PyObject* context_weights(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return call([&]() -> PyObject* {
    Reader r(args, nargs, 15);
    const int batch = r.i(), L = r.i(), nq = r.i(), nkv = r.i(), h = r.i(), layer = r.i();
    const int64_t layers = (int64_t)layer + 1;
    const void* q = r.at(kBf16, {batch, L, nq, h}, "q");
    const float* lse = (const float*)r.at(kF32, {batch, L, nq}, "lse");
    PyObject* store = r.ok ? args[r.k++] : nullptr;
    const int t_cap = r.i();
    void* kv_store = nullptr;
    if (r.ok) r.ok = address(store, kBf16, product({layers, batch, nkv, t_cap, 2, h}), "kv_store", r.dev, &kv_store);
    const int32_t* ctx_len = (const int32_t*)r.at(kI32, {batch}, "ctx_len");
    float* weights = (float*)r.at(kF32, {layers, batch, nkv, t_cap}, "weights");
    const int accumulate = r.i();
    void* st = r.stream();
    return run(r, [&] {
      return (int)g_entries.context_weights(batch, L, nq, nkv, h, layer, q, lse, kv_store, t_cap, ctx_len, weights, accumulate,
                                            st);
    });
  });
}

PyObject* evict_context(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return call([&]() -> PyObject* {
    Reader r(args, nargs, 20);
    const int layers = r.i(), batch = r.i(), nkv = r.i(), h = r.i(), budget = r.i(), recent = r.i();
    PyObject* store = r.ok ? args[r.k++] : nullptr;
    const int t_cap = r.i();
    void* kv_store = nullptr;
    if (r.ok) r.ok = address(store, kBf16, product({layers, batch, nkv, 2, t_cap, h}), "kv_store", r.dev, &kv_store);
    const float* weights = (const float*)r.at(kF32, {layers, batch, nkv, t_cap}, "weights");
    const int32_t* ctx_len = (const int32_t*)r.at(kI32, {batch}, "ctx_len");
    PyObject* to = r.ok ? args[r.k++] : nullptr;
    const int out_cap = r.i();
    void* out_store = nullptr;
    if (r.ok) r.ok = address(to, kBf16, product({layers, batch, nkv, 2, out_cap, h}), "out_store", r.dev, &out_store);
    float* out_weights = (float*)r.at(kF32, {layers, batch, nkv, out_cap}, "out_weights");
    int32_t* out_len = (int32_t*)r.at(kI32, {batch}, "out_len");
    int32_t* pos_offset = (int32_t*)r.at(kI32, {batch}, "pos_offset");
    int32_t* kept = (int32_t*)r.at(kI32, {layers, batch, nkv, budget}, "kept");
    PyObject* work = r.ok ? args[r.k++] : nullptr;
    const size_t bytes = r.size();
    void* ws = nullptr;
    if (r.ok) r.ok = address(work, kU8, (int64_t)std::min<size_t>(bytes, INT64_MAX), "workspace", r.dev, &ws);
    void* st = r.stream();
    return run(r, [&] {
      return (int)g_entries.evict_context(layers, batch, nkv, h, budget, recent, kv_store, t_cap, weights, ctx_len, out_store,
                                          out_cap, out_weights, out_len, pos_offset, kept, ws, bytes, st);
    });
  });
}

// arg(tensor, dtype, n, what, device): the check alone
PyObject* arg(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return call([&]() -> PyObject* {
    if (nargs != 5 || !THPDtype_Check(a[1])) {
      PyErr_SetString(PyExc_TypeError, "arg(tensor, dtype, n, what, device)");
      return nullptr;
    }
    const long long n = PyLong_AsLongLong(a[2]);
    const char* what = PyUnicode_AsUTF8(a[3]);
    const long dev = PyLong_AsLong(a[4]);
    void* p = nullptr;
    if (PyErr_Occurred() || !address(a[0], ((THPDtype*)a[1])->scalar_type, n, what, (int)dev, &p)) return nullptr;
    if (!p) Py_RETURN_NONE;
    return PyLong_FromVoidPtr(p);
  });
}

// bind(shared_attention, context_weights, evict_context): addresses of the entry points
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (nargs != 3) {
    PyErr_SetString(PyExc_TypeError, "bind takes three addresses");
    return nullptr;
  }
  g_entries = {(decltype(&fpd_shared_attention))PyLong_AsVoidPtr(a[0]), (decltype(&fpd_context_weights))PyLong_AsVoidPtr(a[1]),
               (decltype(&fpd_evict_context))PyLong_AsVoidPtr(a[2])};
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {{"shared_attention", (PyCFunction)(void (*)(void))shared_attention, METH_FASTCALL, nullptr},
                           {"context_weights", (PyCFunction)(void (*)(void))context_weights, METH_FASTCALL, nullptr},
                           {"evict_context", (PyCFunction)(void (*)(void))evict_context, METH_FASTCALL, nullptr},
                           {"arg", (PyCFunction)(void (*)(void))arg, METH_FASTCALL, nullptr},
                           {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&g_module);
  if (m && PyModule_AddStringConstant(m, "torch_version", FPD_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
