// The binding's argument marshalling for the calls that a decode step makes several times in
// every layer: torch tensors checked (device, dtype, layout, size) and turned into addresses
// here instead of in Python, where that takes longer than the kernels (plan 8.6 -> 4.2 us a
// call on an MI355X's host). The C functions are those that the ctypes binding has loaded;
// their addresses are handed over at import. Every function returns the call's status, or
// raises TypeError or ValueError for a tensor that does not fit, as the other bindings do.

#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <exception>
#include <string>

#include "sparse_ffn.h"

namespace {

decltype(&kv_cache_plan) f_plan;
decltype(&kv_cache_append) f_append;
decltype(&kv_cache_attend) f_attend;
decltype(&residual_norm) f_norm;

constexpr at::ScalarType kAny = at::ScalarType::Undefined;

bool fail(PyObject* kind, const std::string& what) {
  PyErr_SetString(kind, what.c_str());
  return false;
}

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    fail(PyExc_TypeError, std::string(name) + " must be a torch tensor or None");
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.is_cuda()) return &t;
  fail(PyExc_ValueError, std::string(name) + " must be a GPU tensor (got " + t.device().str() + ")");
  return nullptr;
}

bool right_type(const at::Tensor& t, const char* name, at::ScalarType dtype) {
  return dtype == kAny || t.scalar_type() == dtype ||
         fail(PyExc_ValueError, std::string(name) + " must be " + at::toString(dtype) + " (got " + at::toString(t.scalar_type()) + ")");
}

// The address of a contiguous tensor of at least `numel` values (None: null).
bool address(PyObject* o, const char* name, at::ScalarType dtype, int64_t numel, void** out) {
  *out = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  if (!t->is_contiguous()) return fail(PyExc_ValueError, std::string(name) + " must be contiguous");
  if (!right_type(*t, name, dtype)) return false;
  if (t->numel() < numel)
    return fail(PyExc_ValueError, std::string(name) + " holds " + std::to_string(t->numel()) + " elements, needs " + std::to_string(numel));
  *out = t->data_ptr();
  return true;
}
bool ints(PyObject* o, const char* name, int64_t numel, void** out) { return address(o, name, at::kInt, numel, out); }

// Tokens' heads [T, heads, dh], perhaps parts of wider rows: address and token stride. T < 0
// and heads < 0 are taken from the tensor, otherwise they have to be its.
bool token_rows(PyObject* o, const char* name, at::ScalarType dtype, int64_t* T, int64_t* heads, int64_t dh, void** out, int64_t* stride) {
  const at::Tensor* t = tensor(o, name);
  if (!t || !right_type(*t, name, dtype)) return false;
  if (t->dim() != 3 || t->size(2) != dh || (*heads >= 0 && t->size(1) != *heads) || (*T >= 0 && t->size(0) != *T))
    return fail(PyExc_ValueError, std::string(name) + " must be [" + (*T < 0 ? "T" : std::to_string(*T)) + ", " +
                                      (*heads < 0 ? "heads" : std::to_string(*heads)) + ", " + std::to_string(dh) + "]");
  *T = t->size(0);
  *heads = t->size(1);
  if (t->stride(2) != 1 || (t->stride(1) != dh && *heads > 1))
    return fail(PyExc_ValueError, std::string(name) + ": the heads of a token must lie one after the other");
  *out = t->data_ptr();
  *stride = *T > 1 ? t->stride(0) : *heads * dh;
  return true;
}

bool count(Py_ssize_t n, Py_ssize_t want) {
  return n == want || fail(PyExc_TypeError, "expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
}
void* pointer(PyObject* o) { return PyLong_AsVoidPtr(o); }
bool fits(int64_t v, const char* name) { return v <= INT32_MAX || fail(PyExc_ValueError, std::string(name) + " is too large"); }
PyObject* status(int st) { return PyErr_Occurred() ? nullptr : PyLong_FromLong(st); }

// The status of a library call, during which other Python threads may run (a launch can wait
// for room in the queue). The caller's arguments keep the tensors and the structure alive. No
// exception comes out of the library's functions.
template <class Call>
PyObject* status_of(Call call) {
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = call();
  Py_END_ALLOW_THREADS
  return status(st);
}

at::ScalarType cache_type(const sfn_kv* kv) { return kv->dtype == SFN_BF16 ? at::kBFloat16 : at::kFloat; }
at::ScalarType weight_type(const sfn_norm* n) { return n->wdtype == SFN_BF16 ? at::kBFloat16 : at::kFloat; }

// (plan, append, attend, norm): the addresses of the library's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 4)) return nullptr;
  f_plan = reinterpret_cast<decltype(f_plan)>(pointer(a[0]));
  f_append = reinterpret_cast<decltype(f_append)>(pointer(a[1]));
  f_attend = reinterpret_cast<decltype(f_attend)>(pointer(a[2]));
  f_norm = reinterpret_cast<decltype(f_norm)>(pointer(a[3]));
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

// (sfn_kv address, held_len, ctx_len, new_len, table, free_pages, n_free, n_free_out, cu,
// kv_len, pos, slot, status, stream)
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 14)) return nullptr;
  const sfn_kv* kv = static_cast<const sfn_kv*>(pointer(a[0]));
  void* p[13];
  if (!kv) return status(SFN_EINVAL);
  if (!ints(a[1], "held_len", 0, &p[1]) || !ints(a[4], "table", 0, &p[4]) || !ints(a[11], "slot", 0, &p[11])) return nullptr;
  const int64_t R = p[1] ? THPVariable_Unpack(a[1]).numel() : 0, T = p[11] ? THPVariable_Unpack(a[11]).numel() : 0;
  int64_t cols = 0;
  if (p[4]) {
    const at::Tensor& t = THPVariable_Unpack(a[4]);
    if (t.dim() != 2 || t.size(0) != R) {
      fail(PyExc_ValueError, "table must be [" + std::to_string(R) + ", max_pages]");
      return nullptr;
    }
    cols = t.size(1);
  }
  if (!ints(a[2], "ctx_len", R, &p[2]) || !ints(a[3], "new_len", R, &p[3]) || !ints(a[5], "free_pages", kv->n_pages, &p[5]) ||
      !ints(a[6], "n_free", 1, &p[6]) || !ints(a[7], "n_free_out", 1, &p[7]) || !ints(a[8], "cu", R + 1, &p[8]) ||
      !ints(a[9], "kv_len", R, &p[9]) || !ints(a[10], "pos", T, &p[10]) || !ints(a[12], "status", 1, &p[12]))
    return nullptr;
  if (!fits(R, "R") || !fits(cols, "max_pages") || !fits(T, "the number of slots")) return nullptr;
  void* stream = pointer(a[13]);
  if (PyErr_Occurred()) return nullptr;
  auto i = [&](int k) { return static_cast<int32_t*>(p[k]); };
  return status_of([&] {
    return f_plan(kv, (int32_t)R, (int32_t)cols, (int32_t)T, i(1), i(2), i(3), i(4), i(5), i(6), i(7), i(8), i(9), i(10), i(11), i(12),
                  stream);
  });
}

// (sfn_kv address, k, v, slot, q, q_out, pos, rope, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  const sfn_kv* kv = static_cast<const sfn_kv*>(pointer(a[0]));
  if (!kv) return status(SFN_EINVAL);
  const at::ScalarType dt = cache_type(kv);
  void *k, *v, *q = nullptr, *slot, *q_out, *pos, *rope;
  int64_t T = -1, ks, vs, qs = 0, h_kv = kv->h_kv, h_q = -1, n_pos = 0, rot = 0;
  if (!token_rows(a[1], "k", dt, &T, &h_kv, kv->dh, &k, &ks) || !token_rows(a[2], "v", dt, &T, &h_kv, kv->dh, &v, &vs)) return nullptr;
  if (a[4] == Py_None) h_q = 0;
  else if (!token_rows(a[4], "q", dt, &T, &h_q, kv->dh, &q, &qs)) return nullptr;
  if (!ints(a[3], "slot", T, &slot) || !address(a[5], "q_out", dt, T * h_q * kv->dh, &q_out) || !ints(a[6], "pos", T, &pos) ||
      !address(a[7], "rope", at::kFloat, 0, &rope))
    return nullptr;
  if (rope) {
    const at::Tensor& t = THPVariable_Unpack(a[7]);
    if (t.dim() != 2) {
      fail(PyExc_ValueError, "rope must be [n_pos, rot]");
      return nullptr;
    }
    n_pos = t.size(0);
    rot = t.size(1);
  }
  if (!fits(T, "T") || !fits(h_q, "h_q") || !fits(n_pos, "n_pos") || !fits(rot, "rot")) return nullptr;
  void* stream = pointer(a[8]);
  if (PyErr_Occurred()) return nullptr;
  return status_of([&] {
    return f_append(kv, (int32_t)T, (int32_t)h_q, q, qs, k, ks, v, vs, static_cast<int32_t*>(pos), static_cast<int32_t*>(slot),
                    static_cast<float*>(rope), (int32_t)n_pos, (int32_t)rot, q_out, stream);
  });
}

// (sfn_kv address, q, table, cu, kv_len, out, ws, max_new, max_len, scale, window, stream)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 12)) return nullptr;
  const sfn_kv* kv = static_cast<const sfn_kv*>(pointer(a[0]));
  if (!kv) return status(SFN_EINVAL);
  const at::ScalarType dt = cache_type(kv);
  void *q, *table, *cu, *kv_len, *out, *ws;
  int64_t T = -1, h_q = -1, qs, R = 0, cols = 0;
  if (!token_rows(a[1], "q", dt, &T, &h_q, kv->dh, &q, &qs) || !ints(a[2], "table", 0, &table)) return nullptr;
  if (table) {
    const at::Tensor& t = THPVariable_Unpack(a[2]);
    if (t.dim() != 2) {
      fail(PyExc_ValueError, "table must be [R, max_pages]");
      return nullptr;
    }
    R = t.size(0);
    cols = t.size(1);
  }
  if (!ints(a[3], "cu", R + 1, &cu) || !ints(a[4], "kv_len", R, &kv_len) || !address(a[5], "out", dt, T * h_q * kv->dh, &out) ||
      !address(a[6], "ws", kAny, 0, &ws))
    return nullptr;
  const size_t ws_bytes = ws ? THPVariable_Unpack(a[6]).nbytes() : 0;
  const long long max_new = PyLong_AsLongLong(a[7]), max_len = PyLong_AsLongLong(a[8]), window = PyLong_AsLongLong(a[10]);
  const double scale = PyFloat_AsDouble(a[9]);
  void* stream = pointer(a[11]);
  if (PyErr_Occurred()) return nullptr;
  if (!fits(T, "T") || !fits(h_q, "h_q") || !fits(R, "R") || !fits(cols, "max_pages") || !fits(max_new, "max_new") ||
      !fits(max_len, "max_len") || !fits(window, "window"))
    return nullptr;
  auto clamp = [](long long v) { return (int32_t)(v < -1 ? -1 : v); };
  return status_of([&] {
    return f_attend(kv, (int32_t)R, (int32_t)T, (int32_t)h_q, q, qs, static_cast<int32_t*>(table), (int32_t)cols,
                    static_cast<int32_t*>(cu), static_cast<int32_t*>(kv_len), clamp(max_new), clamp(max_len), (float)scale,
                    clamp(window), out, ws, ws_bytes, stream);
  });
}

// (sfn_norm address, h, y, h_out, x_out, gate, stream)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 7)) return nullptr;
  const sfn_norm* nm = static_cast<const sfn_norm*>(pointer(a[0]));
  if (!nm) return status(SFN_EINVAL);
  if (nm->d < 1) return status(SFN_ESHAPE);
  auto code = [](const at::Tensor& t) { return t.scalar_type() == at::kBFloat16 ? SFN_BF16 : t.scalar_type() == at::kFloat ? SFN_F32 : -1; };
  void *h, *y, *h_out, *x_out, *gate;
  if (!address(a[1], "h", kAny, 0, &h)) return nullptr;
  const at::Tensor* th = a[1] == Py_None ? nullptr : &THPVariable_Unpack(a[1]);
  const at::Tensor* ty = a[2] == Py_None ? nullptr : tensor(a[2], "y");
  if (PyErr_Occurred()) return nullptr;
  if ((th && code(*th) < 0) || (ty && code(*ty) < 0)) {
    fail(PyExc_ValueError, "h and y must be bfloat16 or float32");
    return nullptr;
  }
  // rows of another length are refused, also where their values happen to fill whole rows
  const int64_t d = nm->d;
  auto rows = [&](const at::Tensor& t, const char* name) {
    return (t.dim() > 0 && t.size(-1) == d) || fail(PyExc_ValueError, std::string(name) + " must be [T, " + std::to_string(d) + "]");
  };
  if ((th && !rows(*th, "h")) || (ty && !rows(*ty, "y"))) return nullptr;
  const int64_t T = th ? th->numel() / d : 0;
  int64_t stride = 0;
  if (a[5] != Py_None) {
    const at::Tensor* tg = tensor(a[5], "gate");
    if (!tg || !rows(*tg, "gate")) return nullptr;
    stride = tg->dim() == 1 ? 0 : d;
  }
  if (!address(a[2], "y", kAny, T * d, &y) || !address(a[3], "h_out", th ? th->scalar_type() : kAny, T * d, &h_out) ||
      !address(a[4], "x_out", weight_type(nm), T * d, &x_out) || !address(a[5], "gate", weight_type(nm), stride ? T * d : d, &gate))
    return nullptr;
  if (!fits(T, "T")) return nullptr;
  void* stream = pointer(a[6]);
  if (PyErr_Occurred()) return nullptr;
  const int hdt = th ? code(*th) : SFN_F32, ydt = ty ? code(*ty) : SFN_F32;
  return status_of([&] { return f_norm(nm, (int32_t)T, h, hdt, y, ydt, gate, stride, h_out, x_out, stream); });
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);

// F with its C++ exceptions raised as Python's: torch throws for a tensor without storage or
// strides, and no exception may pass through the interpreter's C frames.
template <Fast F>
PyObject* raising(PyObject* self, PyObject* const* a, Py_ssize_t n) noexcept {
  try {
    return F(self, a, n);
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

template <Fast F>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&raising<F>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<bind>("bind"),     method<plan>("plan"), method<append>("append"),
                         method<attend>("attend"), method<norm>("norm"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_args", nullptr, -1, methods};

}  // namespace

#define SFN_TEXT_OF(x) #x
#define SFN_TEXT(x) SFN_TEXT_OF(x)

// The module holds for the torch and the Python that it was built against, which the binding compares.
PyMODINIT_FUNC PyInit__torch_args() {
  PyObject* m = PyModule_Create(&module);
  if (m && (PyModule_AddStringConstant(m, "TORCH_VERSION", TORCH_VERSION) < 0 ||
            PyModule_AddStringConstant(m, "PY_VERSION", SFN_TEXT(PY_MAJOR_VERSION) "." SFN_TEXT(PY_MINOR_VERSION)) < 0))
    Py_CLEAR(m);
  return m;
}
