// Python calls of the entry points whose kernels take a few microseconds: arguments are
// converted by the types of the C declarations, tensors to their data_ptr().  (Through
// ctypes a call of fourteen arguments spends 3.1 us before it reaches the library, more
// than the 2.3 us that writing a token for each of 64 sequences takes the GPU.)
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>
#include <stddef.h>

#include <tuple>
#include <type_traits>
#include <utility>

#include "nb.h"

namespace {

PyObject* g_data_ptr;  // the interned name of the method

bool convert(PyObject* o, int* out) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) return false;
  if (x < INT_MIN || x > INT_MAX) {
    PyErr_SetString(PyExc_OverflowError, "argument does not fit 32 bits");
    return false;
  }
  *out = static_cast<int>(x);
  return true;
}

bool convert(PyObject* o, size_t* out) {
  *out = PyLong_AsSize_t(o);
  return !(*out == static_cast<size_t>(-1) && PyErr_Occurred());
}

template <class T>
bool convert(PyObject* o, T** out) {  // None, an address or a tensor
  if (o == Py_None) {
    *out = nullptr;
    return true;
  }
  PyObject* at = o;
  if (PyLong_Check(o)) Py_INCREF(o);
  else at = PyObject_CallMethodNoArgs(o, g_data_ptr);
  if (!at) return false;
  void* p = PyLong_AsVoidPtr(at);
  Py_DECREF(at);
  *out = static_cast<T*>(p);
  return !(p == nullptr && PyErr_Occurred());
}

template <class... A, size_t... I>
PyObject* apply(nb_status (*fn)(A...), PyObject* const* args, std::index_sequence<I...>) {
  std::tuple<A...> v;
  if (!(convert(args[I], &std::get<I>(v)) && ...)) return nullptr;
  long status;
  Py_BEGIN_ALLOW_THREADS  // a launch waits when the queue of launches is full
  status = static_cast<long>(fn(std::get<I>(v)...));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

template <class... A>
PyObject* apply(nb_status (*fn)(A...), PyObject* const* args, Py_ssize_t n) {
  if (n != static_cast<Py_ssize_t>(sizeof...(A)))
    return PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd",
                        static_cast<Py_ssize_t>(sizeof...(A)), n);
  return apply(fn, args, std::index_sequence_for<A...>{});
}

template <auto Fn>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return apply(Fn, args, n);
}

template <auto Fn>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<Fn>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<&nb_attn_sink_fwd>("nb_attn_sink_fwd"),
                           method<&nb_attn_sink_bwd>("nb_attn_sink_bwd"),
                           method<&nb_kv4_write>("nb_kv4_write"),
                           method<&nb_kv4_read>("nb_kv4_read"),
                           method<&nb_attn_kv4_decode>("nb_attn_kv4_decode"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_call", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__call() {
  g_data_ptr = PyUnicode_InternFromString("data_ptr");
  if (!g_data_ptr) return nullptr;
  PyObject* m = PyModule_Create(&g_module);
  // the binding uses this module only beside a library of the same version
  if (m && PyModule_AddIntConstant(m, "abi_version", NB_ABI_VERSION) < 0) Py_CLEAR(m);
  return m;
}
