// binding.cpp -- the Python calls of the small, often made operators.
//
// A call marshalled through ctypes costs about 2 us for twenty arguments and as
// much again for the Python around it, more than the kernel of a 64-token step
// runs (q/k norm of 64 tokens: 6.6 us a call that way, 3.7 this way).  Here an argument list becomes a C call in one step: each function of
// this module takes the arguments of the entry point of its name in
// include/photon_paged.h (as integers, floats, objects with data_ptr(),
// structures that offer their bytes, or None for a null pointer) and returns
// the status.  The conversions follow from the declarations.  The addresses
// come from the library that the ctypes binding has loaded (bind), so the module
// links against nothing.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstring>
#include <limits>
#include <tuple>
#include <type_traits>
#include <utility>

#include "photon_paged.h"

namespace {

PyObject* g_data_ptr;   // the string "data_ptr"

// int(x) within T's range
template <typename T>
bool to_integer(PyObject* o, T* v) {
  PyObject* n = PyNumber_Long(o);
  if (!n) return false;
  bool ok;
  if constexpr (std::is_signed<T>::value) {
    int over = 0;
    const long long x = PyLong_AsLongLongAndOverflow(n, &over);
    ok = !over && x >= std::numeric_limits<T>::min() && x <= std::numeric_limits<T>::max();
    *v = static_cast<T>(x);
  } else {
    const unsigned long long x = PyLong_AsUnsignedLongLong(n);
    ok = !PyErr_Occurred() && x <= std::numeric_limits<T>::max();
    PyErr_Clear();
    *v = static_cast<T>(x);
  }
  Py_DECREF(n);
  if (!ok) PyErr_Format(PyExc_OverflowError, "%R does not fit the argument", o);
  return ok;
}

bool to_address(PyObject* o, void** v) {
  if (o == Py_None) {
    *v = nullptr;
    return true;
  }
  PyObject* n = PyLong_Check(o) ? Py_NewRef(o) : PyObject_CallMethodNoArgs(o, g_data_ptr);
  if (!n) return false;
  *v = PyLong_AsVoidPtr(n);
  Py_DECREF(n);
  return !PyErr_Occurred();
}

// One argument of C type T: take() converts it, get() passes it.
template <typename T>
struct Arg {
  T v;
  bool take(PyObject* o) {
    if constexpr (std::is_floating_point<T>::value) {
      const double x = PyFloat_AsDouble(o);
      v = static_cast<T>(x);
      return x != -1.0 || !PyErr_Occurred();
    } else {
      return to_integer(o, &v);
    }
  }
  T get() const { return v; }
};
template <typename T>
struct Arg<T*> {
  void* v;
  bool take(PyObject* o) { return to_address(o, &v); }
  T* get() const { return static_cast<T*>(v); }
};
// structures travel by value
template <typename T>
struct StructArg {
  T v;
  bool take(PyObject* o) {
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) return false;
    const bool ok = b.len == (Py_ssize_t)sizeof(T);
    if (ok)
      std::memcpy(&v, b.buf, sizeof(T));
    else
      PyErr_SetString(PyExc_TypeError, "a structure of another size");
    PyBuffer_Release(&b);
    return ok;
  }
  const T* get() const { return &v; }
};
template <>
struct Arg<const photon_paged_shape_t*> : StructArg<photon_paged_shape_t> {};
template <>
struct Arg<const photon_rope_axes_t*> : StructArg<photon_rope_axes_t> {};

template <typename... A, size_t... I>
PyObject* call_with(photon_status_t (*fn)(A...), PyObject* const* argv,
                    std::index_sequence<I...>) {
  std::tuple<Arg<A>...> args;
  if (!(std::get<I>(args).take(argv[I]) && ...)) return nullptr;
  photon_status_t status;
  Py_BEGIN_ALLOW_THREADS;
  status = fn(std::get<I>(args).get()...);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(static_cast<long>(status));
}

template <typename... A>
PyObject* call(photon_status_t (*fn)(A...), const char* name, PyObject* const* argv,
               Py_ssize_t n) {
  if (!fn) return PyErr_Format(PyExc_RuntimeError, "%s: no library is bound", name);
  if (n != (Py_ssize_t)sizeof...(A))
    return PyErr_Format(PyExc_TypeError, "%s takes %zu arguments, not %zd", name, sizeof...(A), n);
  return call_with(fn, argv, std::index_sequence_for<A...>());
}

#define PHOTON_CALLS(X)          \
  X(photon_cache_write_int4)     \
  X(photon_paged_gather_int4)    \
  X(photon_paged_decode_int4)    \
  X(photon_qk_norm_rope)         \
  X(photon_prompt_attention)

#define PHOTON_DEFINE(name)                                                         \
  decltype(&::name) g_##name;                                                       \
  PyObject* py_##name(PyObject*, PyObject* const* argv, Py_ssize_t n) {             \
    return call(g_##name, #name, argv, n);                                          \
  }
PHOTON_CALLS(PHOTON_DEFINE)

// bind(name, address): where the entry point of that name is
PyObject* bind(PyObject*, PyObject* args) {
  const char* name;
  PyObject* at;
  void* address;
  if (!PyArg_ParseTuple(args, "sO", &name, &at) || !to_address(at, &address)) return nullptr;
#define PHOTON_BIND(entry)                                               \
  if (std::strcmp(name, #entry) == 0) {                                  \
    g_##entry = reinterpret_cast<decltype(&::entry)>(address);           \
    Py_RETURN_NONE;                                                      \
  }
  PHOTON_CALLS(PHOTON_BIND)
  return PyErr_Format(PyExc_ValueError, "no call is named %s", name);
}

#define PHOTON_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr},
PyMethodDef g_methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                           PHOTON_CALLS(PHOTON_METHOD){nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  g_data_ptr = PyUnicode_InternFromString("data_ptr");
  return g_data_ptr ? PyModule_Create(&g_module) : nullptr;
}
