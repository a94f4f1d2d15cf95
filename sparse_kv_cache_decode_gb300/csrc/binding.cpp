// The parts of the Python binding that a decoding loop pays for in every call: reading what a tensor is, and passing plain
// numbers to the C ABI.  (On the host of a GB300 a call of kvs_rotate took 9 us through ctypes, 2.3 of them the launch.)
// A check returns None where the tensor is not what it should be; the Python side then says why.
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <tuple>
#include <type_traits>
#include <utility>

#include "../../include/kvs.h"

namespace {

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }
bool is_dtype(const at::Tensor& t, PyObject* dtypes) {
  for (Py_ssize_t i = 0, n = PyTuple_GET_SIZE(dtypes); i < n; ++i) {
    PyObject* d = PyTuple_GET_ITEM(dtypes, i);
    if (THPDtype_Check(d) && reinterpret_cast<THPDtype*>(d)->scalar_type == t.scalar_type()) return true;
  }
  return false;
}
bool wrong_args(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return false;
  PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", got, want);
  return true;
}
PyObject* pointer(const at::Tensor& t) { return PyLong_FromVoidPtr(t.data_ptr()); }

// whole(t, dtypes, shape, device index): the pointer of a contiguous tensor
PyObject* whole(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (wrong_args(n, 4)) return nullptr;
  const at::Tensor* t = tensor(a[0]);
  if (!t || !PyTuple_Check(a[1]) || !PyTuple_Check(a[2])) Py_RETURN_NONE;
  const Py_ssize_t dim = PyTuple_GET_SIZE(a[2]);
  if (t->dim() != dim || !is_dtype(*t, a[1]) || !t->is_contiguous() || t->get_device() != PyLong_AsLong(a[3])) Py_RETURN_NONE;
  for (Py_ssize_t i = 0; i < dim; ++i)
    if (t->size(i) != PyLong_AsLongLong(PyTuple_GET_ITEM(a[2], i))) {
      if (PyErr_Occurred()) return nullptr;
      Py_RETURN_NONE;
    }
  return pointer(*t);
}

// rows(t, dtypes, heads or -1, d, device index): (pointer, token stride, head stride, tokens, heads) of [tokens][heads][d]
PyObject* rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (wrong_args(n, 5)) return nullptr;
  const at::Tensor* t = tensor(a[0]);
  if (!t || !PyTuple_Check(a[1])) Py_RETURN_NONE;
  const long long heads = PyLong_AsLongLong(a[2]), d = PyLong_AsLongLong(a[3]);
  if (t->dim() != 3 || !is_dtype(*t, a[1]) || t->size(2) != d || (heads >= 0 && t->size(1) != heads) || (t->numel() && t->stride(2) != 1) ||
      t->get_device() != PyLong_AsLong(a[4]))
    Py_RETURN_NONE;
  const long long tok = t->size(0), h = t->size(1), s1 = h <= 1 ? d : t->stride(1), s0 = tok <= 1 || !t->numel() ? h * s1 : t->stride(0);
  return Py_BuildValue("(NLLLL)", pointer(*t), s0, s1, tok, h);
}

PyObject* device(PyObject*, PyObject*) { return PyLong_FromLong(c10::cuda::current_device()); }
PyObject* stream(PyObject*, PyObject* index) {
  const long i = PyLong_AsLong(index);
  if (i == -1 && PyErr_Occurred()) return nullptr;
  return PyLong_FromVoidPtr(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)i).stream());
}

// ------------------------------------------------------------------ calls: numbers, None for a null pointer, ctypes pointers
template <typename T>
bool get(PyObject* o, T* out) {
  if constexpr (std::is_pointer_v<T>) {
    if (o == Py_None) {
      *out = nullptr;
      return true;
    }
    if (PyLong_Check(o)) {
      *out = static_cast<T>(PyLong_AsVoidPtr(o));
    } else {      // a ctypes pointer
      PyObject* v = PyObject_GetAttrString(o, "value");
      if (!v) return false;
      *out = v == Py_None ? nullptr : static_cast<T>(PyLong_AsVoidPtr(v));
      Py_DECREF(v);
    }
  } else {
    const long long v = PyLong_AsLongLong(o);
    *out = static_cast<T>(v);
    if (!PyErr_Occurred() && static_cast<long long>(*out) != v) PyErr_SetString(PyExc_OverflowError, "an integer that does not fit 32 bits");
  }
  return !PyErr_Occurred();
}

template <typename... A, size_t... I>
PyObject* call_with(kvs_status (*fn)(A...), PyObject* const* args, std::index_sequence<I...>) {
  std::tuple<A...> v;
  if (!(get(args[I], &std::get<I>(v)) && ...)) return nullptr;
  kvs_status status;
  Py_BEGIN_ALLOW_THREADS      // (a launch may wait for the GPU's queue)
  status = fn(std::get<I>(v)...);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}
template <auto FN, typename... A>
PyObject* call_as(kvs_status (*)(A...), PyObject* const* args, Py_ssize_t n) {
  if (wrong_args(n, sizeof...(A))) return nullptr;
  return call_with<A...>(FN, args, std::index_sequence_for<A...>{});
}
template <auto FN>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call_as<FN>(FN, args, n);
}

// A C++ exception (a tensor without storage, no device) ends here.
template <auto FN, typename... A>
PyObject* guarded(A... a) {
  try {
    return FN(a...);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}
template <auto FN>
PyObject* fast(PyObject* m, PyObject* const* a, Py_ssize_t n) { return guarded<FN>(m, a, n); }
template <auto FN>
PyObject* plain(PyObject* m, PyObject* o) { return guarded<FN>(m, o); }

#define KVS_FAST(fn) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&fast<&fn>))
#define KVS_CALL(name) {#name, KVS_FAST(call<&name>), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"whole", KVS_FAST(whole), METH_FASTCALL, nullptr},
    {"rows", KVS_FAST(rows), METH_FASTCALL, nullptr},
    {"device", &plain<&device>, METH_NOARGS, nullptr},
    {"stream", &plain<&stream>, METH_O, nullptr},
    KVS_CALL(kvs_pool_append),
    KVS_CALL(kvs_pool_attn),
    KVS_CALL(kvs_pool_prefix_attn),
    KVS_CALL(kvs_pool_evict),
    KVS_CALL(kvs_pool_reserve),
    KVS_CALL(kvs_pool_places),
    KVS_CALL(kvs_rotate),
    KVS_CALL(kvs_pool_rotate_append),
    KVS_CALL(kvs_pool_reposition),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "kvs_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kvs_binding(void) { return PyModule_Create(&module); }
