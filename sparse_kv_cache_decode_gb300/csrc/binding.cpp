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

// the current device, or -1 without one
PyObject* device(PyObject*, PyObject*) {
  c10::DeviceIndex i = -1;
  return PyLong_FromLong(c10::cuda::GetDevice(&i) == cudaSuccess ? i : -1);
}
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

// ------------------------------------------------------------------ whole calls: tensors checked and passed on
// Each returns the call's status, or None where a tensor is not what it should be, the device not the current one, or an integer too
// large: the Python side then goes through the same checks one by one and says which.
struct Rows {
  void* p = nullptr;
  long long tok = 0, head = 0, n = 0, heads = 0;
};
struct Parser {
  long index;      // the device
  bool ok = true;

  const at::Tensor* take(PyObject* o, at::ScalarType a, at::ScalarType b) {
    const at::Tensor* t = tensor(o);
    if (t && (t->scalar_type() == a || t->scalar_type() == b) && t->get_device() == index) return t;
    ok = false;
    return nullptr;
  }
  Rows rows(PyObject* o, long long heads, long long d) {
    Rows r;
    const at::Tensor* t = take(o, at::kBFloat16, at::kShort);
    if (!t) return r;
    if (t->dim() != 3 || t->size(2) != d || (heads >= 0 && t->size(1) != heads) || (t->numel() && t->stride(2) != 1)) {
      ok = false;
      return r;
    }
    r.p = t->data_ptr();
    r.n = t->size(0);
    r.heads = t->size(1);
    r.head = r.heads <= 1 ? d : t->stride(1);
    r.tok = r.n <= 1 || !t->numel() ? r.heads * r.head : t->stride(0);
    return r;
  }
  // rows whose heads lie together
  Rows tokens(PyObject* o, long long heads, long long d) {
    const Rows r = rows(o, heads, d);
    ok = ok && r.head == d && r.tok >= heads * d;
    return r;
  }
  // a contiguous tensor of n (or a x b) elements; None: a null pointer where it may be left out
  template <typename T>
  T* vec(PyObject* o, at::ScalarType type, long long n, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    const at::Tensor* t = take(o, type, type);
    if (!t) return nullptr;
    if (t->dim() != 1 || t->size(0) != n || !t->is_contiguous()) ok = false;
    return static_cast<T*>(t->data_ptr());
  }
  // [n], or [n_axis] rows of [n] that may be parts of longer ones
  const int* positions(PyObject* o, long long n_axis, long long n, long long* stride) {
    const at::Tensor* t = take(o, at::kInt, at::kInt);
    if (!t) return nullptr;
    const auto dim = t->dim();
    if (dim < 1 || dim > 2 || t->size(dim - 1) != n || (dim == 2 && t->size(0) != n_axis) || (n > 1 && t->stride(dim - 1) != 1)) {
      ok = false;
      return nullptr;
    }
    *stride = dim == 1 || n_axis == 1 ? 0 : t->stride(0);
    return static_cast<const int*>(t->data_ptr());
  }
  template <typename T>
  T number(PyObject* o) {
    T v{};
    if (ok && !get(o, &v)) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  kvs_stream_t stream(PyObject* o) {
    ok = ok && index >= 0;
    if (!ok) return nullptr;
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
    PyObject* v = PyLong_Check(o) ? (Py_INCREF(o), o) : PyObject_GetAttrString(o, "cuda_stream");
    const kvs_stream_t s = v ? static_cast<kvs_stream_t>(PyLong_AsVoidPtr(v)) : nullptr;
    Py_XDECREF(v);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return s;
  }
  bool here() const { return ok && index >= 0 && c10::cuda::current_device() == index; }
};
template <typename F>
PyObject* go(const Parser& p, F f) {
  if (!p.here()) Py_RETURN_NONE;
  kvs_status status;
  Py_BEGIN_ALLOW_THREADS
  status = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}
constexpr long long kInt = 0x7fffffff;

// rotate(handle, d, n_axis, q, pos, q_out, k, k_out, q_norm, k_norm, stream)
PyObject* rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (wrong_args(n, 11)) return nullptr;
  const at::Tensor* t = tensor(a[3]);
  Parser p{t ? (long)t->get_device() : -1};
  const auto* h = p.number<const kvs_rope*>(a[0]);
  const int d = p.number<int>(a[1]), n_axis = p.number<int>(a[2]);
  const Rows q = p.rows(a[3], -1, d), qo = p.rows(a[5], q.heads, d);
  Rows k, ko;
  if ((a[6] == Py_None) != (a[7] == Py_None)) Py_RETURN_NONE;
  if (a[6] != Py_None) {
    k = p.rows(a[6], -1, d);
    ko = p.rows(a[7], k.heads, d);
  }
  if (!p.ok || qo.n != q.n || (a[6] != Py_None && (k.n != q.n || ko.n != q.n)) || q.n > kInt || q.heads > kInt || k.heads > kInt) Py_RETURN_NONE;
  long long ps = 0;
  const int* pos = p.positions(a[4], n_axis, q.n, &ps);
  const auto *qn = p.vec<const float>(a[8], at::kFloat, d, true), *kn = p.vec<const float>(a[9], at::kFloat, d, true);
  const kvs_stream_t s = p.stream(a[10]);
  return go(p, [&] {
    return kvs_rotate(h, q.p, q.tok, q.head, (int)q.heads, qn, qo.p, qo.tok, qo.head, k.p, k.tok, k.head, (int)k.heads, kn, ko.p, ko.tok, ko.head,
                      pos, ps, (int)q.n, s);
  });
}

// rotate_append(pool, rope, index, H_q, H_kv, d, n_axis, layer, q, k, v, pos, place, q_out, q_norm, k_norm, stream)
PyObject* rotate_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (wrong_args(n, 17)) return nullptr;
  Parser p{-1};
  p.index = p.number<int>(a[2]);
  auto* h = p.number<kvs_pool*>(a[0]);
  const auto* rope = p.number<const kvs_rope*>(a[1]);
  const int hq = p.number<int>(a[3]), hk = p.number<int>(a[4]), d = p.number<int>(a[5]), n_axis = p.number<int>(a[6]), layer = p.number<int>(a[7]);
  if (!p.ok) Py_RETURN_NONE;
  const Rows q = p.tokens(a[8], hq, d), k = p.tokens(a[9], hk, d), v = p.tokens(a[10], hk, d), qo = p.tokens(a[13], hq, d);
  if (!p.ok || k.n != q.n || v.n != q.n || qo.n != q.n || k.tok != v.tok || q.n > kInt) Py_RETURN_NONE;
  long long ps = 0;
  const int* pos = p.positions(a[11], n_axis, q.n, &ps);
  const auto* place = p.vec<const long long>(a[12], at::kLong, q.n);
  const auto *qn = p.vec<const float>(a[14], at::kFloat, d, true), *kn = p.vec<const float>(a[15], at::kFloat, d, true);
  const kvs_stream_t s = p.stream(a[16]);
  return go(p, [&] { return kvs_pool_rotate_append(h, rope, layer, q.p, q.tok, k.p, v.p, k.tok, qn, kn, pos, ps, place, (int)q.n, qo.p, qo.tok, s); });
}

// reserve(pool, index, n_req, held, table, ring, state, ctx_len, cu_q, place, pos, pos_delta, stream)
PyObject* reserve(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (wrong_args(n, 13)) return nullptr;
  Parser p{-1};
  p.index = p.number<int>(a[1]);
  auto* h = p.number<kvs_pool*>(a[0]);
  const int n_req = p.number<int>(a[2]);
  auto *held = p.number<int*>(a[3]), *table = p.number<int*>(a[4]), *ring = p.number<int*>(a[5]), *state = p.number<int*>(a[6]);
  const int* ctx = p.vec<const int>(a[7], at::kInt, n_req);
  const int *cu = nullptr, *delta = nullptr;
  long long* place = nullptr;
  int* pos = nullptr;
  long long n_tok = 0;
  if (a[8] != Py_None) {
    const at::Tensor* t = tensor(a[9]);
    if (!t || t->dim() != 1 || (n_tok = t->size(0)) > kInt) Py_RETURN_NONE;
    cu = p.vec<const int>(a[8], at::kInt, n_req + 1ll);
    place = p.vec<long long>(a[9], at::kLong, n_tok);
    pos = p.vec<int>(a[10], at::kInt, n_tok, true);
    delta = p.vec<const int>(a[11], at::kInt, n_req, true);
  } else if (a[9] != Py_None || a[10] != Py_None || a[11] != Py_None) {
    Py_RETURN_NONE;
  }
  const kvs_stream_t s = p.stream(a[12]);
  return go(p, [&] { return kvs_pool_reserve(h, ctx, held, table, ring, state, n_req, cu, delta, (int)n_tok, place, pos, s); });
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
    {"rotate", KVS_FAST(rotate), METH_FASTCALL, nullptr},
    {"rotate_append", KVS_FAST(rotate_append), METH_FASTCALL, nullptr},
    {"reserve", KVS_FAST(reserve), METH_FASTCALL, nullptr},
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
