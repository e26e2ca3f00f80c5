// The binding's marshalling of the single-token calls (module _call).
//
// These calls take the GPU 1 to 6 us, and Python's own time for one through
// ctypes was 4 us more than the C entry's 4: some 0.7 us to read a tensor's
// shape, strides, type, device and address, and 0.1 us per argument. Here the
// same reads and the same refusals take 1 to 2 us (a call, through ctypes and so, us:
// rotation of five tokens 8.6 and 5.2, attention over 77 tokens 8.5 and 4.8, write
// of four tokens 7.1 and 3.8, dense layer of one token 7.7 and 5.8). Nothing is
// computed or kept: the C entries' addresses and torch's dtype objects apart, every
// call stands for itself.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "wave.h"

namespace {

decltype(&wave_linear_bias) g_linear;
decltype(&wave_rotary) g_rotary;
decltype(&wave_kv_write_tokens) g_write;
decltype(&wave_token_attn) g_attn;
PyObject *g_bf16, *g_f32, *g_i32;                                         // torch's dtypes
PyObject *s_shape, *s_stride, *s_dtype, *s_device, *s_ptr, *s_contiguous, *s_nbytes;  // attribute names

constexpr int kMostDims = 4;

bool as_int64(PyObject* o, int64_t* v) {
  *v = PyLong_AsLongLong(o);
  return *v != -1 || !PyErr_Occurred();
}
bool as_int32(PyObject* o, int32_t* v) {
  int64_t w;
  if (!as_int64(o, &w)) return false;
  if (w < INT32_MIN || w > INT32_MAX) {
    PyErr_Format(PyExc_OverflowError, "%lld does not fit 32 bits", (long long)w);
    return false;
  }
  *v = (int32_t)w;
  return true;
}
bool as_pointer(PyObject* o, void** p) {
  int64_t v = 0;
  if (o != Py_None && !as_int64(o, &v)) return false;
  *p = reinterpret_cast<void*>((intptr_t)v);
  return true;
}
// A method's result as an integer.
bool ask(PyObject* t, PyObject* method, int64_t* v) {
  PyObject* r = PyObject_CallMethodNoArgs(t, method);
  if (!r) return false;
  const bool ok = as_int64(r, v);
  Py_DECREF(r);
  return ok;
}
// A tuple of integers into v (at most kMostDims); its length, or -1. Steals t.
int dims(PyObject* t, int64_t* v) {
  if (!t) return -1;
  int n = -1;
  if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) > kMostDims) {
    PyErr_SetString(PyExc_ValueError, "a tensor of at most four dimensions is wanted");
  } else {
    n = (int)PyTuple_GET_SIZE(t);
    for (int i = 0; i < n; ++i)
      if (!as_int64(PyTuple_GET_ITEM(t, i), v + i)) {
        n = -1;
        break;
      }
  }
  Py_DECREF(t);
  return n;
}
int shape_of(PyObject* t, int64_t* v) { return dims(PyObject_GetAttr(t, s_shape), v); }

// The type and device of t are those wanted: 1, 0, or -1 with an error set.
int is_kind(PyObject* t, PyObject* dtype, int64_t index) {
  PyObject* have = PyObject_GetAttr(t, s_dtype);
  if (!have) return -1;
  Py_DECREF(have);
  if (have != dtype) return 0;
  int64_t device;
  if (!ask(t, s_device, &device)) return -1;
  return device == index;
}

bool refuse(PyObject* t, const char* what, int64_t rows, int64_t width, PyObject* dtype, int64_t index) {
  if (PyErr_Occurred()) return false;
  PyObject* shape = PyObject_GetAttr(t, s_shape);
  PyObject* stride = PyObject_CallMethodNoArgs(t, s_stride);
  PyObject* have = PyObject_GetAttr(t, s_dtype);
  if (shape && stride && have)
    PyErr_Format(PyExc_ValueError,
                 "%s: %lld rows of %lld contiguous %S elements on cuda:%lld are wanted, got shape %S, strides %S, %S",
                 what, (long long)rows, (long long)width, dtype, (long long)index, shape, stride, have);
  Py_XDECREF(shape);
  Py_XDECREF(stride);
  Py_XDECREF(have);
  return false;
}

struct Rows {
  void* p;
  int64_t ld;
};
// Address and row stride of a CUDA tensor read as `rows` rows of `width`
// contiguous elements: [rows][width], or [rows][heads][d] with contiguous
// heads. A kernel would read a host tensor's address, or past a short one, as
// readily as a good one, so both are refused here.
bool rows_of(PyObject* t, const char* what, int64_t rows, int64_t width, PyObject* dtype, int64_t index, Rows* r) {
  int64_t n[kMostDims], st[kMostDims];
  const int nd = shape_of(t, n);
  if (nd < 0 || dims(PyObject_CallMethodNoArgs(t, s_stride), st) != nd) return refuse(t, what, rows, width, dtype, index);
  bool ok = (nd == 2 || nd == 3) && n[0] == rows;
  if (ok && nd == 3)
    ok = n[1] * n[2] == width && st[2] == 1 && (st[1] == n[2] || n[1] == 1);
  else if (ok)
    ok = n[1] == width && st[1] == 1;
  if (!ok || is_kind(t, dtype, index) != 1) return refuse(t, what, rows, width, dtype, index);
  int64_t p;
  if (!ask(t, s_ptr, &p)) return false;
  r->p = reinterpret_cast<void*>((intptr_t)p);
  r->ld = rows > 1 ? st[0] : width;
  return true;
}
bool contiguous(const Rows& r, int64_t rows, int64_t width, const char* what) {
  if (rows <= 1 || r.ld == width) return true;
  PyErr_Format(PyExc_ValueError, "%s must be contiguous", what);
  return false;
}
// [rows][heads][d] of a tensor.
bool heads_of(PyObject* t, const char* what, int64_t d, int64_t* rows, int64_t* heads) {
  int64_t n[kMostDims];
  const int nd = shape_of(t, n);
  if (nd == 3 && n[2] == d && n[0] <= INT32_MAX && n[1] <= INT32_MAX) {
    *rows = n[0];
    *heads = n[1];
    return true;
  }
  if (nd >= 0) PyErr_Format(PyExc_ValueError, "%s is [rows][heads][%lld]", what, (long long)d);
  return false;
}

// A Python sequence of int32 values, appended to v.
bool ints_of(PyObject* o, std::vector<int32_t>& v) {
  PyObject* seq = PySequence_Fast(o, "a sequence of integers is wanted");
  if (!seq) return false;
  bool ok = true;
  for (Py_ssize_t i = 0; ok && i < PySequence_Fast_GET_SIZE(seq); ++i) {
    int32_t x;
    ok = as_int32(PySequence_Fast_GET_ITEM(seq, i), &x);
    if (ok) v.push_back(x);
  }
  Py_DECREF(seq);
  return ok;
}
bool exactly(const std::vector<int32_t>& v, size_t n, const char* what) {
  if (v.size() == n) return true;
  PyErr_Format(PyExc_ValueError, "%s: %zu values wanted, got %zu", what, n, v.size());
  return false;
}
// A sequence of (chunk, level) pairs as a wave_node array.
bool nodes_of(PyObject* o, std::vector<int32_t>& v) {
  static_assert(sizeof(wave_node) == 2 * sizeof(int32_t), "two int32 a node");
  PyObject* seq = PySequence_Fast(o, "a sequence of (chunk, level) pairs is wanted");
  if (!seq) return false;
  bool ok = true;
  for (Py_ssize_t i = 0; ok && i < PySequence_Fast_GET_SIZE(seq); ++i) {
    ok = ints_of(PySequence_Fast_GET_ITEM(seq, i), v);
    if (ok && v.size() != 2 * (size_t)(i + 1)) {
      PyErr_SetString(PyExc_ValueError, "a node is a (chunk, level) pair");
      ok = false;
    }
  }
  Py_DECREF(seq);
  return ok;
}
const wave_node* as_nodes(const std::vector<int32_t>& v) { return reinterpret_cast<const wave_node*>(v.data()); }

bool counted(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments wanted, got %zd", want, got);
  return false;
}

template <class F>
PyObject* call(F f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

// bind(linear_bias, rotary, write, attn, bfloat16, float32, int32): the C entries' addresses,
// torch's dtypes.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[4];
  if (!counted(n, 7)) return nullptr;
  for (int i = 0; i < 4; ++i)
    if (!as_pointer(a[i], p + i)) return nullptr;
  std::memcpy(&g_linear, p, sizeof(void*));
  std::memcpy(&g_rotary, p + 1, sizeof(void*));
  std::memcpy(&g_write, p + 2, sizeof(void*));
  std::memcpy(&g_attn, p + 3, sizeof(void*));
  g_bf16 = Py_NewRef(a[4]);
  g_f32 = Py_NewRef(a[5]);
  g_i32 = Py_NewRef(a[6]);
  Py_RETURN_NONE;
}

// linear_bias(handle, device, A, W, Y, bias, R, act, stream)
PyObject* linear_bias(PyObject*, PyObject* const* a, Py_ssize_t count) {
  void *h, *stream, *bias = nullptr;
  int64_t index, n[kMostDims], wn[kMostDims];
  int32_t act;
  Rows A, W, Y, R{nullptr, 0};
  if (!counted(count, 9) || !as_pointer(a[0], &h) || !as_int64(a[1], &index) || !as_int32(a[7], &act) ||
      !as_pointer(a[8], &stream))
    return nullptr;
  const int nd = shape_of(a[2], n), wd = nd < 0 ? -1 : shape_of(a[3], wn);
  if (wd < 0) return nullptr;
  if (nd != 2 || wd < 1 || n[0] > INT32_MAX || n[1] > INT32_MAX || wn[0] > INT32_MAX) {
    PyErr_SetString(PyExc_ValueError, "A is [M][K] and W is [N][K]");
    return nullptr;
  }
  const int64_t M = n[0], K = n[1], N = wn[0];
  if (!rows_of(a[2], "A", M, K, g_bf16, index, &A) || !rows_of(a[3], "W", N, K, g_bf16, index, &W) ||
      !contiguous(W, N, K, "W") || !rows_of(a[4], "Y", M, N, g_bf16, index, &Y))
    return nullptr;
  if (a[5] != Py_None) {
    int64_t bn[kMostDims], numel = 1, flat, p;
    const int bd = shape_of(a[5], bn);
    for (int i = 0; i < bd; ++i) numel *= bn[i];
    if (bd < 0 || !ask(a[5], s_contiguous, &flat) || !flat || numel != N || is_kind(a[5], g_bf16, index) != 1)
      return refuse(a[5], "bias", 1, N, g_bf16, index), nullptr;
    if (!ask(a[5], s_ptr, &p)) return nullptr;
    bias = reinterpret_cast<void*>((intptr_t)p);
  }
  if (a[6] != Py_None && !rows_of(a[6], "R", M, N, g_bf16, index, &R)) return nullptr;
  return call([&] {
    return g_linear(static_cast<wave_kv*>(h), A.p, A.ld, (int32_t)M, (int32_t)K, W.p, (int32_t)N, bias, R.p, R.ld, act,
                    Y.p, Y.ld, stream);
  });
}

// rotary(handle, device, d, spec, positions, Q, K, Qout, Kout, stream)
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t count) {
  void *h, *spec, *stream;
  int64_t index, d, rows, qh, kh = 0, krows;
  Rows pos, Q, K{nullptr, 0}, Qo, Ko{nullptr, 0};
  if (!counted(count, 10) || !as_pointer(a[0], &h) || !as_int64(a[1], &index) || !as_int64(a[2], &d) ||
      !as_pointer(a[3], &spec) || !as_pointer(a[9], &stream) || !heads_of(a[5], "Q", d, &rows, &qh))
    return nullptr;
  if (!rows_of(a[4], "positions", rows, 3, g_i32, index, &pos) || !contiguous(pos, rows, 3, "positions") ||
      !rows_of(a[5], "Q", rows, qh * d, g_bf16, index, &Q) || !rows_of(a[7], "Qout", rows, qh * d, g_bf16, index, &Qo))
    return nullptr;
  if (a[6] != Py_None && (!heads_of(a[6], "K", d, &krows, &kh) ||
                          !rows_of(a[6], "K", rows, kh * d, g_bf16, index, &K) ||
                          !rows_of(a[8], "Kout", rows, kh * d, g_bf16, index, &Ko)))
    return nullptr;
  return call([&] {
    return g_rotary(static_cast<wave_kv*>(h), static_cast<const wave_rotary_spec*>(spec),
                    static_cast<const int32_t*>(pos.p), (int32_t)rows, Q.p, Q.ld, (int32_t)qh, Qo.p, Qo.ld, K.p, K.ld,
                    (int32_t)kh, Ko.p, Ko.ld, stream);
  });
}

// write_tokens(handle, device, width, entries, first, counts, K, V, stream)
PyObject* write_tokens(PyObject*, PyObject* const* a, Py_ssize_t count) try {
  void *h, *stream;
  int64_t index, width, rows = 0;
  std::vector<int32_t> nodes, first, counts;
  Rows K, V;
  if (!counted(count, 9) || !as_pointer(a[0], &h) || !as_int64(a[1], &index) || !as_int64(a[2], &width) ||
      !as_pointer(a[8], &stream) || !nodes_of(a[3], nodes) || !ints_of(a[4], first))
    return nullptr;
  const size_t n = nodes.size() / 2;
  if (a[5] == Py_None) counts.assign(n, 1);
  else if (!ints_of(a[5], counts)) return nullptr;
  if (!exactly(first, n, "first") || !exactly(counts, n, "counts")) return nullptr;
  for (int32_t c : counts) rows += c;
  if (!rows_of(a[6], "K", rows, width, g_bf16, index, &K) || !rows_of(a[7], "V", rows, width, g_bf16, index, &V))
    return nullptr;
  return call([&] {
    return g_write(static_cast<wave_kv*>(h), (int32_t)n, as_nodes(nodes), first.data(), counts.data(), K.p, K.ld, V.p,
                   V.ld, stream);
  });
} catch (const std::bad_alloc&) {
  return PyErr_NoMemory();
}

// token_attn(handle, device, d, active, policy, Q, O, own_tokens, lse, workspace, stream)
PyObject* token_attn(PyObject*, PyObject* const* a, Py_ssize_t count) try {
  void *h, *stream;
  int64_t index, d, rows, qh, ws = 0, bytes = 0;
  int32_t policy;
  std::vector<int32_t> nodes, own;
  Rows Q, O, lse{nullptr, 0};
  if (!counted(count, 11) || !as_pointer(a[0], &h) || !as_int64(a[1], &index) || !as_int64(a[2], &d) ||
      !as_int32(a[4], &policy) || !as_pointer(a[10], &stream) || !nodes_of(a[3], nodes) ||
      !heads_of(a[5], "Q", d, &rows, &qh))
    return nullptr;
  const int64_t n = (int64_t)nodes.size() / 2;
  if (a[7] != Py_None && (!ints_of(a[7], own) || !exactly(own, (size_t)n, "own_tokens"))) return nullptr;
  if (!rows_of(a[5], "Q", n, qh * d, g_bf16, index, &Q) || !rows_of(a[6], "O", n, qh * d, g_bf16, index, &O)) return nullptr;
  if (a[8] != Py_None && (!rows_of(a[8], "lse", n, qh, g_f32, index, &lse) || !contiguous(lse, n, qh, "lse")))
    return nullptr;
  if (a[9] != Py_None) {
    int64_t device, flat;
    if (!ask(a[9], s_device, &device) || !ask(a[9], s_contiguous, &flat)) return nullptr;
    if (device != index || !flat) {
      PyErr_Format(PyExc_ValueError, "workspace: a contiguous tensor on cuda:%lld is wanted", (long long)index);
      return nullptr;
    }
    PyObject* size = PyObject_GetAttr(a[9], s_nbytes);
    if (!size) return nullptr;
    const bool ok = as_int64(size, &bytes);
    Py_DECREF(size);
    if (!ok || !ask(a[9], s_ptr, &ws)) return nullptr;
  }
  return call([&] {
    return g_attn(static_cast<wave_kv*>(h), as_nodes(nodes), (int32_t)n, policy, a[7] == Py_None ? nullptr : own.data(),
                  (int32_t)qh, Q.p, Q.ld, O.p, O.ld, static_cast<float*>(lse.p),
                  reinterpret_cast<void*>((intptr_t)ws), (uint64_t)bytes, stream);
  });
} catch (const std::bad_alloc&) {
  return PyErr_NoMemory();
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef g_methods[] = {
    {"bind", fast(bind), METH_FASTCALL, nullptr},
    {"linear_bias", fast(linear_bias), METH_FASTCALL, nullptr},
    {"rotary", fast(rotary), METH_FASTCALL, nullptr},
    {"write_tokens", fast(write_tokens), METH_FASTCALL, nullptr},
    {"token_attn", fast(token_attn), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_call", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__call() {
  const struct {
    PyObject** at;
    const char* name;
  } names[] = {{&s_shape, "shape"},    {&s_stride, "stride"},     {&s_dtype, "dtype"},  {&s_device, "get_device"},
               {&s_ptr, "data_ptr"},   {&s_contiguous, "is_contiguous"}, {&s_nbytes, "nbytes"}};
  for (const auto& n : names)
    if (!(*n.at = PyUnicode_InternFromString(n.name))) return nullptr;
  return PyModule_Create(&g_module);
}
