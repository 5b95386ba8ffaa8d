// call.cpp -- the serving calls of the Python binding, natively.
//
// A call on a short cache takes 5 to 10 us on the device; reading nine tensors
// through Python, two allocations and a foreign call with two dozen arguments
// took 12 us of the host's time beside the 5 of the library. Here the accepted
// call costs 2 to 4 (one short decode 17.8 -> 9.8 us a call, an eviction in
// given buffers 15.4 -> 6.8): the arguments are read from the tensors themselves, the
// outputs allocated and the C entry point called on the tensors' device and its
// current stream.
//
// Each function returns None where anything about the arguments is not plainly
// right (or the library refuses them); psa.py then goes through the same call
// in Python, which says what is wrong. It never raises by itself.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <climits>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "psa.h"

namespace {

struct Library {
  decltype(&psa_decode) decode = nullptr;
  decltype(&psa_decode_workspace_size) decode_size = nullptr;
  decltype(&psa_key_weight) weight = nullptr;
  decltype(&psa_key_weight_workspace_size) weight_size = nullptr;
  decltype(&psa_cache_evict) evict = nullptr;
  decltype(&psa_cache_evict_workspace_size) evict_size = nullptr;
} g;

// The tensor of a Python object that is exactly a contiguous CUDA tensor.
const at::Tensor* tensor(PyObject* o) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.defined() && t.is_cuda() && t.layout() == at::kStrided && t.is_contiguous() ? &t : nullptr;
}

// One call's problem: device, and whether all arguments so far were right.
struct Args {
  const at::Tensor* like = nullptr;
  bool ok = true;

  // A 4-dimensional tensor's sizes.
  const at::Tensor* first(PyObject* o, int (&n)[4]) {
    const at::Tensor* t = tensor(o);
    if (!t || t->dim() != 4 || (like && t->device() != like->device())) {
      ok = false;
      return nullptr;
    }
    for (int i = 0; i < 4; ++i) {
      if (t->size(i) > INT_MAX) ok = false;
      n[i] = static_cast<int>(t->size(i));
    }
    return t;
  }
  // The address of an argument of this shape and type; None stays null.
  template <typename T = void>
  T* at(PyObject* o, at::IntArrayRef shape, at::ScalarType type) {
    if (o == Py_None || !ok) return nullptr;
    const at::Tensor* t = tensor(o);
    if (!t || t->scalar_type() != type || t->device() != like->device() || t->sizes() != shape) {
      ok = false;
      return nullptr;
    }
    return static_cast<T*>(t->data_ptr());
  }
  // The workspace given, or a new one of `need` bytes (held by `own`).
  char* workspace(PyObject* o, size_t need, at::Tensor& own, size_t& bytes) {
    if (!ok) return nullptr;
    if (o == Py_None) {
      if (need == 0) {
        ok = false;
        return nullptr;
      }
      own = at::empty({static_cast<int64_t>(need)}, like->options().dtype(at::kByte));
      bytes = need;
      return static_cast<char*>(own.data_ptr());
    }
    const at::Tensor* t = tensor(o);
    if (!t || t->scalar_type() != at::kByte || t->device() != like->device() ||
        static_cast<size_t>(t->numel()) < need) {
      ok = false;
      return nullptr;
    }
    bytes = static_cast<size_t>(t->numel());
    return static_cast<char*>(t->data_ptr());
  }
};

// psa_dtype of a 16-bit tensor, or -1.
int dtype16(const at::Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? PSA_BF16 : (t.scalar_type() == at::kHalf ? PSA_FP16 : -1);
}

// The stream that is current on the tensors' device, if that device is the current one.
bool stream_of(const at::Tensor& t, void*& stream) {
  if (c10::cuda::current_device() != t.get_device()) return false;
  stream = c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
  return true;
}

bool to_int(PyObject* o, int& v) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  const long n = PyLong_AsLongAndOverflow(o, &over);
  if (over || n < INT_MIN || n > INT_MAX) return false;
  v = static_cast<int>(n);
  return true;
}

PyObject* keep(PyObject* given, const at::Tensor& made) {
  return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(given);
}

// decode(q, k_cache, v_cache, cache_len, k_prefix, v_prefix, prefix_len, ws, out, lse, want_lse)
PyObject* decode_call(PyObject* const* a) {
  Args x;
  int n[4], kn[4], pn[4];
  const at::Tensor* q = x.first(a[0], n);
  if (!q) return nullptr;
  x.like = q;
  const int dt = dtype16(*q);
  const int B = n[0], Hq = n[1], T = n[2], d = n[3];
  int Bp = 1, P = 0, C = 0, Hkv = 0;
  if (a[4] != Py_None) {
    if (!x.first(a[4], pn) || a[5] == Py_None) return nullptr;
    Bp = pn[0], Hkv = pn[1], P = pn[2];
  } else if (a[5] != Py_None || a[6] != Py_None) {
    return nullptr;
  }
  if (a[1] != Py_None) {
    if (!x.first(a[1], kn) || a[2] == Py_None) return nullptr;
    C = kn[2];
    if (Hkv == 0) Hkv = kn[1];
  } else if (a[2] != Py_None || a[3] != Py_None || a[4] == Py_None) {
    return nullptr;
  }
  if (dt < 0 || !x.ok) return nullptr;
  const at::ScalarType type = q->scalar_type();
  const int64_t pre[4] = {Bp, Hkv, P, d}, own[4] = {B, Hkv, C, d}, rows[3] = {B, Hq, T}, nb[1] = {B}, np[1] = {Bp};
  const void* kp = x.at(a[4], pre, type);
  const void* vp = x.at(a[5], pre, type);
  const int* plen = x.at<int>(a[6], np, at::kInt);
  const void* kc = x.at(a[1], own, type);
  const void* vc = x.at(a[2], own, type);
  const int* clen = x.at<int>(a[3], nb, at::kInt);
  at::Tensor ws_own, out_own, lse_own;
  size_t bytes = 0;
  void* out = x.at(a[8], q->sizes(), type);
  float* lse = x.at<float>(a[9], rows, at::kFloat);
  const int want = PyObject_IsTrue(a[10]);
  void* stream = nullptr;
  if (!x.ok || want < 0 || !stream_of(*q, stream)) return nullptr;
  char* ws = x.workspace(a[7], g.decode_size(B, Hq, Hkv, T, d, Bp, P, C), ws_own, bytes);
  if (!x.ok) return nullptr;
  if (a[8] == Py_None) {
    out_own = at::empty_like(*q);
    out = out_own.data_ptr();
  }
  if (a[9] == Py_None && want) {
    lse_own = at::empty(rows, q->options().dtype(at::kFloat));
    lse = static_cast<float*>(lse_own.data_ptr());
  }
  int status;
  const void* qp = q->data_ptr();
  Py_BEGIN_ALLOW_THREADS;
  status = g.decode(qp, kp, vp, plen, kc, vc, clen, B, Hq, Hkv, T, d, Bp, P, C, dt, out, lse, ws, bytes, stream);
  Py_END_ALLOW_THREADS;
  if (status != PSA_OK) return nullptr;
  PyObject* o = keep(a[8], out_own);
  if (!o || (a[9] == Py_None && !want)) return o;
  PyObject* l = keep(a[9], lse_own);
  if (!l) {
    Py_DECREF(o);
    return nullptr;
  }
  PyObject* both = PyTuple_New(2);
  if (!both) {
    Py_DECREF(o);
    Py_DECREF(l);
    return nullptr;
  }
  PyTuple_SET_ITEM(both, 0, o);
  PyTuple_SET_ITEM(both, 1, l);
  return both;
}

// key_weight(q, k, lse, key_len, causal, score, ws, out)
PyObject* weight_call(PyObject* const* a) {
  Args x;
  int n[4], kn[4];
  const at::Tensor* q = x.first(a[0], n);
  if (!q) return nullptr;
  x.like = q;
  if (!x.first(a[1], kn) || !x.ok || a[2] == Py_None) return nullptr;
  const int dt = dtype16(*q), B = n[0], Hq = n[1], T = n[2], d = n[3], Bk = kn[0], Hkv = kn[1], C = kn[2];
  if (dt < 0) return nullptr;
  const int64_t keys[4] = {Bk, Hkv, C, d}, slots[3] = {Bk, Hkv, C}, rows[3] = {B, Hq, T}, nk[1] = {Bk};
  const void* k = x.at(a[1], keys, q->scalar_type());
  const float* lse = x.at<float>(a[2], rows, at::kFloat);
  const int* len = x.at<int>(a[3], nk, at::kInt);
  const int causal = a[4] == Py_True ? 1 : (a[4] == Py_False ? 0 : -1);  // (psa.py says what else counts as one)
  const float* score = x.at<float>(a[5], slots, at::kFloat);
  float* out = x.at<float>(a[7], slots, at::kFloat);
  at::Tensor ws_own, out_own;
  size_t bytes = 0;
  void* stream = nullptr;
  if (!x.ok || causal < 0 || !stream_of(*q, stream)) return nullptr;
  char* ws = x.workspace(a[6], g.weight_size(B, Hq, Hkv, T, d, Bk, C), ws_own, bytes);
  if (!x.ok) return nullptr;
  if (a[7] == Py_None) {
    out_own = at::empty(slots, q->options().dtype(at::kFloat));
    out = static_cast<float*>(out_own.data_ptr());
  }
  int status;
  const void* qp = q->data_ptr();
  Py_BEGIN_ALLOW_THREADS;
  status = g.weight(qp, k, lse, len, score, B, Hq, Hkv, T, d, Bk, C, causal, dt, out, ws, bytes, stream);
  Py_END_ALLOW_THREADS;
  return status == PSA_OK ? keep(a[7], out_own) : nullptr;
}

// cache_evict(k, v, score, budget, pos, cache_len, sink, recent, ws, out): `out` is the tuple of six buffers
PyObject* evict_call(PyObject* const* a) {
  Args x;
  int n[4], on[4], budget, sink, recent;
  const at::Tensor* k = x.first(a[0], n);
  if (!k) return nullptr;
  x.like = k;
  if (!x.ok || dtype16(*k) < 0 || a[1] == Py_None || a[2] == Py_None || !to_int(a[3], budget) ||
      !to_int(a[6], sink) || !to_int(a[7], recent) || budget <= 0)
    return nullptr;
  const int B = n[0], Hkv = n[1], C = n[2], d = n[3];
  const at::ScalarType type = k->scalar_type();
  const int64_t slots[3] = {B, Hkv, C}, nb[1] = {B}, kb[3] = {B, Hkv, budget};
  const void* v = x.at(a[1], k->sizes(), type);
  const float* score = x.at<float>(a[2], slots, at::kFloat);
  const int* pos = x.at<int>(a[4], slots, at::kInt);
  const int* len = x.at<int>(a[5], nb, at::kInt);
  const size_t need = g.evict_size(B, Hkv, C, budget);
  void* stream = nullptr;
  if (!x.ok || need == 0 || !stream_of(*k, stream)) return nullptr;
  at::Tensor ws_own;
  size_t bytes = 0;
  char* ws = x.workspace(a[8], need, ws_own, bytes);
  if (!x.ok) return nullptr;
  PyObject* out;
  if (a[9] == Py_None) {
    const int64_t rows[4] = {B, Hkv, budget, d};
    const at::TensorOptions o = k->options();
    const at::Tensor made[6] = {at::empty(rows, o),
                                at::empty(rows, o),
                                at::empty(kb, o.dtype(at::kFloat)),
                                at::empty(kb, o.dtype(at::kInt)),
                                at::empty(nb, o.dtype(at::kInt)),
                                at::empty(kb, o.dtype(at::kInt))};
    out = PyTuple_New(6);
    for (int i = 0; out && i < 6; ++i) {
      PyObject* t = THPVariable_Wrap(made[i]);
      if (!t) Py_CLEAR(out);
      if (out) PyTuple_SET_ITEM(out, i, t);
    }
    if (!out) return nullptr;
  } else {
    if (!PyTuple_CheckExact(a[9]) || PyTuple_GET_SIZE(a[9]) != 6) return nullptr;
    out = Py_NewRef(a[9]);
  }
  PyObject* buf[6];
  for (int i = 0; i < 6; ++i) {
    buf[i] = PyTuple_GET_ITEM(out, i);
    if (buf[i] == Py_None) x.ok = false;
  }
  if (x.ok) x.first(buf[0], on);
  int status = PSA_ERR_ARG;
  if (x.ok) {
    const int C_out = on[2];
    const int64_t rows[4] = {B, Hkv, C_out, d}, places[3] = {B, Hkv, C_out};
    void* ko = x.at(buf[0], rows, type);
    void* vo = x.at(buf[1], rows, type);
    float* so = x.at<float>(buf[2], places, at::kFloat);
    int* po = x.at<int>(buf[3], places, at::kInt);
    int* lo = x.at<int>(buf[4], nb, at::kInt);
    int* kept = x.at<int>(buf[5], kb, at::kInt);
    const void* kp = k->data_ptr();
    if (x.ok) {
      Py_BEGIN_ALLOW_THREADS;
      status = g.evict(kp, v, score, pos, len, B, Hkv, C, d, budget, sink, recent, C_out, ko, vo, so, po, lo, kept, ws,
                       bytes, stream);
      Py_END_ALLOW_THREADS;
    }
  }
  if (status != PSA_OK) Py_CLEAR(out);
  return out;
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  PyObject* r = nullptr;
  try {
    if (n == N && g.decode) r = F(a);
  } catch (const std::exception&) {
    r = nullptr;  // (a tensor without storage, an allocation that failed: psa.py meets it again)
  }
  if (r) return r;
  PyErr_Clear();
  Py_RETURN_NONE;
}

// bind(six addresses): the entry points of the loaded library, in Library's order.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = n == 6 ? PyLong_AsVoidPtr(a[i]) : nullptr;
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "six addresses are required");
      return nullptr;
    }
  }
  g.decode = reinterpret_cast<decltype(g.decode)>(p[0]);
  g.decode_size = reinterpret_cast<decltype(g.decode_size)>(p[1]);
  g.weight = reinterpret_cast<decltype(g.weight)>(p[2]);
  g.weight_size = reinterpret_cast<decltype(g.weight_size)>(p[3]);
  g.evict = reinterpret_cast<decltype(g.evict)>(p[4]);
  g.evict_size = reinterpret_cast<decltype(g.evict_size)>(p[5]);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"bind", fast(bind), METH_FASTCALL, nullptr},
    {"decode", fast(call<decode_call, 11>), METH_FASTCALL, nullptr},
    {"key_weight", fast(call<weight_call, 8>), METH_FASTCALL, nullptr},
    {"cache_evict", fast(call<evict_call, 10>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the PyTorch and Python whose layouts are compiled in (psa.py uses
// the module with no other)
PyMODINIT_FUNC PyInit__call() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", PSA_BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
