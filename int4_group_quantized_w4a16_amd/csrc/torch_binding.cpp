// The Python call path of the serving operators: tensors in, tensor out.
//
// A call of a few microseconds on the GPU must not spend ten on the way there:
// attribute checks in Python, ctypes conversions and torch.empty cost 9-10 us
// per call (measured on the append and linear decode steps), this module about
// 1 us on top of the launch.  It holds no arithmetic and no checks of its own
// beyond "this is an ordinary valid call": anything else, a refusal by the C
// ABI included, returns None, and the full checks in __init__.py then say what
// is wrong.
//
// The entry points are those of the libkaio.so that __init__.py loaded; their
// addresses are handed over by bind().

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/kaio.h"

namespace {

decltype(&kaio_linear_w4a16) g_linear;
decltype(&kaio_rope_append) g_rope;
decltype(&kaio_paged_attention) g_attention;
decltype(&kaio_paged_attention_workspace_size) g_workspace;

// the tensor behind obj, or null if it is not one that the fast path takes
const at::Tensor* tensor(PyObject* obj, at::ScalarType type, int64_t rank, int device) {
  if (!THPVariable_Check(obj)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(obj);
  if (!t.defined() || !t.is_cuda() || t.scalar_type() != type || t.dim() != rank || t.get_device() != device ||
      !t.is_contiguous())
    return nullptr;
  return &t;
}

bool fits(int64_t v) { return v >= 0 && v < (int64_t(1) << 31); }

// stream of an ordinary call: the current one of the current device, if that is the tensors' device
bool stream_of(int device, void** out) {
  if (c10::hip::current_device() != device) return false;
  *out = c10::hip::getCurrentHIPStream(device).stream();
  return true;
}

PyObject* none() { Py_RETURN_NONE; }

template <typename F>
PyObject* guarded(F body) {   // no C++ exception leaves the module
  try {
    return body();
  } catch (...) {
    return none();
  }
}

// linear(x, w, s, bias | None, activation code, residual | None, y | None)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 7 || !g_linear || !THPVariable_Check(a[0])) return none();
    const at::Tensor& x0 = THPVariable_Unpack(a[0]);
    if (!x0.defined() || !x0.is_cuda()) return none();
    const int dev = x0.get_device();
    const at::Tensor *x = tensor(a[0], at::kHalf, 2, dev), *w = tensor(a[1], at::kInt, 2, dev),
                     *s = tensor(a[2], at::kHalf, 2, dev), *b = nullptr, *r = nullptr;
    if (!x || !w || !s) return none();
    const int64_t M = x->size(0), K = x->size(1), N = w->size(1);
    if (K % 128 || w->size(0) != K / 8 || s->size(0) != K / 128 || s->size(1) != N || !fits(M) || !fits(N) || !fits(K))
      return none();
    if (a[3] != Py_None && (!(b = tensor(a[3], at::kHalf, 1, dev)) || b->size(0) != N)) return none();
    if (a[5] != Py_None && (!(r = tensor(a[5], at::kHalf, 2, dev)) || r->size(0) != M || r->size(1) != N)) return none();
    const long act = PyLong_AsLong(a[4]);
    if (act < 0) {
      PyErr_Clear();
      return none();
    }
    void* stream;
    if (!stream_of(dev, &stream)) return none();
    at::Tensor made;
    const at::Tensor* y;
    if (a[6] == Py_None) {
      made = at::empty({M, N}, x->options());
      y = &made;
    } else if (!(y = tensor(a[6], at::kHalf, 2, dev)) || y->size(0) != M || y->size(1) != N) {
      return none();
    }
    if (g_linear(x->data_ptr(), static_cast<const uint32_t*>(w->data_ptr()), s->data_ptr(), b ? b->data_ptr() : nullptr,
                 r ? r->data_ptr() : nullptr, y->data_ptr(), (uint32_t)M, (uint32_t)N, (uint32_t)K, 128,
                 static_cast<kaio_activation>(act), stream) != KAIO_OK)
      return none();
    if (a[6] == Py_None) return THPVariable_Wrap(std::move(made));
    Py_INCREF(a[6]);
    return a[6];
  });
}

const kaio_paged_kv* paged_of(PyObject* address) {
  void* p = PyLong_AsVoidPtr(address);
  if (!p) PyErr_Clear();
  return static_cast<const kaio_paged_kv*>(p);
}
at::ScalarType type_of(const kaio_paged_kv& kv) { return kv.dtype == KAIO_DTYPE_BF16 ? at::kBFloat16 : at::kHalf; }

const at::Tensor* heads(PyObject* obj, const kaio_paged_kv& kv, int device) {
  const at::Tensor* t = tensor(obj, type_of(kv), 3, device);
  return t && t->size(2) == kv.head_dim && fits(t->size(0)) && fits(t->size(1)) ? t : nullptr;
}

// rope_append(q, k, v, positions, inv_freq, sections, kv address, device, interleaved, q_out | None)
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 10 || !g_rope) return none();
    const kaio_paged_kv* kv = paged_of(a[6]);
    const int dev = (int)PyLong_AsLong(a[7]);
    if (!kv) return none();
    const at::Tensor *q = heads(a[0], *kv, dev), *k = heads(a[1], *kv, dev), *v = heads(a[2], *kv, dev),
                     *pos = tensor(a[3], at::kInt, 2, dev), *inv = tensor(a[4], at::kDouble, 1, dev);
    if (!q || !k || !v || !pos || !inv) return none();
    const int64_t T = q->size(0), hkv = kv->kv_heads;
    if (k->size(0) != T || v->size(0) != T || k->size(1) != hkv || v->size(1) != hkv) return none();
    if (!PyList_Check(a[5]) && !PyTuple_Check(a[5])) return none();
    const Py_ssize_t axes = PySequence_Fast_GET_SIZE(a[5]);
    if (axes < 1 || axes > 8 || pos->size(0) != axes || pos->size(1) != T) return none();
    uint32_t sections[8];
    int64_t sum = 0;
    for (Py_ssize_t i = 0; i < axes; ++i) {
      const long c = PyLong_AsLong(PySequence_Fast_GET_ITEM(a[5], i));
      if (c < 0 || c > 4096) {
        PyErr_Clear();
        return none();
      }
      sections[i] = (uint32_t)c;
      sum += c;
    }
    if (sum != inv->size(0)) return none();
    void* stream;
    if (!stream_of(dev, &stream)) return none();
    at::Tensor made;
    const at::Tensor* out;
    if (a[9] == Py_None) {
      made = at::empty_like(*q);
      out = &made;
    } else if (!(out = heads(a[9], *kv, dev)) || out->sizes() != q->sizes()) {
      return none();
    }
    if (g_rope(kv, q->data_ptr(), k->data_ptr(), v->data_ptr(), static_cast<const int32_t*>(pos->data_ptr()),
               static_cast<const double*>(inv->data_ptr()), sections, (uint32_t)axes, a[8] == Py_True, out->data_ptr(),
               (uint32_t)T, (uint32_t)q->size(1), stream) != KAIO_OK)
      return none();
    if (a[9] == Py_None) return THPVariable_Wrap(std::move(made));
    Py_INCREF(a[9]);
    return a[9];
  });
}

// attention(q, kv address, device, max_new, scale, window, sinks, out | None, workspace | None)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 9 || !g_attention) return none();
    const kaio_paged_kv* kv = paged_of(a[1]);
    const int dev = (int)PyLong_AsLong(a[2]);
    const long max_new = PyLong_AsLong(a[3]), window = PyLong_AsLong(a[5]), sinks = PyLong_AsLong(a[6]);
    const double scale = PyFloat_AsDouble(a[4]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return none();
    }
    if (!kv || kv->kv_heads == 0 || !fits(max_new) || !fits(window) || !fits(sinks)) return none();
    const at::Tensor* q = heads(a[0], *kv, dev);
    if (!q || q->size(1) % kv->kv_heads) return none();
    const uint32_t T = (uint32_t)q->size(0), hq = (uint32_t)q->size(1);
    void* stream;
    if (!stream_of(dev, &stream)) return none();
    at::Tensor made, scratch;
    const at::Tensor *out, *ws = nullptr;
    if (a[7] == Py_None) {
      made = at::empty_like(*q);
      out = &made;
    } else if (!(out = heads(a[7], *kv, dev)) || out->sizes() != q->sizes()) {
      return none();
    }
    const size_t need = g_workspace(kv, T, hq, (uint32_t)max_new);
    if (a[8] != Py_None) {
      if (!(ws = tensor(a[8], at::kByte, 1, dev))) return none();
    } else if (need) {
      scratch = at::empty({(int64_t)need}, q->options().dtype(at::kByte));
      ws = &scratch;
    }
    if (g_attention(kv, q->data_ptr(), out->data_ptr(), T, hq, (uint32_t)max_new, (float)scale, (uint32_t)window,
                    (uint32_t)sinks, ws ? ws->data_ptr() : nullptr, ws ? (size_t)ws->numel() : 0, stream) != KAIO_OK)
      return none();
    if (a[7] == Py_None) return THPVariable_Wrap(std::move(made));
    Py_INCREF(a[7]);
    return a[7];
  });
}

// bind(linear, rope_append, paged_attention, workspace_size): addresses of the C entry points
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
    return nullptr;
  }
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_linear = reinterpret_cast<decltype(g_linear)>(p[0]);
  g_rope = reinterpret_cast<decltype(g_rope)>(p[1]);
  g_attention = reinterpret_cast<decltype(g_attention)>(p[2]);
  g_workspace = reinterpret_cast<decltype(g_workspace)>(p[3]);
  return none();
}

#define KAIO_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KAIO_METHOD(linear), KAIO_METHOD(rope_append), KAIO_METHOD(attention), KAIO_METHOD(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  // the torch whose headers this was compiled with: tensors of another one need not be laid out alike
  if (m && PyModule_AddStringConstant(m, "torch_version", KAIO_TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
