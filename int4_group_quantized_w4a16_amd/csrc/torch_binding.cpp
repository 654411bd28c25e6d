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
decltype(&kaio_quantize_rows) g_quantize;
decltype(&kaio_linear_w8a8) g_linear8;
decltype(&kaio_linear_w8a8_workspace_size) g_linear8_workspace;
decltype(&kaio_moe_w4a16) g_moe;
decltype(&kaio_moe_w4a16_workspace_size) g_moe_workspace;

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

// the tensor behind obj, of the given shape; absent: obj is None
const at::Tensor* shaped(PyObject* obj, at::ScalarType type, at::IntArrayRef shape, int device) {
  const at::Tensor* t = tensor(obj, type, (int64_t)shape.size(), device);
  return t && t->sizes() == shape ? t : nullptr;
}
bool optional(PyObject* obj, at::ScalarType type, at::IntArrayRef shape, int device, const at::Tensor** out) {
  *out = nullptr;
  return obj == Py_None || (*out = shaped(obj, type, shape, device));
}
// the caller's tensor, or one made here
bool output(PyObject* obj, at::ScalarType type, at::IntArrayRef shape, const at::Tensor& like, at::Tensor* made,
            const at::Tensor** out) {
  if (obj != Py_None) return (*out = shaped(obj, type, shape, like.get_device())) != nullptr;
  *made = at::empty(shape, like.options().dtype(type));
  *out = made;
  return true;
}
bool scratch_of(PyObject* obj, size_t need, const at::Tensor& like, at::Tensor* made, const at::Tensor** out) {
  *out = nullptr;
  if (obj != Py_None) return (*out = tensor(obj, at::kByte, 1, like.get_device())) != nullptr;
  if (need) {
    *made = at::empty({(int64_t)need}, like.options().dtype(at::kByte));
    *out = made;
  }
  return true;
}
PyObject* result(PyObject* given, at::Tensor&& made) {
  if (given == Py_None) return THPVariable_Wrap(std::move(made));
  Py_INCREF(given);
  return given;
}
void* data(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
bool half_type(const at::Tensor& t) { return t.scalar_type() == at::kHalf || t.scalar_type() == at::kBFloat16; }
kaio_dtype dtype_of(at::ScalarType t) { return t == at::kHalf ? KAIO_DTYPE_F16 : KAIO_DTYPE_BF16; }

// quantize_rows(x, q | None, scale | None)
PyObject* quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 3 || !g_quantize || !THPVariable_Check(a[0])) return none();
    const at::Tensor& x = THPVariable_Unpack(a[0]);
    if (!x.defined() || !x.is_cuda() || !half_type(x) || x.dim() != 2 || !x.is_contiguous()) return none();
    const int64_t M = x.size(0), K = x.size(1);
    if (!fits(M) || !fits(K)) return none();
    void* stream;
    if (!stream_of(x.get_device(), &stream)) return none();
    at::Tensor made_q, made_s;
    const at::Tensor *q, *s;
    if (!output(a[1], at::kChar, {M, K}, x, &made_q, &q) || !output(a[2], at::kFloat, {M}, x, &made_s, &s)) return none();
    if (g_quantize(dtype_of(x.scalar_type()), x.data_ptr(), static_cast<int8_t*>(q->data_ptr()),
                   static_cast<float*>(s->data_ptr()), (uint32_t)M, (uint32_t)K, stream) != KAIO_OK)
      return none();
    PyObject *pq = result(a[1], std::move(made_q)), *ps = result(a[2], std::move(made_s));
    PyObject* both = PyTuple_Pack(2, pq, ps);
    Py_XDECREF(pq);
    Py_XDECREF(ps);
    return both;
  });
}

// linear8(x, w, w_scale, x_scale | None, bias | None, activation code, residual | None, y | None, workspace | None);
PyObject* linear8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 9 || !g_linear8 || !THPVariable_Check(a[0])) return none();
    const at::Tensor& x = THPVariable_Unpack(a[0]);
    if (!x.defined() || !x.is_cuda() || x.dim() != 2 || !x.is_contiguous()) return none();
    const int dev = x.get_device();
    const bool rounded = a[3] != Py_None;
    at::ScalarType type = x.scalar_type();
    if (rounded) {   // the type of y, residual or bias, the first that is there
      if (type != at::kChar) return none();
      PyObject* const of = a[7] != Py_None ? a[7] : a[6] != Py_None ? a[6] : a[4];
      if (of != Py_None && !THPVariable_Check(of)) return none();
      type = of == Py_None ? at::kHalf : THPVariable_Unpack(of).scalar_type();
    }
    if (type != at::kHalf && type != at::kBFloat16) return none();
    const at::Tensor* w = tensor(a[1], at::kChar, 2, dev);
    if (!w) return none();
    const int64_t M = x.size(0), K = x.size(1), N = w->size(0);
    if (w->size(1) != K || !fits(M) || !fits(N) || !fits(K)) return none();
    const at::Tensor *ws = shaped(a[2], at::kFloat, {N}, dev), *xs, *b, *r, *y, *scratch;
    if (!ws || !optional(a[3], at::kFloat, {M}, dev, &xs) || !optional(a[4], type, {N}, dev, &b) ||
        !optional(a[6], type, {M, N}, dev, &r))
      return none();
    const long act = PyLong_AsLong(a[5]);
    if (act < 0) {
      PyErr_Clear();
      return none();
    }
    void* stream;
    if (!stream_of(dev, &stream)) return none();
    at::Tensor made, made_scratch;
    const size_t need = g_linear8_workspace((uint32_t)M, (uint32_t)N, (uint32_t)K, rounded);
    if (!output(a[7], type, {M, N}, x, &made, &y) || !scratch_of(a[8], need, x, &made_scratch, &scratch)) return none();
    if (g_linear8(dtype_of(type), x.data_ptr(), static_cast<const float*>(data(xs)), static_cast<const int8_t*>(w->data_ptr()),
                  static_cast<const float*>(ws->data_ptr()), data(b), data(r), y->data_ptr(), (uint32_t)M, (uint32_t)N,
                  (uint32_t)K, static_cast<kaio_activation>(act), data(scratch), scratch ? (size_t)scratch->numel() : 0,
                  stream) != KAIO_OK)
      return none();
    return result(a[7], std::move(made));
  });
}

// moe(x, experts address, device, top_k, normalize, activation code, residual | None, y | None, workspace | None)
PyObject* moe(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 9 || !g_moe) return none();
    const auto* e = static_cast<const kaio_experts*>(PyLong_AsVoidPtr(a[1]));
    const int dev = (int)PyLong_AsLong(a[2]);
    const long top = PyLong_AsLong(a[3]), act = PyLong_AsLong(a[5]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return none();
    }
    if (!e || top < 1 || !fits(top) || act < 0) return none();
    const at::Tensor* x = tensor(a[0], at::kHalf, 2, dev);
    if (!x || x->size(1) != e->hidden || !fits(x->size(0))) return none();
    const uint32_t T = (uint32_t)x->size(0);
    const at::Tensor *r, *y, *scratch;
    if (!optional(a[6], at::kHalf, x->sizes(), dev, &r)) return none();
    void* stream;
    if (!stream_of(dev, &stream)) return none();
    at::Tensor made, made_scratch;
    const size_t need = g_moe_workspace(e, T, (uint32_t)top);
    if (!output(a[7], at::kHalf, x->sizes(), *x, &made, &y) || !scratch_of(a[8], need, *x, &made_scratch, &scratch)) return none();
    if (g_moe(e, x->data_ptr(), data(r), y->data_ptr(), T, (uint32_t)top, a[4] == Py_True, static_cast<kaio_activation>(act),
              data(scratch), scratch ? (size_t)scratch->numel() : 0, stream) != KAIO_OK)
      return none();
    return result(a[7], std::move(made));
  });
}

// bind(linear, rope_append, paged_attention, its workspace size, quantize_rows, linear_w8a8, its workspace size,
// moe_w4a16, its workspace size): addresses of the C entry points
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr Py_ssize_t kEntries = 9;
  if (n != kEntries) {
    PyErr_SetString(PyExc_TypeError, "bind takes nine addresses");
    return nullptr;
  }
  void* p[kEntries];
  for (int i = 0; i < kEntries; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_linear = reinterpret_cast<decltype(g_linear)>(p[0]);
  g_rope = reinterpret_cast<decltype(g_rope)>(p[1]);
  g_attention = reinterpret_cast<decltype(g_attention)>(p[2]);
  g_workspace = reinterpret_cast<decltype(g_workspace)>(p[3]);
  g_quantize = reinterpret_cast<decltype(g_quantize)>(p[4]);
  g_linear8 = reinterpret_cast<decltype(g_linear8)>(p[5]);
  g_linear8_workspace = reinterpret_cast<decltype(g_linear8_workspace)>(p[6]);
  g_moe = reinterpret_cast<decltype(g_moe)>(p[7]);
  g_moe_workspace = reinterpret_cast<decltype(g_moe_workspace)>(p[8]);
  return none();
}

#define KAIO_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KAIO_METHOD(linear), KAIO_METHOD(rope_append), KAIO_METHOD(attention),
                         KAIO_METHOD(quantize_rows), KAIO_METHOD(linear8), KAIO_METHOD(moe), KAIO_METHOD(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  // the torch whose headers this was compiled with: tensors of another one need not be laid out alike
  if (m && PyModule_AddStringConstant(m, "torch_version", KAIO_TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
