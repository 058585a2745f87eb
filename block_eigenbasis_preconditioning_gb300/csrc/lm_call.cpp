// The ordinary calls of layer norm, distillation and sampling for the
// interpreter: outputs, workspace and launch in one native call.  A call on a few
// rows takes the GPU 5 us; allocations through Python's torch.empty and the
// argument conversion of ctypes alone take 6 to 14 us.
//
// Each function takes the tensors on the current device and stream with all
// outputs left to it, and gives the new tensors.  It gives None for whatever else
// it is handed and for what the library refuses: lm.py's own way then takes the
// call, or says what is wrong with it.
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>

#include "dobb.h"

namespace {

using at::Tensor;

// A call's tensors, numbers and stream; ok turns false at the first thing that is not
// as the call has to be.
struct Call {
  bool ok = true;
  int device = -1;  // the current one, asked for at the first tensor on a GPU

  bool want(bool c) { return ok = ok && c; }

  // a tensor on the current device; none: None may stand for it
  const Tensor* tensor(PyObject* o, bool none = false) {
    if (none && o == Py_None) return nullptr;
    if (!want(THPVariable_Check(o))) return nullptr;
    const Tensor& t = THPVariable_Unpack(o);
    if (!want(t.is_cuda() && t.layout() == at::kStrided)) return nullptr;
    if (device < 0) device = c10::cuda::current_device();
    want(t.get_device() == device);
    return &t;
  }
  dobb_dtype dtype(at::ScalarType t) {
    want(t == at::kFloat || t == at::kBFloat16);
    return t == at::kFloat ? DOBB_F32 : DOBB_BF16;
  }
  // the row stride of a matrix with contiguous rows
  int64_t rows(const Tensor& t) {
    if (!want(t.dim() == 2)) return 0;
    const int64_t n = t.size(0), cols = t.size(1);
    want((cols <= 1 || t.stride(1) == 1) && (n <= 1 || t.stride(0) >= cols));
    return n <= 1 ? std::max(t.stride(0), cols) : t.stride(0);
  }
  void* vector(const Tensor* t, int64_t n, at::ScalarType type) {
    if (!t || !want(t->numel() == n && t->is_contiguous() && t->scalar_type() == type)) return nullptr;
    return t->data_ptr();
  }
  float number(PyObject* o) {
    if (!want(PyFloat_Check(o) || PyLong_Check(o))) return 0.f;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return (float)v;
  }
  Tensor empty(at::IntArrayRef sizes, at::ScalarType type) const {
    return at::empty(sizes, at::TensorOptions().dtype(type).device(at::kCUDA, device));
  }
  cudaStream_t stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
};

// f without the interpreter's lock, which comes back where f throws, too (a tensor without
// memory has no data pointer)
template <typename F>
bool launched(F f) {
  struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
  } unlocked;
  return f() == DOBB_OK;
}

PyObject* tuple(std::initializer_list<Tensor> tensors) {
  PyObject* r = PyTuple_New((Py_ssize_t)tensors.size());
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : tensors) {
    PyObject* o = nullptr;
    if (t.defined()) {
      o = THPVariable_Wrap(t);
    } else {
      Py_INCREF(Py_None);
      o = Py_None;
    }
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// x, weight, bias, eps, out_dtype -> out, mean, rstd
PyObject* layer_norm(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  if (!c.want(n == 5)) Py_RETURN_NONE;
  const Tensor *x = c.tensor(arg[0]), *w = c.tensor(arg[1], true), *b = c.tensor(arg[2], true);
  const float eps = c.number(arg[3]);
  c.want(arg[4] == Py_None || THPDtype_Check(arg[4]));
  if (!c.ok) Py_RETURN_NONE;
  const at::ScalarType otype = arg[4] == Py_None ? x->scalar_type() : reinterpret_cast<THPDtype*>(arg[4])->scalar_type;
  const dobb_dtype xd = c.dtype(x->scalar_type()), od = c.dtype(otype);
  const int64_t stride = c.rows(*x);
  if (!c.ok) Py_RETURN_NONE;
  const int64_t rows = x->size(0), dim = x->size(1);
  const at::ScalarType ptype = w ? w->scalar_type() : b ? b->scalar_type() : at::kFloat;
  const dobb_dtype pd = c.dtype(ptype);
  const void *wp = c.vector(w, dim, ptype), *bp = c.vector(b, dim, ptype);
  if (!c.ok) Py_RETURN_NONE;
  const Tensor out = c.empty({rows, dim}, otype), mean = c.empty({rows}, at::kFloat), rstd = c.empty({rows}, at::kFloat);
  if (!launched([&] {
        return dobb_layer_norm(x->data_ptr(), xd, rows, dim, stride, wp, bp, pd, eps, out.data_ptr(), od, dim,
                               static_cast<float*>(mean.data_ptr()), static_cast<float*>(rstd.data_ptr()), c.stream());
      }))
    Py_RETURN_NONE;
  return tuple({out, mean, rstd});
  END_HANDLE_TH_ERRORS
}

// grad, x, mean, rstd, weight, dtype -> dx, dweight, dbias
PyObject* layer_norm_backward(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  if (!c.want(n == 6 && THPDtype_Check(arg[5]))) Py_RETURN_NONE;
  const Tensor *g = c.tensor(arg[0]), *x = c.tensor(arg[1]), *mean = c.tensor(arg[2]), *rstd = c.tensor(arg[3]), *w = c.tensor(arg[4], true);
  if (!c.ok) Py_RETURN_NONE;
  const at::ScalarType ptype = w ? w->scalar_type() : at::kFloat, dtype = reinterpret_cast<THPDtype*>(arg[5])->scalar_type;
  const dobb_dtype gd = c.dtype(g->scalar_type()), xd = c.dtype(x->scalar_type()), pd = c.dtype(ptype), dd = c.dtype(dtype);
  const int64_t gstride = c.rows(*g), stride = c.rows(*x);
  if (!c.ok || !c.want(g->sizes() == x->sizes())) Py_RETURN_NONE;
  const int64_t rows = x->size(0), dim = x->size(1);
  const void *wp = c.vector(w, dim, ptype), *mp = c.vector(mean, rows, at::kFloat), *rp = c.vector(rstd, rows, at::kFloat);
  const size_t bytes = c.ok ? dobb_layer_norm_backward_bytes(rows, dim) : 0;
  if (bytes == 0) Py_RETURN_NONE;
  const Tensor dx = c.empty({rows, dim}, x->scalar_type()), dw = c.empty({dim}, dtype), db = c.empty({dim}, dtype);
  const Tensor ws = c.empty({(int64_t)bytes}, at::kByte);
  if (!launched([&] {
        return dobb_layer_norm_backward(g->data_ptr(), gd, gstride, x->data_ptr(), xd, rows, dim, stride, wp, pd,
                                        static_cast<const float*>(mp), static_cast<const float*>(rp), dx.data_ptr(), dim, dw.data_ptr(),
                                        db.data_ptr(), dd, 0, ws.data_ptr(), bytes, c.stream());
      }))
    Py_RETURN_NONE;
  return tuple({dx, dw, db});
  END_HANDLE_TH_ERRORS
}

// logits, ids, teacher, scale, teacher_scale, grad_loss -> loss, dlogits, stats
PyObject* distill(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  if (!c.want(n == 6)) Py_RETURN_NONE;
  const Tensor *x = c.tensor(arg[0]), *ids = c.tensor(arg[1]), *t = c.tensor(arg[2]), *g = c.tensor(arg[5], true);
  const float scale = c.number(arg[3]), teacher_scale = c.number(arg[4]);
  if (!c.ok) Py_RETURN_NONE;
  const dobb_dtype xd = c.dtype(x->scalar_type()), td = c.dtype(t->scalar_type());
  const int64_t stride = c.rows(*x);
  c.want(ids->scalar_type() == at::kInt || ids->scalar_type() == at::kLong);
  if (!c.ok || !c.want(ids->dim() == 2 && ids->size(0) == x->size(0) && t->sizes() == ids->sizes() && ids->is_contiguous() &&
                       t->is_contiguous()))
    Py_RETURN_NONE;
  const int64_t rows = x->size(0), vocab = x->size(1), k = ids->size(1);
  const void* gp = c.vector(g, rows, at::kFloat);
  if (!c.want(k >= 1 && k <= DOBB_MAX_TEACHER)) Py_RETURN_NONE;
  const Tensor out = g ? c.empty({rows, vocab}, x->scalar_type()) : Tensor();
  const Tensor stats = c.empty({3, rows}, at::kFloat);
  float* f = static_cast<float*>(stats.data_ptr());
  if (!launched([&] {
        return dobb_distill(x->data_ptr(), xd, rows, vocab, stride, ids->data_ptr(), (int)ids->element_size(), t->data_ptr(), td, (int)k,
                            scale, teacher_scale, f + 2 * rows, f, f + rows, static_cast<const float*>(gp), g ? out.data_ptr() : nullptr,
                            vocab, nullptr, c.stream());
      }))
    Py_RETURN_NONE;
  return tuple({stats.select(0, 2), out, stats});
  END_HANDLE_TH_ERRORS
}

// logits, noise, scale, top_k, top_p, min_p -> tokens, logp
PyObject* sample(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  if (!c.want(n == 6)) Py_RETURN_NONE;
  const Tensor *x = c.tensor(arg[0]), *e = c.tensor(arg[1]);
  if (!c.ok) Py_RETURN_NONE;
  const dobb_dtype xd = c.dtype(x->scalar_type());
  const int64_t stride = c.rows(*x), nstride = c.rows(*e);
  if (!c.ok || !c.want(e->scalar_type() == at::kFloat && e->sizes() == x->sizes())) Py_RETURN_NONE;
  const int64_t rows = x->size(0), vocab = x->size(1);
  // one value, or one per row
  const void* each[4] = {};
  float one[4] = {1.f, 1.f, 1.f, 1.f};
  int64_t top_k = 0;
  for (int i = 0; i < 4 && c.ok; ++i) {
    PyObject* o = arg[2 + i];
    if (THPVariable_Check(o)) {
      const Tensor* t = c.tensor(o);
      each[i] = c.vector(t, rows, i == 1 ? at::kInt : at::kFloat);
    } else if (i != 1) {
      one[i] = c.number(o);
    } else if (c.want(PyLong_Check(o))) {
      int over = 0;
      top_k = PyLong_AsLongLongAndOverflow(o, &over);
      c.want(!over && top_k >= 0 && top_k < (1ll << 31));
    }
  }
  if (!c.ok) Py_RETURN_NONE;
  const Tensor tokens = c.empty({rows}, at::kInt), logp = c.empty({rows}, at::kFloat);
  if (!launched([&] {
        return dobb_sample(x->data_ptr(), xd, rows, vocab, stride, static_cast<const float*>(e->data_ptr()), nstride, one[0], (int)top_k,
                           one[2], one[3], static_cast<const float*>(each[0]), static_cast<const int32_t*>(each[1]),
                           static_cast<const float*>(each[2]), static_cast<const float*>(each[3]), static_cast<int32_t*>(tokens.data_ptr()),
                           static_cast<float*>(logp.data_ptr()), c.stream());
      }))
    Py_RETURN_NONE;
  return tuple({tokens, logp});
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<layer_norm>("layer_norm"), method<layer_norm_backward>("layer_norm_backward"), method<distill>("distill"),
                         method<sample>("sample"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lm_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lm_call() { return PyModule_Create(&module); }
