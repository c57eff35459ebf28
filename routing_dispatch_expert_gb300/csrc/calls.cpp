// The calls around the experts as Python makes them, each in one step: the tensors' checks, the outputs' memory and the
// entry point of include/moe.h. On small tensors a call is bound by the host, and the same steps in Python take as long
// as memory and launch together or longer: one row's norm 5.2 us here and 11.6 there, sort and rows of 256 tokens to 8
// experts each 12.5 and 23, the routing gradient 3.9 and 8.7 (the launch alone 2.5).
//
// Arguments that are not all as the entry point wants them, and calls that it refuses, return None: the binding in moe.py
// then goes through them one by one and finds the words. Nothing has been launched in that case: an entry point refuses
// before its first launch. What goes wrong behind that, a launch, raises MoeError at once.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <pybind11/pybind11.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "../../include/moe.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

PyTypeObject* config_type = nullptr;  // moe.MoeConfig
PyObject* error_type = nullptr;       // moe.MoeError

constexpr ScalarType kF32 = ScalarType::Float, kInt = ScalarType::Int, kByte = ScalarType::Byte;

const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// Whether o is None (t stays null) or a tensor.
bool maybe(PyObject* o, const Tensor*& t) {
  t = o == Py_None ? nullptr : tensor(o);
  return t || o == Py_None;
}

int element_type(ScalarType s) {
  return s == kF32 ? MOE_TYPE_F32 : s == ScalarType::BFloat16 ? MOE_TYPE_BF16 : s == ScalarType::Half ? MOE_TYPE_F16 : -1;
}

// Everything has to be on the current device, in memory of its own (a wrapper's tensor has none, nor one whose storage was
// given up, whatever their addresses) and without a tangent of forward mode, of which the outputs would know nothing.
struct Here {
  int device = -1;
  bool holds(const Tensor& t) {
    if (!t.is_cuda() || t._fw_grad(0).defined()) return false;
    if (t.numel() && !(t.has_storage() && t.storage().data())) return false;
    if (device < 0) device = c10::cuda::current_device();
    return t.get_device() == device;
  }
  bool whole(const Tensor& t, ScalarType type, IntArrayRef shape) {
    return holds(t) && t.scalar_type() == type && t.sizes().equals(shape) && t.is_contiguous();
  }
  bool matrix(const Tensor& t) { return holds(t) && t.dim() == 2 && t.is_contiguous(); }
  // a matrix whose rows may lie apart: elements from row to row
  bool rows(const Tensor& t, int64_t& ld) {
    if (!holds(t) || t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1)) return false;
    ld = t.size(0) > 1 ? t.stride(0) : t.size(1);
    return true;
  }
  Tensor make(IntArrayRef shape, ScalarType type) const {
    return at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, (c10::DeviceIndex)device), std::nullopt);
  }
  moe_stream_t stream() const {
    return reinterpret_cast<moe_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
  }
};

void* address(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
void* address(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

bool config(PyObject* o, moe_config& c) {
  if (!config_type || !PyObject_TypeCheck(o, config_type)) return false;
  Py_buffer view;
  if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE)) {
    PyErr_Clear();
    return false;
  }
  const bool fits = view.len == (Py_ssize_t)sizeof(moe_config);
  if (fits) std::memcpy(&c, view.buf, sizeof(moe_config));
  PyBuffer_Release(&view);
  return fits && c.T >= 0 && c.k > 0 && c.E > 0;
}
int64_t groups(const moe_config& c) { return c.placement ? c.placement->n_slots : c.E; }

bool number(PyObject* o, float& f) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  f = (float)v;
  return true;
}

PyObject* wrapped(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

template <class... T>
PyObject* tuple_of(const T&... t) {
  PyObject* out = PyTuple_New(sizeof...(T));
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (PyObject* o : {wrapped(t)...}) {
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

#define WANT(condition) \
  do {                  \
    if (!(condition)) Py_RETURN_NONE; \
  } while (0)

// After a call: goes on where it was made, returns None where it was refused.
#define MADE(rc)                                                                                     \
  do {                                                                                               \
    if ((rc) == MOE_ERR_INVALID || (rc) == MOE_ERR_UNSUPPORTED || (rc) == MOE_ERR_WORKSPACE) Py_RETURN_NONE; \
    if ((rc) != MOE_OK) return failed(rc);                                                           \
  } while (0)

PyObject* failed(int rc) {
  PyObject* error = PyObject_CallFunction(error_type, "is", rc, moe_last_error());
  if (error) PyErr_SetObject(error_type, error);
  Py_XDECREF(error);
  return nullptr;
}

PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 2 || !PyType_Check(args[0]) || !PyExceptionClass_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "the classes of a configuration and of an error");
    return nullptr;
  }
  config_type = reinterpret_cast<PyTypeObject*>(Py_NewRef(args[0]));
  error_type = Py_NewRef(args[1]);
  Py_RETURN_NONE;
}

// (x, weight, residual, eps, fp8, with_y) -> (y, total, q, s)
PyObject* rms_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor *x, *w, *r;
  float eps;
  Here here;
  int64_t ldx = 0, ldr = 0;
  WANT(n == 6 && (x = tensor(args[0])) && maybe(args[1], w) && maybe(args[2], r) && number(args[3], eps) && here.rows(*x, ldx));
  const bool fp8 = PyObject_IsTrue(args[4]) == 1, with_y = PyObject_IsTrue(args[5]) == 1;
  const ScalarType kind = x->scalar_type();
  const int type = element_type(kind);
  const int64_t rows = x->size(0), cols = x->size(1);
  WANT(type >= 0 && cols > 0);
  WANT(!w || here.whole(*w, kind, {cols}) || here.whole(*w, kF32, {cols}));
  WANT(!r || (here.rows(*r, ldr) && r->sizes().equals(x->sizes()) && (r->scalar_type() == kind || r->scalar_type() == kF32)));
  Tensor y, total, q, s;
  int rc;
  {
    pybind11::gil_scoped_release others;
    if (r) total = here.make({rows, cols}, r->scalar_type());
    if (with_y) y = here.make({rows, cols}, kind);
    if (fp8) {
      q = here.make({rows, cols}, kByte);
      s = here.make({rows, (cols + 127) / 128}, kF32);
    }
    rc = moe_rms_norm(address(x), type, rows, cols, ldx, address(r), r ? element_type(r->scalar_type()) : 0, ldr, address(w),
                      w ? element_type(w->scalar_type()) : type, eps, address(y), address(total), address(q),
                      static_cast<float*>(address(s)), here.stream());
  }
  MADE(rc);
  return tuple_of(y, total, q, s);
  END_HANDLE_TH_ERRORS
}

// (dy, total, weight, eps, dtotal, weight_gradient, ws) -> (dx, dresidual, dweight)
PyObject* rms_norm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor *dy, *t, *w, *dt, *given;
  float eps;
  Here here;
  int64_t ldt = 0;
  WANT(n == 7 && (dy = tensor(args[0])) && (t = tensor(args[1])) && maybe(args[2], w) && number(args[3], eps) &&
       maybe(args[4], dt) && maybe(args[6], given));
  WANT(here.matrix(*dy) && here.rows(*t, ldt) && t->sizes().equals(dy->sizes()));
  const ScalarType kind = dy->scalar_type(), of = t->scalar_type();
  const int type = element_type(kind);
  const int64_t rows = dy->size(0), cols = dy->size(1);
  WANT(type >= 0 && cols > 0 && (of == kind || of == kF32) && (!dt || here.whole(*dt, of, dy->sizes())));
  WANT(!w || here.whole(*w, kind, {cols}) || here.whole(*w, kF32, {cols}));
  const bool wanted = w && PyObject_IsTrue(args[5]) == 1;
  size_t bytes = 0;
  if (wanted) WANT(moe_rms_norm_backward_workspace_size(rows, cols, &bytes) == MOE_OK);
  WANT(!given || here.whole(*given, kByte, {given->numel()}));
  Tensor dx, dr, dw, ws;
  int rc;
  {
    pybind11::gil_scoped_release others;
    dx = here.make({rows, cols}, kind);
    if (of != kind) dr = here.make({rows, cols}, of);
    if (wanted) {
      dw = here.make({cols}, w->scalar_type());
      ws = given ? *given : here.make({(int64_t)bytes}, kByte);
    }
    rc = moe_rms_norm_backward(address(dy), type, rows, cols, address(t), element_type(of), ldt, address(dt), address(w),
                               w ? element_type(w->scalar_type()) : type, eps, address(dx), address(dr), address(dw), address(ws),
                               ws.defined() ? (size_t)ws.numel() : 0, here.stream());
  }
  MADE(rc);
  PyObject* out = tuple_of(dx, dr, dw);
  if (out && !dr.defined()) {  // the residual's is dx itself
    PyObject* same = PyTuple_GET_ITEM(out, 0);
    Py_INCREF(same);
    Py_DECREF(PyTuple_GET_ITEM(out, 1));
    PyTuple_SET_ITEM(out, 1, same);
  }
  return out;
  END_HANDLE_TH_ERRORS
}

// (cfg, topk_idx, topk_w, ws) -> (counts, offsets, inv_pos, row_token, row_weight)
PyObject* sort_tokens(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  moe_config c;
  const Tensor *idx, *w, *given;
  Here here;
  WANT(n == 4 && config(args[0], c) && (idx = tensor(args[1])) && maybe(args[2], w) && maybe(args[3], given));
  const int64_t T = c.T, k = c.k, G = groups(c);
  WANT(here.whole(*idx, kInt, {T, k}) && (!w || here.whole(*w, kF32, {T, k})) &&
       (!given || here.whole(*given, kByte, {given->numel()})));
  size_t bytes = 0;
  WANT(moe_sort_tokens_workspace_size(&c, &bytes) == MOE_OK);
  Tensor counts, offsets, inv, token, weight, ws;
  int rc;
  {
    pybind11::gil_scoped_release others;
    if (given)
      ws = *given;
    else if (bytes)
      ws = here.make({(int64_t)bytes}, kByte);
    counts = here.make({G}, kInt);
    offsets = here.make({G + 1}, kInt);
    inv = here.make({T, k}, kInt);
    token = here.make({T * k}, kInt);
    if (w) weight = here.make({T * k}, kF32);
    rc = moe_sort_tokens(&c, static_cast<const int32_t*>(address(idx)), static_cast<const float*>(address(w)),
                         static_cast<int32_t*>(address(counts)), static_cast<int32_t*>(address(offsets)),
                         static_cast<int32_t*>(address(inv)), static_cast<int32_t*>(address(token)),
                         static_cast<float*>(address(weight)), address(ws), ws.defined() ? (size_t)ws.numel() : 0, here.stream());
  }
  MADE(rc);
  return tuple_of(counts, offsets, inv, token, weight);
  END_HANDLE_TH_ERRORS
}

// (cfg, x, inv_pos, offsets, scales) -> (xd, xd_scales)
PyObject* permute(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  moe_config c;
  const Tensor *x, *inv, *offsets, *scales;
  Here here;
  int64_t ldx = 0;
  WANT(n == 5 && config(args[0], c) && (x = tensor(args[1])) && (inv = tensor(args[2])) && (offsets = tensor(args[3])) &&
       maybe(args[4], scales));
  const int64_t T = c.T, k = c.k;
  WANT(here.rows(*x, ldx) && x->size(0) == T && x->size(1) > 0);
  const ScalarType kind = x->scalar_type();
  const int64_t cols = x->size(1), blocks = (cols + 127) / 128;
  WANT(kind == kByte || (!scales && element_type(kind) >= 0));
  WANT(here.whole(*inv, kInt, {T, k}) && here.whole(*offsets, kInt, {groups(c) + 1}) && (!scales || here.whole(*scales, kF32, {T, blocks})));
  Tensor xd, xs;
  int rc;
  {
    pybind11::gil_scoped_release others;
    xd = here.make({T * k, cols}, kind);
    if (scales) xs = here.make({T * k, blocks}, kF32);
    rc = moe_permute(&c, address(x), (int32_t)x->element_size(), cols, ldx, static_cast<const float*>(address(scales)),
                     static_cast<const int32_t*>(address(inv)), static_cast<const int32_t*>(address(offsets)), address(xd),
                     static_cast<float*>(address(xs)), here.stream());
  }
  MADE(rc);
  return scales ? tuple_of(xd, xs) : wrapped(xd);
  END_HANDLE_TH_ERRORS
}

// (cfg, yd, inv_pos, weights, base) -> y
PyObject* unpermute(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  moe_config c;
  const Tensor *yd, *inv, *w, *base;
  Here here;
  WANT(n == 5 && config(args[0], c) && (yd = tensor(args[1])) && (inv = tensor(args[2])) && maybe(args[3], w) && maybe(args[4], base));
  const int64_t T = c.T, k = c.k;
  WANT(here.matrix(*yd) && yd->size(0) == T * k && yd->size(1) > 0);
  const ScalarType kind = yd->scalar_type();
  const int64_t cols = yd->size(1);
  WANT(element_type(kind) >= 0 && here.whole(*inv, kInt, {T, k}) && (!w || here.whole(*w, kF32, {T, k})) &&
       (!base || here.whole(*base, kind, {T, cols})));
  Tensor y;
  int rc;
  {
    pybind11::gil_scoped_release others;
    y = here.make({T, cols}, kind);
    rc = moe_unpermute(&c, address(yd), element_type(kind), cols, static_cast<const int32_t*>(address(inv)),
                       static_cast<const float*>(address(w)), address(base), address(y), here.stream());
  }
  MADE(rc);
  return wrapped(y);
  END_HANDLE_TH_ERRORS
}

// (cfg, dy, yd, inv_pos, offsets, weights) -> (dyd, dweights)
PyObject* unpermute_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  moe_config c;
  const Tensor *dy, *yd, *inv, *offsets, *w;
  Here here;
  WANT(n == 6 && config(args[0], c) && (dy = tensor(args[1])) && maybe(args[2], yd) && (inv = tensor(args[3])) &&
       (offsets = tensor(args[4])) && maybe(args[5], w));
  const int64_t T = c.T, k = c.k;
  WANT(here.matrix(*dy) && dy->size(0) == T && dy->size(1) > 0);
  const ScalarType kind = dy->scalar_type();
  const int64_t cols = dy->size(1);
  WANT(element_type(kind) >= 0 && (!yd || here.whole(*yd, kind, {T * k, cols})) && here.whole(*inv, kInt, {T, k}) &&
       here.whole(*offsets, kInt, {groups(c) + 1}) && (!w || here.whole(*w, kF32, {T, k})));
  Tensor dyd, dw;
  int rc;
  {
    pybind11::gil_scoped_release others;
    dyd = here.make({T * k, cols}, kind);
    if (yd) dw = here.make({T, k}, kF32);
    rc = moe_unpermute_backward(&c, address(dy), address(yd), element_type(kind), cols, static_cast<const int32_t*>(address(inv)),
                                static_cast<const int32_t*>(address(offsets)), static_cast<const float*>(address(w)), address(dyd),
                                static_cast<float*>(address(dw)), here.stream());
  }
  MADE(rc);
  return tuple_of(dyd, dw);
  END_HANDLE_TH_ERRORS
}

// (cfg, logits, topk_idx, dtopk_w) -> dlogits
PyObject* route_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  moe_config c;
  const Tensor *z, *idx, *dw;
  Here here;
  WANT(n == 4 && config(args[0], c) && (z = tensor(args[1])) && (idx = tensor(args[2])) && (dw = tensor(args[3])));
  const int64_t T = c.T, E = c.E, k = c.k;
  const ScalarType kind = z->scalar_type();
  WANT((kind == kF32 || kind == ScalarType::BFloat16) && here.whole(*z, kind, {T, E}) && here.whole(*idx, kInt, {T, k}) &&
       here.whole(*dw, kF32, {T, k}));
  Tensor out;
  int rc;
  {
    pybind11::gil_scoped_release others;
    out = here.make({T, E}, kind);
    rc = moe_route_backward(&c, address(z), element_type(kind), static_cast<const int32_t*>(address(idx)),
                            static_cast<const float*>(address(dw)), address(out), here.stream());
  }
  MADE(rc);
  return wrapped(out);
  END_HANDLE_TH_ERRORS
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(bind), CALL(rms_norm), CALL(rms_norm_backward), CALL(sort_tokens), CALL(permute),
                         CALL(unpermute), CALL(unpermute_backward), CALL(route_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
