// Python binding of the operators around the loss: argument checks, outputs and workspaces
// (allocated by torch), the current stream, and one call of the C ABI.
//
// These calls are short: a step of a few tokens takes the GPU two to five microseconds, and
// marshalled through ctypes it took the host nine to fifteen. Here the checks, the allocations
// and the call are made without the interpreter in between (embed 5.9 us instead of 8.7, norm with
// a checkpoint 6.8 instead of 12, norm_bwd 8.1 instead of 14.9, about 2.3 of each for a launch).
// The module does not link the library; bind() hands it the addresses of the functions in the
// library that ckl.lib() loaded.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "../../include/ckl.h"

namespace {

struct Api {
  decltype(&ckl_embed) embed;
  decltype(&ckl_embed_grad_workspace_bytes) embed_grad_ws;
  decltype(&ckl_embed_grad) embed_grad;
  decltype(&ckl_act8_pack) pack;
  decltype(&ckl_act8_unpack) unpack;
  decltype(&ckl_act8_weight_grad_workspace_bytes) weight_grad_ws;
  decltype(&ckl_act8_weight_grad) weight_grad;
  decltype(&ckl_norm) norm;
  decltype(&ckl_norm_bwd_workspace_bytes) norm_bwd_ws;
  decltype(&ckl_norm_bwd) norm_bwd;
} api;
PyObject* ckl_error = nullptr;  // the binding's CKLError(code, what)

// A handle as the binding describes it: (address, V, d, bf16?, device index).
struct Ctx {
  ckl_handle h;
  int64_t V, d;
  at::ScalarType dtype;
  int index;
};

// A checkpoint as Act8 describes it: (q, scale, rstd, T, cols, format, device index, has rstd).
struct Ckpt {
  const void* q;
  const uint8_t* scale;
  const float* rstd;
  int64_t T, cols;
  ckl_act8_format fmt;
  int index;
  bool has_rstd;
};

struct Raised {};  // a Python error is set

int64_t to_int(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
double to_double(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool to_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}
template <typename... A>
[[noreturn]] void refuse(PyObject* type, const char* format, A... a) {
  PyErr_Format(type, format, a...);
  throw Raised{};
}

Ctx ctx_of(PyObject* t) {
  Ctx c;
  c.h = static_cast<ckl_handle>(PyLong_AsVoidPtr(PyTuple_GET_ITEM(t, 0)));
  c.V = to_int(PyTuple_GET_ITEM(t, 1));
  c.d = to_int(PyTuple_GET_ITEM(t, 2));
  c.dtype = to_bool(PyTuple_GET_ITEM(t, 3)) ? at::kBFloat16 : at::kFloat;
  c.index = (int)to_int(PyTuple_GET_ITEM(t, 4));
  return c;
}

Ckpt ckpt_of(const Ctx& c, PyObject* t) {
  Ckpt k;
  k.q = PyLong_AsVoidPtr(PyTuple_GET_ITEM(t, 0));
  k.scale = static_cast<const uint8_t*>(PyLong_AsVoidPtr(PyTuple_GET_ITEM(t, 1)));
  k.rstd = static_cast<const float*>(PyLong_AsVoidPtr(PyTuple_GET_ITEM(t, 2)));
  k.T = to_int(PyTuple_GET_ITEM(t, 3));
  k.cols = to_int(PyTuple_GET_ITEM(t, 4));
  k.fmt = static_cast<ckl_act8_format>(to_int(PyTuple_GET_ITEM(t, 5)));
  k.index = (int)to_int(PyTuple_GET_ITEM(t, 6));
  k.has_rstd = to_bool(PyTuple_GET_ITEM(t, 7));
  if (k.index != c.index) refuse(PyExc_ValueError, "the checkpoint must be on the handle's device");
  return k;
}

void has_shape(const Ckpt& k, int64_t T, int64_t cols) {
  if (k.T != T || k.cols != cols)
    refuse(PyExc_ValueError, "the checkpoint must be %lld x %lld", (long long)T, (long long)cols);
}

const at::Tensor& tensor_of(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

void dense(const Ctx& c, const char* name, const at::Tensor& t) {
  if (!t.is_cuda() || t.get_device() != c.index || !t.is_contiguous())
    refuse(PyExc_ValueError, "%s must be a contiguous tensor on the handle's device", name);
}

// A dense tensor of the handle's dtype on its device, of this shape where one is given.
const at::Tensor& rows(const Ctx& c, const char* name, PyObject* o, const at::IntArrayRef* shape) {
  const at::Tensor& t = tensor_of(name, o);
  if (t.scalar_type() != c.dtype)
    refuse(PyExc_TypeError, "%s must be torch.%s", name,
           c.dtype == at::kBFloat16 ? "bfloat16" : "float32");
  if (shape && t.sizes() != *shape) refuse(PyExc_ValueError, "%s has the wrong shape", name);
  dense(c, name, t);
  return t;
}
const at::Tensor& rows(const Ctx& c, const char* name, PyObject* o, at::IntArrayRef shape) {
  return rows(c, name, o, &shape);
}
const at::Tensor* rows_or_none(const Ctx& c, const char* name, PyObject* o, at::IntArrayRef shape) {
  return o == Py_None ? nullptr : &rows(c, name, o, &shape);
}

const at::Tensor& f32(const Ctx& c, const char* name, PyObject* o, at::IntArrayRef shape) {
  const at::Tensor& t = tensor_of(name, o);
  if (t.scalar_type() != at::kFloat || t.sizes() != shape)
    refuse(PyExc_TypeError, "%s must be a float32 tensor of the result's shape", name);
  dense(c, name, t);
  return t;
}

at::Tensor make(const Ctx& c, at::IntArrayRef shape, at::ScalarType dtype) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(at::kCUDA, (c10::DeviceIndex)c.index));
}

// The given output, or a new one (which adding to makes no sense of).
at::Tensor f32_out(const Ctx& c, const char* name, PyObject* o, at::IntArrayRef shape,
                   bool accumulate) {
  if (o != Py_None) return f32(c, name, o, shape);
  if (accumulate) refuse(PyExc_ValueError, "accumulate needs %s", name);
  return make(c, shape, at::kFloat);
}

at::Tensor workspace(const Ctx& c, PyObject* o, size_t bytes) {
  if (o == Py_None) return make(c, {(int64_t)bytes}, at::kByte);
  const at::Tensor& t = tensor_of("workspace", o);
  if (t.scalar_type() != at::kByte) refuse(PyExc_TypeError, "workspace must be uint8");
  dense(c, "workspace", t);
  return t;
}

const uint8_t* mask_of(const Ctx& c, PyObject* o, int64_t T) {
  if (o == Py_None) return nullptr;
  const at::Tensor& m = tensor_of("mask", o);
  if (m.scalar_type() != at::kByte || m.numel() != T)
    refuse(PyExc_TypeError, "mask must be a uint8 tensor with an entry for each id");
  dense(c, "mask", m);
  return static_cast<const uint8_t*>(m.const_data_ptr());
}

const at::Tensor& ids_of(const Ctx& c, PyObject* o) {
  const at::Tensor& t = tensor_of("ids", o);
  if (t.scalar_type() != at::kInt) refuse(PyExc_TypeError, "ids must be int32");
  dense(c, "ids", t);
  return t;
}

void* stream_of(const Ctx& c) {
  return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)c.index).stream();
}

// One call of the library, without the interpreter's lock (it may wait for the GPU).
template <typename F>
void call(const char* what, F&& f) {
  ckl_status code;
  Py_BEGIN_ALLOW_THREADS
  code = f();
  Py_END_ALLOW_THREADS
  if (code == CKL_OK) return;
  PyObject* e = PyObject_CallFunction(ckl_error, "is", (int)code, what);
  if (e) {
    PyErr_SetObject(ckl_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

// Where the parts of a new checkpoint lie in one buffer: rstd, q from a multiple of 16 on, scale.
struct NewCkpt {
  at::Tensor buf;
  Ckpt k;
};
NewCkpt new_ckpt(const Ctx& c, int64_t T, int64_t cols, int fmt, bool rstd) {
  const int64_t at = rstd ? (4 * T + 15) / 16 * 16 : 0, nb = (cols + 31) / 32;
  NewCkpt n;
  n.buf = make(c, {at + T * (cols + nb)}, at::kByte);
  uint8_t* p = static_cast<uint8_t*>(n.buf.mutable_data_ptr());
  n.k = Ckpt{p + at,  p + at + T * cols, rstd ? reinterpret_cast<float*>(p) : nullptr, T, cols,
             static_cast<ckl_act8_format>(fmt), c.index, rstd};
  return n;
}
PyObject* describe(const Ckpt& k) {
  PyObject* t = PyTuple_New(8);
  if (!t) throw Raised{};
  PyTuple_SET_ITEM(t, 0, PyLong_FromVoidPtr(const_cast<void*>(k.q)));
  PyTuple_SET_ITEM(t, 1, PyLong_FromVoidPtr(const_cast<uint8_t*>(k.scale)));
  PyTuple_SET_ITEM(t, 2, PyLong_FromVoidPtr(const_cast<float*>(k.rstd)));
  PyTuple_SET_ITEM(t, 3, PyLong_FromLongLong(k.T));
  PyTuple_SET_ITEM(t, 4, PyLong_FromLongLong(k.cols));
  PyTuple_SET_ITEM(t, 5, PyLong_FromLong(k.fmt));
  PyTuple_SET_ITEM(t, 6, PyLong_FromLong(k.index));
  PyTuple_SET_ITEM(t, 7, PyBool_FromLong(k.has_rstd));
  return t;
}

PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}
PyObject* tuple_of(std::initializer_list<PyObject*> items) {  // takes the references
  PyObject* t = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (t) PyTuple_SET_ITEM(t, i++, o);
    else Py_XDECREF(o);
  }
  return t;
}

// embed(ctx, ids, W, mask, scale, V_total, v0, out, sync)
PyObject* embed(PyObject* const* a) {
  const Ctx c = ctx_of(a[0]);
  const at::Tensor& ids = ids_of(c, a[1]);
  const int64_t T = ids.numel();
  const uint8_t* mask = mask_of(c, a[3], T);
  const at::Tensor& W = rows(c, "W", a[2], {c.V, c.d});
  const float scale = (float)to_double(a[4]);
  const int64_t V_total = a[5] == Py_None ? c.V : to_int(a[5]), v0 = to_int(a[6]);
  c10::DimVector shape(ids.sizes());
  shape.push_back(c.d);
  const at::Tensor out = a[7] == Py_None ? make(c, shape, c.dtype) : rows(c, "out", a[7], shape);
  const int sync = to_bool(a[8]);
  void* s = stream_of(c);
  call("ckl_embed", [&] {
    return api.embed(c.h, static_cast<const int32_t*>(ids.const_data_ptr()), mask,
                     W.const_data_ptr(), T, V_total, v0, scale, out.mutable_data_ptr(), s, sync);
  });
  return a[7] == Py_None ? THPVariable_Wrap(out) : same(a[7]);
}

// embed_grad(ctx, ids, dX, mask, scale, V_total, v0, dW, accumulate, workspace, sync)
PyObject* embed_grad(PyObject* const* a) {
  const Ctx c = ctx_of(a[0]);
  const at::Tensor& ids = ids_of(c, a[1]);
  const int64_t T = ids.numel();
  const uint8_t* mask = mask_of(c, a[3], T);
  c10::DimVector shape(ids.sizes());
  shape.push_back(c.d);
  const at::Tensor& dX = rows(c, "dX", a[2], shape);
  const float scale = (float)to_double(a[4]);
  const int64_t V_total = a[5] == Py_None ? c.V : to_int(a[5]), v0 = to_int(a[6]);
  const int accumulate = to_bool(a[8]), sync = to_bool(a[10]);
  const at::Tensor dW = f32_out(c, "dW", a[7], {c.V, c.d}, accumulate);
  size_t bytes = 0;
  if (a[9] == Py_None)
    call("ckl_embed_grad_workspace_bytes", [&] { return api.embed_grad_ws(c.h, T, &bytes); });
  const at::Tensor ws = workspace(c, a[9], bytes);
  void* s = stream_of(c);
  call("ckl_embed_grad", [&] {
    return api.embed_grad(c.h, static_cast<const int32_t*>(ids.const_data_ptr()), mask,
                          dX.const_data_ptr(), T, V_total, v0, scale, accumulate,
                          static_cast<float*>(dW.mutable_data_ptr()), ws.mutable_data_ptr(),
                          (size_t)ws.numel(), s, sync);
  });
  return a[7] == Py_None ? THPVariable_Wrap(dW) : same(a[7]);
}

// act8_pack(ctx, x, format, checkpoint or None) -> (buffer, description), or None where given
PyObject* act8_pack(PyObject* const* a) {
  const Ctx c = ctx_of(a[0]);
  const at::Tensor& x = rows(c, "x", a[1], nullptr);
  if (x.dim() != 2) refuse(PyExc_ValueError, "x must be T x cols");
  const int64_t T = x.size(0), cols = x.size(1);
  NewCkpt n;
  if (a[3] == Py_None) {
    n = new_ckpt(c, T, cols, (int)to_int(a[2]), false);
  } else {
    n.k = ckpt_of(c, a[3]);
    has_shape(n.k, T, cols);
  }
  void* s = stream_of(c);
  call("ckl_act8_pack", [&] {
    return api.pack(c.h, x.const_data_ptr(), T, cols, n.k.fmt, const_cast<void*>(n.k.q),
                    const_cast<uint8_t*>(n.k.scale), s);
  });
  if (a[3] != Py_None) return same(Py_None);
  return tuple_of({THPVariable_Wrap(n.buf), describe(n.k)});
}

// act8_unpack(ctx, checkpoint, out)
PyObject* act8_unpack(PyObject* const* a) {
  const Ctx c = ctx_of(a[0]);
  const Ckpt k = ckpt_of(c, a[1]);
  const int64_t shape[2] = {k.T, k.cols};
  const at::Tensor out = a[2] == Py_None ? make(c, shape, c.dtype) : rows(c, "out", a[2], shape);
  void* s = stream_of(c);
  call("ckl_act8_unpack", [&] {
    return api.unpack(c.h, k.q, k.scale, k.T, k.cols, k.fmt, out.mutable_data_ptr(), s);
  });
  return a[2] == Py_None ? THPVariable_Wrap(out) : same(a[2]);
}

// act8_weight_grad(ctx, dY, checkpoint, dW, accumulate, workspace, sync)
PyObject* act8_weight_grad(PyObject* const* a) {
  const Ctx c = ctx_of(a[0]);
  const Ckpt k = ckpt_of(c, a[2]);
  const at::Tensor& dY = rows(c, "dY", a[1], nullptr);
  if (dY.dim() != 2 || dY.size(0) != k.T)
    refuse(PyExc_ValueError, "dY must be T x n, a row for each row of the checkpoint");
  const int64_t n = dY.size(1);
  const int accumulate = to_bool(a[4]), sync = to_bool(a[6]);
  const at::Tensor dW = f32_out(c, "dW", a[3], {n, k.cols}, accumulate);
  size_t bytes = 0;
  if (a[5] == Py_None)
    call("ckl_act8_weight_grad_workspace_bytes",
         [&] { return api.weight_grad_ws(c.h, k.T, n, k.cols, &bytes); });
  const at::Tensor ws = workspace(c, a[5], bytes);
  void* s = stream_of(c);
  call("ckl_act8_weight_grad", [&] {
    return api.weight_grad(c.h, dY.const_data_ptr(), k.T, n, k.q, k.scale, k.cols, k.fmt,
                           accumulate, static_cast<float*>(dW.mutable_data_ptr()),
                           ws.mutable_data_ptr(), (size_t)ws.numel(), s, sync);
  });
  return a[3] == Py_None ? THPVariable_Wrap(dW) : same(a[3]);
}

// norm(ctx, x, gain, residual, eps, format or -1, y, s, checkpoint) -> (y, s, buffer, description);
// y, s and the checkpoint may be None: new ones (buffer and description None where not new)
PyObject* norm(PyObject* const* a) {
  const Ctx c = ctx_of(a[0]);
  const at::Tensor& x0 = tensor_of("x", a[1]);
  const int64_t T = x0.dim() > 0 ? x0.size(0) : 0, shape[2] = {T, c.d};
  const at::Tensor& x = rows(c, "x", a[1], shape);
  const at::Tensor& gain = rows(c, "gain", a[2], {c.d});
  const at::Tensor* res = rows_or_none(c, "residual", a[3], shape);
  const float eps = (float)to_double(a[4]);
  const int fmt = (int)to_int(a[5]);
  const at::Tensor y = a[6] == Py_None ? make(c, shape, c.dtype) : rows(c, "out[0]", a[6], shape);
  at::Tensor sum;
  if (res) sum = a[7] == Py_None ? make(c, shape, c.dtype) : rows(c, "out[1]", a[7], shape);
  NewCkpt n;
  n.k = Ckpt{};
  if (fmt >= 0 && a[8] == Py_None) {
    n = new_ckpt(c, T, c.d, fmt, true);
  } else if (fmt >= 0) {
    n.k = ckpt_of(c, a[8]);
    has_shape(n.k, T, c.d);
  }
  void* s = stream_of(c);
  call("ckl_norm", [&] {
    return api.norm(c.h, x.const_data_ptr(), res ? res->const_data_ptr() : nullptr,
                    gain.const_data_ptr(), T, eps, n.k.fmt,
                    res ? sum.mutable_data_ptr() : nullptr, y.mutable_data_ptr(),
                    const_cast<void*>(n.k.q), const_cast<uint8_t*>(n.k.scale),
                    const_cast<float*>(n.k.rstd), s);
  });
  const bool fresh = n.buf.defined();
  return tuple_of({a[6] == Py_None ? THPVariable_Wrap(y) : same(a[6]),
                   !res ? same(a[1]) : a[7] == Py_None ? THPVariable_Wrap(sum) : same(a[7]),
                   fresh ? THPVariable_Wrap(n.buf) : same(Py_None),
                   fresh ? describe(n.k) : same(Py_None)});
}

// norm_bwd(ctx, dY, checkpoint, gain, d_residual, dX, dgain, accumulate, workspace) -> (dX, dgain)
PyObject* norm_bwd(PyObject* const* a) {
  const Ctx c = ctx_of(a[0]);
  const Ckpt k = ckpt_of(c, a[2]);
  has_shape(k, k.T, c.d);
  if (!k.has_rstd)
    refuse(PyExc_ValueError, "the checkpoint has no rstd: it is not one of a norm");
  const int64_t shape[2] = {k.T, c.d};
  const at::Tensor& dY = rows(c, "dY", a[1], shape);
  const at::Tensor& gain = rows(c, "gain", a[3], {c.d});
  const at::Tensor* dS = rows_or_none(c, "d_residual", a[4], shape);
  const int accumulate = to_bool(a[7]);
  const at::Tensor dX = a[5] == Py_None ? make(c, shape, c.dtype) : rows(c, "dX", a[5], shape);
  const at::Tensor dgain = f32_out(c, "dgain", a[6], {c.d}, accumulate);
  size_t bytes = 0;
  if (a[8] == Py_None)
    call("ckl_norm_bwd_workspace_bytes", [&] { return api.norm_bwd_ws(c.h, k.T, &bytes); });
  const at::Tensor ws = workspace(c, a[8], bytes);
  void* s = stream_of(c);
  call("ckl_norm_bwd", [&] {
    return api.norm_bwd(c.h, dY.const_data_ptr(), k.q, k.scale, k.rstd, gain.const_data_ptr(),
                        dS ? dS->const_data_ptr() : nullptr, k.T, k.fmt, accumulate,
                        dX.mutable_data_ptr(), static_cast<float*>(dgain.mutable_data_ptr()),
                        ws.mutable_data_ptr(), (size_t)ws.numel(), s);
  });
  return tuple_of({a[5] == Py_None ? THPVariable_Wrap(dX) : same(a[5]),
                   a[6] == Py_None ? THPVariable_Wrap(dgain) : same(a[6])});
}

// bind(CKLError, addresses in the order of Api)
PyObject* bind(PyObject* const* a) {
  Py_XDECREF(ckl_error);
  ckl_error = same(a[0]);
  void** p = reinterpret_cast<void**>(&api);
  for (size_t i = 0; i < sizeof(Api) / sizeof(void*); ++i)
    p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[1], (Py_ssize_t)i));
  if (PyErr_Occurred()) throw Raised{};
  return same(Py_None);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments wanted, %zd given", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define CKL_ENTRY(f, n) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CKL_ENTRY(bind, 2),
                         CKL_ENTRY(embed, 9),
                         CKL_ENTRY(embed_grad, 11),
                         CKL_ENTRY(act8_pack, 4),
                         CKL_ENTRY(act8_unpack, 3),
                         CKL_ENTRY(act8_weight_grad, 7),
                         CKL_ENTRY(norm, 9),
                         CKL_ENTRY(norm_bwd, 9),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ckl_ops", nullptr, -1, methods, nullptr, nullptr,
                      nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ckl_ops() { return PyModule_Create(&module); }
