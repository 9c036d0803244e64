// Native front of the calls that are made once per token or per training
// step: fp8_linear_act, fp8_linear_act_backward, fp8_layer_norm and
// fp8_layer_norm_backward.  Marshalling only, like the Python binding
// (api.py), which stays the place of every check and message: a function here
// takes the common case -- plain contiguous tensors of the right types and
// sizes on the current device -- and returns None for anything else, which
// then goes through api.py.  It returns an int (the status) where the library
// refuses, and the call's result otherwise.
//
// Why: in Python the checks, the output's allocation and 20 ctypes arguments
// cost about 6 us a call beside the launch's 3.5 us, more than the kernels of
// one token take.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/fp8mot.h"

namespace {

PyObject* g_parameter = nullptr;     // torch.nn.Parameter
PyObject* g_raw_stream = nullptr;    // torch._C._cuda_getCurrentRawStream
PyObject* g_get_device = nullptr;    // torch._C._cuda_getDevice

struct Skip {};   // not the common case

// A plain tensor (or parameter) of the call's device.
struct Call {
  int dev = -1;

  const at::Tensor& plain(PyObject* o) {
    if (!THPVariable_CheckExact(o) && (PyObject*)Py_TYPE(o) != g_parameter) throw Skip();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided || !t.is_cuda() || !t.is_contiguous()) throw Skip();
    const int d = t.get_device();
    if (dev < 0) dev = d;
    if (d != dev) throw Skip();
    return t;
  }
  const at::Tensor& of(PyObject* o, at::ScalarType type, int64_t n = -1) {
    const at::Tensor& t = plain(o);
    if (t.scalar_type() != type || (n >= 0 && t.numel() != n)) throw Skip();
    return t;
  }
  // BF16 or FP32, or None
  const void* floats(PyObject* o, int64_t n, int* elem) {
    *elem = FP8MOT_ELEM_BF16;
    if (o == Py_None) return nullptr;
    const at::Tensor& t = plain(o);
    if (t.numel() != n) throw Skip();
    *elem = elem_of(t);
    return t.const_data_ptr();
  }
  static int elem_of(const at::Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return FP8MOT_ELEM_BF16;
    if (t.scalar_type() == at::kFloat) return FP8MOT_ELEM_F32;
    throw Skip();
  }
  const float* scale(PyObject* o, int64_t n) { return static_cast<const float*>(of(o, at::kFloat, n).const_data_ptr()); }
  // the given output, or a new one
  at::Tensor output(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    if (o == Py_None) return at::empty(shape, like.options().dtype(type));
    int64_t n = 1;
    for (int64_t s : shape) n *= s;
    return of(o, type, n);
  }
  at::Tensor scratch(PyObject* o, size_t bytes, const at::Tensor& like) {
    if (o != Py_None) return of(o, at::kByte);
    if (bytes == 0) return at::Tensor();
    return at::empty({(int64_t)bytes}, like.options().dtype(at::kByte));
  }
  // the current stream of the device, which has to be the current one
  hipStream_t stream() {
    PyObject* d = PyObject_CallNoArgs(g_get_device);
    if (d == nullptr) throw Skip();
    const long cur = PyLong_AsLong(d);
    Py_DECREF(d);
    if (cur != dev) throw Skip();
    PyObject* idx = PyLong_FromLong(dev);
    PyObject* s = idx != nullptr ? PyObject_CallOneArg(g_raw_stream, idx) : nullptr;
    Py_XDECREF(idx);
    if (s == nullptr) throw Skip();
    void* p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    return static_cast<hipStream_t>(p);
  }
};

int small_int(PyObject* o) {
  if (!PyLong_Check(o)) throw Skip();
  const long v = PyLong_AsLong(o);
  if ((v == -1 && PyErr_Occurred()) || v < -1000 || v > 1000) throw Skip();
  return (int)v;
}

bool flag(PyObject* o) {
  if (o == Py_True) return true;
  if (o == Py_False) return false;
  throw Skip();
}

void* data(const at::Tensor& t) { return t.defined() ? const_cast<void*>(t.const_data_ptr()) : nullptr; }

bool out_type(int kind, at::ScalarType* t) {
  if (kind < 0 || kind > 2) return false;
  *t = kind == FP8MOT_OUT_BF16 ? at::kBFloat16 : (kind == FP8MOT_OUT_FP8 ? at::kByte : at::kFloat);
  return true;
}

PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (r == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

// Runs a call's body; what is not the common case, or fails on the way (an
// allocation, say), is left to api.py.
template <class F>
PyObject* guarded(F body) {
  try {
    return body();
  } catch (const Skip&) {
  } catch (const std::exception&) {
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

template <class F>
int without_gil(F f) {
  int st = 0;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st;
}

// (qx, qw, sx, sw, bias, act, residual, out_kind, sy, rowwise, pre, out, accum, workspace)
PyObject* linear_act(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 14) throw Skip();
    Call c;
    const at::Tensor& qx = c.of(a[0], at::kByte);
    const at::Tensor& qw = c.of(a[1], at::kByte);
    if (qw.dim() != 2 || qx.dim() < 1 || qx.size(-1) != qw.size(1)) throw Skip();
    const int64_t N = qw.size(0), K = qw.size(1);
    if (K == 0) throw Skip();
    const int64_t M = qx.numel() / K;
    const bool rowwise = flag(a[9]);
    const float* sx = c.scale(a[2], rowwise ? M : 1);
    const float* sw = c.scale(a[3], rowwise ? N : 1);
    int bias_elem, res_elem;
    const void* bias = c.floats(a[4], N, &bias_elem);
    const int act = small_int(a[5]), kind = small_int(a[7]), accum = small_int(a[12]);
    const void* residual = c.floats(a[6], M * N, &res_elem);
    at::ScalarType type;
    if (!out_type(kind, &type)) throw Skip();
    const float* sy = kind == FP8MOT_OUT_FP8 ? c.scale(a[8], 1) : nullptr;
    at::DimVector shape(qx.sizes());
    shape.back() = N;
    const at::Tensor out = c.output(a[11], shape, type, qx);
    at::Tensor pre;
    if (a[10] == Py_True) pre = at::empty(shape, qx.options().dtype(at::kBFloat16));
    else if (a[10] != Py_False && a[10] != Py_None) pre = c.of(a[10], at::kBFloat16, M * N);
    const at::Tensor ws = c.scratch(a[13], fp8_linear_act_workspace(M, N, K), qx);
    const hipStream_t stream = c.stream();
    const int st = without_gil([&] {
      return fp8_linear_act(static_cast<const uint8_t*>(data(qx)), static_cast<const uint8_t*>(data(qw)), data(out),
                            M, N, K, sx, sw, rowwise, bias, bias_elem, act, residual, res_elem,
                            static_cast<uint16_t*>(data(pre)), kind, sy, accum, data(ws),
                            ws.defined() ? (size_t)ws.numel() : 0, stream);
    });
    if (st != FP8MOT_OK) return PyLong_FromLong(st);
    return pre.defined() ? tuple_of({out, pre}) : THPVariable_Wrap(out);
  });
}

// (dy, pre, act, dz, dbias, workspace)
PyObject* linear_act_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 6) throw Skip();
    Call c;
    const at::Tensor& dy = c.of(a[0], at::kBFloat16);
    if (dy.dim() == 0 || dy.size(-1) == 0) throw Skip();
    const int64_t N = dy.size(-1), M = dy.numel() / N;
    const void* pre = a[1] == Py_None ? nullptr : data(c.of(a[1], at::kBFloat16, M * N));
    const int act = small_int(a[2]);
    const at::Tensor dz = c.output(a[3], dy.sizes(), at::kBFloat16, dy);
    const at::Tensor db = c.output(a[4], {N}, at::kFloat, dy);
    const at::Tensor ws = c.scratch(a[5], fp8_linear_act_backward_workspace(M, N), dy);
    const hipStream_t stream = c.stream();
    const int st = without_gil([&] {
      return fp8_linear_act_backward(static_cast<const uint16_t*>(data(dy)), static_cast<const uint16_t*>(pre), act,
                                     static_cast<uint16_t*>(data(dz)), static_cast<float*>(data(db)), M, N, data(ws),
                                     ws.defined() ? (size_t)ws.numel() : 0, stream);
    });
    if (st != FP8MOT_OK) return PyLong_FromLong(st);
    return tuple_of({dz, db});
  });
}

// (x, weight, bias, eps, out_kind, sy, stats, out)
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 8 || !PyFloat_Check(a[3])) throw Skip();
    Call c;
    const at::Tensor& x = c.plain(a[0]);
    const int x_elem = Call::elem_of(x);
    if (x.dim() == 0 || x.size(-1) == 0) throw Skip();
    const int64_t H = x.size(-1), rows = x.numel() / H;
    int w_elem, b_elem;
    const void* w = c.floats(a[1], H, &w_elem);
    const void* b = c.floats(a[2], H, &b_elem);
    if (w != nullptr && b != nullptr && w_elem != b_elem) throw Skip();
    const int kind = small_int(a[4]);
    at::ScalarType type;
    if (!out_type(kind, &type)) throw Skip();
    const float* sy = kind == FP8MOT_OUT_FP8 ? c.scale(a[5], 1) : nullptr;
    const at::Tensor out = c.output(a[7], x.sizes(), type, x);
    at::Tensor mean, rstd;
    if (flag(a[6])) {
      mean = at::empty(x.sizes().slice(0, x.dim() - 1), x.options().dtype(at::kFloat));
      rstd = at::empty(x.sizes().slice(0, x.dim() - 1), x.options().dtype(at::kFloat));
    }
    const float eps = (float)PyFloat_AS_DOUBLE(a[3]);
    const hipStream_t stream = c.stream();
    const int st = without_gil([&] {
      return fp8_layer_norm(data(x), x_elem, w, b, w != nullptr ? w_elem : b_elem, data(out), kind, sy,
                            static_cast<float*>(data(mean)), static_cast<float*>(data(rstd)), rows, H, eps, stream);
    });
    if (st != FP8MOT_OK) return PyLong_FromLong(st);
    return mean.defined() ? tuple_of({out, mean, rstd}) : THPVariable_Wrap(out);
  });
}

// (dy, x, weight, mean, rstd, dres, dx, dweight, dbias, workspace)
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 10 || a[0] == Py_None) throw Skip();
    Call c;
    const at::Tensor& x = c.plain(a[1]);
    const int x_elem = Call::elem_of(x);
    if (x.dim() == 0 || x.size(-1) == 0) throw Skip();
    const int64_t H = x.size(-1), rows = x.numel() / H;
    int dy_elem, w_elem;
    const void* dy = c.floats(a[0], x.numel(), &dy_elem);
    const void* w = c.floats(a[2], H, &w_elem);
    const float* mean = c.scale(a[3], rows);
    const float* rstd = c.scale(a[4], rows);
    const void* dres = a[5] == Py_None ? nullptr : data(c.of(a[5], x.scalar_type(), x.numel()));
    const at::Tensor dx = c.output(a[6], x.sizes(), x.scalar_type(), x);
    const at::Tensor dw = c.output(a[7], {H}, at::kFloat, x);
    const at::Tensor db = c.output(a[8], {H}, at::kFloat, x);
    const at::Tensor ws = c.scratch(a[9], fp8_layer_norm_backward_workspace(rows, H), x);
    const hipStream_t stream = c.stream();
    const int st = without_gil([&] {
      return fp8_layer_norm_backward(dy, dy_elem, data(x), x_elem, w, w_elem, mean, rstd, dres, data(dx),
                                     static_cast<float*>(data(dw)), static_cast<float*>(data(db)), rows, H, data(ws),
                                     ws.defined() ? (size_t)ws.numel() : 0, stream);
    });
    if (st != FP8MOT_OK) return PyLong_FromLong(st);
    return tuple_of({dx, dw, db});
  });
}

PyMethodDef methods[] = {
    {"linear_act", (PyCFunction)(void (*)(void))linear_act, METH_FASTCALL, nullptr},
    {"linear_act_backward", (PyCFunction)(void (*)(void))linear_act_backward, METH_FASTCALL, nullptr},
    {"layer_norm", (PyCFunction)(void (*)(void))layer_norm, METH_FASTCALL, nullptr},
    {"layer_norm_backward", (PyCFunction)(void (*)(void))layer_norm_backward, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

PyObject* attr(const char* mod, const char* name) {
  PyObject* m = PyImport_ImportModule(mod);
  if (m == nullptr) return nullptr;
  PyObject* o = PyObject_GetAttrString(m, name);
  Py_DECREF(m);
  return o;
}

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
  g_parameter = attr("torch.nn", "Parameter");
  g_raw_stream = g_parameter ? attr("torch._C", "_cuda_getCurrentRawStream") : nullptr;
  g_get_device = g_raw_stream ? attr("torch._C", "_cuda_getDevice") : nullptr;
  if (g_get_device == nullptr) return nullptr;
  return PyModule_Create(&module);
}
