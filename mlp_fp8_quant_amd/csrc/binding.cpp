// Native front of the calls that are made once per token or per training
// step: fp8_linear_act, fp8_layer_norm, the calls with a scale for each block of
// 128, fp8_residual_norm and the backward passes.  Marshalling only, like the Python binding
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
#include <ATen/hip/EmptyTensor.h>
#include <ATen/record_function.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/fp8mot.h"

namespace {

PyObject* g_parameter = nullptr;     // torch.nn.Parameter
PyObject* g_raw_stream = nullptr;    // torch._C._cuda_getCurrentRawStream
PyObject* g_get_device = nullptr;    // torch._C._cuda_getDevice

struct Skip {};   // not the common case

// Whether anything would see, or change, what at::empty does: a dispatch mode or
// a transform of this thread, a profiler, deterministic algorithms (which fill
// new tensors).
bool watched() {
  return !(c10::impl::tls_local_dispatch_key_set().included_ - c10::default_included_set).empty() ||
         at::hasCallbacks() || at::globalContext().deterministicAlgorithms();
}

// A plain tensor (or parameter) of the call's device.
struct Call {
  int dev = -1;
  const bool seen = watched();

  // A new tensor on `like`'s device.  Where nothing watches, straight from its
  // allocator: at::empty's way through the dispatcher takes longer than that (0.9
  // us instead of 0.4).
  at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) const {
    if (seen) return at::empty(shape, like.options().dtype(type));
    return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
  }

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
    if (o == Py_None) return fresh(shape, type, like);
    int64_t n = 1;
    for (int64_t s : shape) n *= s;
    return of(o, type, n);
  }
  at::Tensor scratch(PyObject* o, size_t bytes, const at::Tensor& like) {
    if (o != Py_None) return of(o, at::kByte);
    if (bytes == 0) return at::Tensor();
    return fresh({(int64_t)bytes}, at::kByte, like);
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
    if (a[10] == Py_True) pre = c.fresh(shape, at::kBFloat16, qx);
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
      mean = c.fresh(x.sizes().slice(0, x.dim() - 1), at::kFloat, x);
      rstd = c.fresh(x.sizes().slice(0, x.dim() - 1), at::kFloat, x);
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

int64_t blocks128(int64_t n) { return (n + 127) / 128; }
int64_t code_columns(int64_t n) { return (n + 15) / 16 * 16; }

// Codes and scales of a block-scaled result of `cols` columns, as api.py's
// _codes: lead's rows of codes, lead_scales' of scales.
void block_codes(Call& c, PyObject* out, PyObject* scales, at::DimVector lead, at::DimVector lead_scales,
                 int64_t cols, const at::Tensor& like, at::Tensor* q, at::Tensor* s) {
  lead.push_back(code_columns(cols));
  lead_scales.push_back(blocks128(cols));
  *q = c.output(out, lead, at::kByte, like);
  *s = c.output(scales, lead_scales, at::kFloat, like);
}

// (x, tile, transpose, out, scales)
PyObject* quant_block(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 5) throw Skip();
    Call c;
    const at::Tensor& x = c.plain(a[0]);
    const int elem = Call::elem_of(x);
    const bool tile = flag(a[1]), transpose = flag(a[2]);
    if (x.dim() == 0 || x.size(-1) == 0 || ((tile || transpose) && x.dim() != 2)) throw Skip();
    const int64_t K = x.size(-1), M = x.numel() / K;
    at::DimVector lead(x.sizes().slice(0, x.dim() - 1));
    if (transpose) lead = {K};
    at::DimVector lead_scales(lead);
    if (tile) lead_scales = {blocks128(lead[0])};
    at::Tensor q, s;
    block_codes(c, a[3], a[4], lead, lead_scales, transpose ? M : K, x, &q, &s);
    const hipStream_t stream = c.stream();
    const int st = without_gil([&] {
      return fp8_quant_block(data(x), elem, static_cast<uint8_t*>(data(q)), static_cast<float*>(data(s)), M, K, tile,
                             transpose, stream);
    });
    if (st != FP8MOT_OK) return PyLong_FromLong(st);
    return tuple_of({q, s});
  });
}

// (g, u, out, scales)
PyObject* silu_mul_block(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 4) throw Skip();
    Call c;
    const at::Tensor& g = c.of(a[0], at::kBFloat16);
    const at::Tensor& u = c.of(a[1], at::kBFloat16);
    if (g.dim() == 0 || g.size(-1) == 0 || g.sizes() != u.sizes()) throw Skip();
    const int64_t K = g.size(-1), M = g.numel() / K;
    const at::DimVector lead(g.sizes().slice(0, g.dim() - 1));
    at::Tensor q, s;
    block_codes(c, a[2], a[3], lead, lead, K, g, &q, &s);
    const hipStream_t stream = c.stream();
    const int st = without_gil([&] {
      return silu_mul_2in_block(static_cast<const uint16_t*>(data(g)), static_cast<const uint16_t*>(data(u)),
                                static_cast<uint8_t*>(data(q)), static_cast<float*>(data(s)), M, K, stream);
    });
    if (st != FP8MOT_OK) return PyLong_FromLong(st);
    return tuple_of({q, s});
  });
}

// (qx, qw, sx, sw, bias, act, residual, out_kind, sy, pre, out)
PyObject* linear_block(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 11) throw Skip();
    Call c;
    const at::Tensor& qx = c.of(a[0], at::kByte);
    const at::Tensor& qw = c.of(a[1], at::kByte);
    if (qw.dim() != 2 || qx.dim() < 1 || qx.size(-1) != qw.size(1)) throw Skip();
    const int64_t N = qw.size(0), K = qw.size(1);
    if (K == 0) throw Skip();
    const int64_t M = qx.numel() / K, kb = blocks128(K);
    const float* sx = c.scale(a[2], M * kb);
    const at::Tensor& sw = c.of(a[3], at::kFloat);
    const bool w_rows = sw.numel() != blocks128(N) * kb;
    if (w_rows && sw.numel() != N * kb) throw Skip();
    int bias_elem, res_elem;
    const void* bias = c.floats(a[4], N, &bias_elem);
    const int act = small_int(a[5]), kind = small_int(a[7]);
    const void* residual = c.floats(a[6], M * N, &res_elem);
    at::ScalarType type;
    if (!out_type(kind, &type)) throw Skip();
    const float* sy = kind == FP8MOT_OUT_FP8 ? c.scale(a[8], 1) : nullptr;
    at::DimVector shape(qx.sizes());
    shape.back() = N;
    const at::Tensor out = c.output(a[10], shape, type, qx);
    at::Tensor pre;
    if (a[9] == Py_True) pre = c.fresh(shape, at::kBFloat16, qx);
    else if (a[9] != Py_False && a[9] != Py_None) pre = c.of(a[9], at::kBFloat16, M * N);
    const hipStream_t stream = c.stream();
    const int st = without_gil([&] {
      return fp8_linear_block(static_cast<const uint8_t*>(data(qx)), static_cast<const uint8_t*>(data(qw)), data(out),
                              M, N, K, sx, static_cast<const float*>(data(sw)), w_rows, bias, bias_elem, act, residual,
                              res_elem, static_cast<uint16_t*>(data(pre)), kind, sy, stream);
    });
    if (st != FP8MOT_OK) return PyLong_FromLong(st);
    return pre.defined() ? tuple_of({out, pre}) : THPVariable_Wrap(out);
  });
}

// gate [H] or [gates, H], or None (1 gate)
const void* gate_of(Call& c, PyObject* o, int64_t rows, int64_t H, int64_t* gates, int* elem) {
  *gates = 1;
  *elem = FP8MOT_ELEM_BF16;
  if (o == Py_None) return nullptr;
  const at::Tensor& t = c.plain(o);
  *elem = Call::elem_of(t);
  if ((t.dim() != 1 && t.dim() != 2) || t.size(-1) != H) throw Skip();
  if (t.dim() == 2) *gates = t.size(0);
  if (*gates < 1 || rows % *gates != 0) throw Skip();
  return t.const_data_ptr();
}
float real(PyObject* o) {
  if (!PyFloat_Check(o)) throw Skip();
  return (float)PyFloat_AS_DOUBLE(o);
}
PyObject* wrap_or_none(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

// (x, weight, hidden, gate, post_weight, alpha, eps, out_kind, sy, stats, out, stream_out)
PyObject* residual_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 12) throw Skip();
    Call c;
    const at::Tensor& x = c.plain(a[0]);
    const int x_elem = Call::elem_of(x);
    if (x.dim() == 0 || x.size(-1) == 0) throw Skip();
    const int64_t H = x.size(-1), rows = x.numel() / H;
    if (rows == 0) throw Skip();   // (a NULL pointer below is None)
    int w_elem, h_elem, g_elem, p_elem;
    const void* w = c.floats(a[1], H, &w_elem);
    const void* h = c.floats(a[2], x.numel(), &h_elem);
    int64_t gates;
    const void* gate = gate_of(c, a[3], rows, H, &gates, &g_elem);
    const void* post = c.floats(a[4], H, &p_elem);
    if (w != nullptr && post != nullptr && w_elem != p_elem) throw Skip();
    const float alpha = real(a[5]), eps = real(a[6]);
    const int kind = small_int(a[7]);
    const float* sy = nullptr;
    at::Tensor y, scales, r, rstd, post_rstd;
    const at::DimVector lead(x.sizes().slice(0, x.dim() - 1));
    if (kind == FP8MOT_OUT_FP8_BLOCK) {
      if (a[10] != Py_None) throw Skip();
      block_codes(c, Py_None, Py_None, lead, lead, H, x, &y, &scales);
    } else {
      at::ScalarType type;
      if (!out_type(kind, &type)) throw Skip();
      if (kind == FP8MOT_OUT_FP8) sy = c.scale(a[8], 1);
      y = c.output(a[10], x.sizes(), type, x);
    }
    if (h != nullptr) r = c.output(a[11], x.sizes(), x.scalar_type(), x);
    const bool stats = flag(a[9]);
    if (stats) {
      rstd = c.fresh(lead, at::kFloat, x);
      if (post != nullptr) post_rstd = c.fresh(lead, at::kFloat, x);
    }
    const hipStream_t stream = c.stream();
    const int st = without_gil([&] {
      return fp8_residual_norm(data(x), x_elem, h, h_elem, gate, g_elem, gates, post, w,
                               w != nullptr ? w_elem : p_elem, data(r), data(y), kind, sy,
                               static_cast<float*>(data(scales)), static_cast<float*>(data(rstd)),
                               static_cast<float*>(data(post_rstd)), rows, H, alpha, eps, stream);
    });
    if (st != FP8MOT_OK) return PyLong_FromLong(st);
    PyObject* result = PyTuple_New(stats ? 4 : 2);
    if (result == nullptr) throw Skip();
    PyTuple_SET_ITEM(result, 0, kind == FP8MOT_OUT_FP8_BLOCK ? tuple_of({y, scales}) : THPVariable_Wrap(y));
    PyTuple_SET_ITEM(result, 1, wrap_or_none(r));
    if (stats) {
      PyTuple_SET_ITEM(result, 2, wrap_or_none(rstd));
      PyTuple_SET_ITEM(result, 3, wrap_or_none(post_rstd));
    }
    return result;
  });
}

// (dy, r, weight, rstd, hidden, gate, post_weight, post_rstd, alpha, dr, dx, dhidden, dweight, dgate, dpost_weight,
//  workspace)
PyObject* residual_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 16 || a[0] == Py_None) throw Skip();
    Call c;
    const at::Tensor& r = c.plain(a[1]);
    const int r_elem = Call::elem_of(r);
    if (r.dim() == 0 || r.size(-1) == 0) throw Skip();
    const int64_t H = r.size(-1), rows = r.numel() / H;
    if (rows == 0) throw Skip();   // (a NULL pointer below is None)
    const at::Tensor& dy = c.plain(a[0]);
    const int h_elem = Call::elem_of(dy);
    if (dy.numel() != r.numel()) throw Skip();
    int w_elem, p_elem, g_elem;
    const void* w = c.floats(a[2], H, &w_elem);
    const float* rstd = c.scale(a[3], rows);
    const void* h = a[4] == Py_None ? nullptr : data(c.of(a[4], dy.scalar_type(), r.numel()));
    int64_t gates;
    const void* gate = gate_of(c, a[5], rows, H, &gates, &g_elem);
    const void* post = c.floats(a[6], H, &p_elem);
    if (w != nullptr && post != nullptr && w_elem != p_elem) throw Skip();
    const float* post_rstd = post != nullptr ? c.scale(a[7], rows) : nullptr;
    const float alpha = real(a[8]);
    const void* dr = a[9] == Py_None ? nullptr : data(c.of(a[9], r.scalar_type(), r.numel()));
    const at::Tensor dx = c.output(a[10], r.sizes(), r.scalar_type(), r);
    at::Tensor dh, dw, dgate, dpost;
    if (h != nullptr) dh = c.output(a[11], r.sizes(), dy.scalar_type(), r);
    else if (a[11] != Py_None) throw Skip();
    if (w != nullptr) dw = c.output(a[12], {H}, at::kFloat, r);
    else if (a[12] != Py_None) throw Skip();
    if (gate != nullptr) dgate = c.output(a[13], THPVariable_Unpack(a[5]).sizes(), at::kFloat, r);
    else if (a[13] != Py_None) throw Skip();
    if (post != nullptr) dpost = c.output(a[14], {H}, at::kFloat, r);
    else if (a[14] != Py_None) throw Skip();
    const at::Tensor ws = c.scratch(a[15], fp8_residual_norm_backward_workspace(rows, H, gates), r);
    const hipStream_t stream = c.stream();
    const int st = without_gil([&] {
      return fp8_residual_norm_backward(data(dy), data(r), r_elem, h, h_elem, gate, g_elem, gates, post, w,
                                        w != nullptr ? w_elem : p_elem, rstd, post_rstd, dr, data(dx), data(dh),
                                        static_cast<float*>(data(dgate)), static_cast<float*>(data(dpost)),
                                        static_cast<float*>(data(dw)), rows, H, alpha, data(ws),
                                        ws.defined() ? (size_t)ws.numel() : 0, stream);
    });
    if (st != FP8MOT_OK) return PyLong_FromLong(st);
    PyObject* result = PyTuple_New(5);
    if (result == nullptr) throw Skip();
    const at::Tensor* outs[5] = {&dx, &dh, &dw, &dgate, &dpost};
    for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(result, i, wrap_or_none(*outs[i]));
    return result;
  });
}

PyMethodDef methods[] = {
    {"linear_act", (PyCFunction)(void (*)(void))linear_act, METH_FASTCALL, nullptr},
    {"linear_act_backward", (PyCFunction)(void (*)(void))linear_act_backward, METH_FASTCALL, nullptr},
    {"layer_norm", (PyCFunction)(void (*)(void))layer_norm, METH_FASTCALL, nullptr},
    {"layer_norm_backward", (PyCFunction)(void (*)(void))layer_norm_backward, METH_FASTCALL, nullptr},
    {"quant_block", (PyCFunction)(void (*)(void))quant_block, METH_FASTCALL, nullptr},
    {"silu_mul_block", (PyCFunction)(void (*)(void))silu_mul_block, METH_FASTCALL, nullptr},
    {"linear_block", (PyCFunction)(void (*)(void))linear_block, METH_FASTCALL, nullptr},
    {"residual_norm", (PyCFunction)(void (*)(void))residual_norm, METH_FASTCALL, nullptr},
    {"residual_norm_backward", (PyCFunction)(void (*)(void))residual_norm_backward, METH_FASTCALL, nullptr},
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
