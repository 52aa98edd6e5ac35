// The usual call of an operator around the head from Python: checks, results' buffers and the
// C ABI's call in one step.  Each function takes what the Python function of its name takes,
// formats as flce_mx_format_t, and returns None for anything but a plain valid call that leaves
// the buffers to it; the Python function then does the checks one by one and raises, or goes
// the long way.  Small calls are bound by the host: a layer norm of one token takes 5.8 us this
// way and 8.8 through ctypes (call 3.9, of which the launch 2.4; three buffers 3.7), its
// backward 9.4 and 14.3, 4-bit log-probs of 4 tokens 9.6 and 13.6, a quantisation 5.2 and 7.3,
// a linear product of one token 5.7 and 11.6, its gradient 7.0 and 13.7, a dropout 5.2 and 8.6,
// log-probs of 4 rows of logits (two launches, five buffers) 9.3 and 17.6.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "flce.h"
#include "mx_layout.h"

namespace {

using at::Tensor;

// A tensor on the current GPU, or nullptr.
const Tensor* gpu_tensor(PyObject* o) {
  if (!THPVariable_Check(o)) return nullptr;
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.layout() != at::kStrided || t.get_device() != c10::hip::current_device())
    return nullptr;
  return &t;
}

bool dtype_id(at::ScalarType s, int& id) {
  id = s == at::kFloat ? FLCE_FP32 : FLCE_BF16;
  return s == at::kFloat || s == at::kBFloat16;
}
at::ScalarType scalar(int id) { return id == FLCE_FP32 ? at::kFloat : at::kBFloat16; }

// An element type given as a torch.dtype, or None for `otherwise`.
bool dtype_arg(PyObject* o, int otherwise, int& id) {
  if (o == Py_None) {
    id = otherwise;
    return true;
  }
  return THPDtype_Check(o) && dtype_id(reinterpret_cast<THPDtype*>(o)->scalar_type, id);
}

bool int_arg(PyObject* o, int64_t& v) {
  v = PyLong_AsLongLong(o);
  if (v != -1 || !PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}
bool float_arg(PyObject* o, float& v) {
  const double d = PyFloat_AsDouble(o);
  v = float(d);
  if (d != -1.0 || !PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}

// A matrix of bf16 or fp32 whose rows are contiguous and apart.
struct Rows {
  const Tensor* t;
  int64_t m, h, ld;
  int dtype;
  bool init(PyObject* o) {
    t = gpu_tensor(o);
    if (!t || t->dim() != 2 || !dtype_id(t->scalar_type(), dtype)) return false;
    m = t->size(0);
    h = t->size(1);
    ld = m > 1 ? t->stride(0) : h;
    return (t->stride(1) == 1 || h <= 1) && ld >= h;
  }
  void* data() const { return t->data_ptr(); }
};

// n contiguous elements of type s (nullptr for None, if `optional`).
bool vector(PyObject* o, at::ScalarType s, int64_t n, bool optional, const Tensor*& t) {
  t = nullptr;
  if (optional && o == Py_None) return true;
  t = gpu_tensor(o);
  return t && t->scalar_type() == s && t->dim() == 1 && t->size(0) == n && t->is_contiguous();
}
void* data(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
template <class T>
T* data_of(const Tensor* t) { return static_cast<T*>(data(t)); }

// weight and bias: of one type, which goes to dtype.
bool params(PyObject* w, PyObject* b, int64_t h, const Tensor*& weight, const Tensor*& bias, int& dtype) {
  dtype = FLCE_BF16;
  PyObject* first = w == Py_None ? b : w;
  weight = bias = nullptr;
  if (first == Py_None) return true;
  const Tensor* t = gpu_tensor(first);
  return t && dtype_id(t->scalar_type(), dtype) && vector(w, t->scalar_type(), h, true, weight) &&
         vector(b, t->scalar_type(), h, true, bias);
}

// Codes and scales of a microscaled matrix of `rows` rows (-1: as many as it has).
bool microscaled(PyObject* c, PyObject* s, int64_t cols, int fmt, int64_t& rows, const Tensor*& codes,
                 const Tensor*& scales) {
  codes = gpu_tensor(c);
  scales = gpu_tensor(s);
  if (!codes || !scales || codes->dim() != 2 || scales->dim() != 2 || cols <= 0 ||
      cols > (int64_t(1) << 20))
    return false;
  if (rows < 0) rows = codes->size(0);
  return codes->scalar_type() == at::kByte && scales->scalar_type() == at::kByte &&
         codes->size(0) == rows && scales->size(0) == rows &&
         codes->size(1) == flce::mx_code_bytes(cols, fmt) && scales->size(1) == flce::mx_scale_bytes(cols) &&
         codes->is_contiguous() && scales->is_contiguous();
}

Tensor buffer(at::IntArrayRef size, at::ScalarType s) {
  return at::empty(size, at::TensorOptions().dtype(s).device(at::kCUDA, c10::hip::current_device()));
}
Tensor workspace(size_t bytes) { return buffer({int64_t(bytes < 256 ? 256 : bytes)}, at::kByte); }

hipStream_t stream() { return c10::hip::getCurrentHIPStream().stream(); }

// The call without the interpreter's lock.
template <class F>
bool run(F f) {
  flce_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st == FLCE_OK;
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* wrap_or_none(const Tensor& t) { return t.defined() ? wrap(t) : Py_NewRef(Py_None); }
PyObject* tuple(std::initializer_list<PyObject*> items) {
  PyObject* r = PyTuple_New(Py_ssize_t(items.size()));
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (r && o) PyTuple_SET_ITEM(r, i, o);
    else Py_XDECREF(o);
    ++i;
  }
  return r;
}

// (x, weight, bias, eps, out_dtype, format) -> (y, mean, rstd[, codes, scales])
PyObject* layer_norm_forward(PyObject* const* a) {
  Rows x;
  const Tensor *weight, *bias;
  float eps;
  int yd, pd;
  int64_t fmt;
  if (!x.init(a[0]) || !params(a[1], a[2], x.h, weight, bias, pd) || !float_arg(a[3], eps) ||
      !dtype_arg(a[4], x.dtype, yd) || !int_arg(a[5], fmt))
    return nullptr;
  const Tensor y = buffer({x.m, x.h}, scalar(yd)), mean = buffer({x.m}, at::kFloat),
               rstd = buffer({x.m}, at::kFloat);
  Tensor codes, scales;
  if (fmt != FLCE_MX_NONE) {
    codes = buffer({x.m, flce::mx_code_bytes(x.h, int(fmt))}, at::kByte);
    scales = buffer({x.m, flce::mx_scale_bytes(x.h)}, at::kByte);
  }
  if (!run([&] {
        return flce_layer_norm_forward(x.data(), x.dtype, x.ld, data(weight), data(bias), pd, x.m, x.h, eps,
                                       y.data_ptr(), yd, x.h, mean.data_ptr<float>(), rstd.data_ptr<float>(),
                                       int(fmt), codes.defined() ? codes.data_ptr() : nullptr,
                                       scales.defined() ? scales.data_ptr() : nullptr, stream());
      }))
    return nullptr;
  if (codes.defined()) return tuple({wrap(y), wrap(mean), wrap(rstd), wrap(codes), wrap(scales)});
  return tuple({wrap(y), wrap(mean), wrap(rstd)});
}

// (dy, x or None, codes, scales, format, mean, rstd, weight, dx_dtype, need_params, param_dtype)
// -> (dx, dweight, dbias)
PyObject* layer_norm_backward(PyObject* const* a) {
  Rows dy, x;
  int64_t fmt, need;
  const Tensor *codes = nullptr, *scales = nullptr, *mean, *rstd, *weight;
  int xd = FLCE_BF16, dxd, pd;
  if (!dy.init(a[0]) || !int_arg(a[4], fmt) || !int_arg(a[9], need)) return nullptr;
  int64_t ldx = dy.h;
  void* xp = nullptr;
  if (a[1] != Py_None) {
    if (!x.init(a[1]) || x.m != dy.m || x.h != dy.h || !dtype_arg(a[8], x.dtype, dxd) || dxd != x.dtype)
      return nullptr;
    xd = x.dtype;
    xp = x.data();
    ldx = x.ld;
  } else if (int64_t m = dy.m; !microscaled(a[2], a[3], dy.h, int(fmt), m, codes, scales) ||
                               !dtype_arg(a[8], dy.dtype, dxd)) {
    return nullptr;
  }
  if (!vector(a[5], at::kFloat, dy.m, false, mean) || !vector(a[6], at::kFloat, dy.m, false, rstd))
    return nullptr;
  if (a[7] != Py_None) {
    const Tensor* bias;
    int given;
    if (!params(a[7], Py_None, dy.h, weight, bias, pd) || !dtype_arg(a[10], pd, given) || given != pd)
      return nullptr;
  } else {
    weight = nullptr;
    if (!dtype_arg(a[10], FLCE_FP32, pd)) return nullptr;
  }
  size_t bytes = 0;
  if (flce_layer_norm_backward_workspace(dy.m, dy.h, &bytes) != FLCE_OK) return nullptr;
  const Tensor ws = workspace(bytes), dx = buffer({dy.m, dy.h}, scalar(dxd));
  Tensor dw, db;
  if (need) {
    dw = buffer({dy.h}, scalar(pd));
    db = buffer({dy.h}, scalar(pd));
  }
  if (!run([&] {
        return flce_layer_norm_backward(
            dy.data(), dy.dtype, dy.ld, xp, xd, ldx, int(fmt), data(codes), data(scales), data(weight), pd,
            data_of<float>(mean), data_of<float>(rstd), dy.m, dy.h, dx.data_ptr(), dxd, dy.h,
            need ? dw.data_ptr() : nullptr, need ? db.data_ptr() : nullptr, ws.data_ptr(), ws.nbytes(), stream());
      }))
    return nullptr;
  return tuple({wrap(dx), wrap_or_none(dw), wrap_or_none(db)});
}

// (x, format) -> (codes, scales)
PyObject* mx_quantize(PyObject* const* a) {
  Rows x;
  int64_t fmt;
  if (!x.init(a[0]) || !int_arg(a[1], fmt) || x.h <= 0) return nullptr;
  const Tensor codes = buffer({x.m, flce::mx_code_bytes(x.h, int(fmt))}, at::kByte),
               scales = buffer({x.m, flce::mx_scale_bytes(x.h)}, at::kByte);
  if (!run([&] {
        return flce_mx_quantize(x.data(), x.dtype, x.ld, x.m, x.h, int(fmt), codes.data_ptr(), scales.data_ptr(),
                                stream());
      }))
    return nullptr;
  return tuple({wrap(codes), wrap(scales)});
}

// (codes, scales, format, cols, dtype) -> values
PyObject* mx_dequantize(PyObject* const* a) {
  int64_t fmt, cols, rows = -1;
  const Tensor *codes, *scales;
  int od;
  if (!int_arg(a[2], fmt) || !int_arg(a[3], cols) || !dtype_arg(a[4], FLCE_BF16, od) ||
      !microscaled(a[0], a[1], cols, int(fmt), rows, codes, scales))
    return nullptr;
  const Tensor out = buffer({rows, cols}, scalar(od));
  if (!run([&] {
        return flce_mx_dequantize(data(codes), data(scales), int(fmt), rows, cols, out.data_ptr(), od, cols,
                                  stream());
      }))
    return nullptr;
  return wrap(out);
}

// X and both parts of a head W in MXFP4.
struct Head {
  Rows x;
  int64_t v = -1;
  const Tensor *codes, *scales;
  bool init(PyObject* X, PyObject* c, PyObject* s) {
    return x.init(X) && x.dtype == FLCE_BF16 && x.t->is_contiguous() &&
           microscaled(c, s, x.h, FLCE_MXFP4, v, codes, scales);
  }
};

// (X, codes, scales, scale, out_dtype) -> logits
PyObject* mxfp4_logits(PyObject* const* a) {
  Head w;
  float scale;
  int od;
  size_t bytes = 0;
  if (!w.init(a[0], a[1], a[2]) || !float_arg(a[3], scale) || !dtype_arg(a[4], FLCE_BF16, od) ||
      flce_mx_workspace_query(w.x.m, w.x.h, w.v, 0, &bytes, nullptr) != FLCE_OK)
    return nullptr;
  const Tensor ws = workspace(bytes), out = buffer({w.x.m, w.v}, scalar(od));
  if (!run([&] {
        return flce_mx_logits(w.x.data(), data(w.codes), data(w.scales), w.x.m, w.x.h, w.v, scale, out.data_ptr(),
                              od, w.v, ws.data_ptr(), ws.nbytes(), stream());
      }))
    return nullptr;
  return wrap(out);
}

// (X, codes, scales, targets, ignore_index, scale, compute_entropy) -> (logprob, lse, entropy)
PyObject* mxfp4_forward(PyObject* const* a) {
  Head w;
  const Tensor* targets;
  int64_t ignore, ent;
  float scale;
  size_t bytes = 0;
  if (!w.init(a[0], a[1], a[2]) || !vector(a[3], at::kLong, w.x.m, false, targets) || !int_arg(a[4], ignore) ||
      !float_arg(a[5], scale) || !int_arg(a[6], ent) ||
      flce_mx_workspace_query(w.x.m, w.x.h, w.v, int(ent), nullptr, &bytes) != FLCE_OK)
    return nullptr;
  const Tensor ws = workspace(bytes), lp = buffer({w.x.m}, at::kFloat), lse = buffer({w.x.m}, at::kFloat);
  Tensor en;
  if (ent) en = buffer({w.x.m}, at::kFloat);
  if (!run([&] {
        return flce_mx_forward(w.x.data(), data(w.codes), data(w.scales), data_of<int64_t>(targets), w.x.m, w.x.h,
                               w.v, ignore, scale, int(ent), lp.data_ptr<float>(), lse.data_ptr<float>(),
                               ent ? en.data_ptr<float>() : nullptr, ws.data_ptr(), ws.nbytes(), stream());
      }))
    return nullptr;
  return tuple({wrap(lp), wrap(lse), wrap_or_none(en)});
}

bool double_arg(PyObject* o, double& v) {
  v = PyFloat_AsDouble(o);
  if (v != -1.0 || !PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}
bool uint_arg(PyObject* o, uint64_t& v) {
  if (!PyLong_Check(o)) return false;
  v = PyLong_AsUnsignedLongLong(o);
  if (v != uint64_t(-1) || !PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}
// A matrix with contiguous rows and the same size as `like`, or None.
bool rows_like(PyObject* o, int64_t m, int64_t h, Rows& r, void*& at) {
  at = nullptr;
  r.dtype = FLCE_BF16;
  r.ld = h;
  if (o == Py_None) return true;
  if (!r.init(o) || r.m != m || r.h != h) return false;
  at = r.data();
  return true;
}
// Contiguous elements of type s and the given size (nullptr for None).
bool block(PyObject* o, at::ScalarType s, at::IntArrayRef size, const Tensor*& t) {
  t = nullptr;
  if (o == Py_None) return true;
  t = gpu_tensor(o);
  return t && t->scalar_type() == s && t->sizes() == size && t->is_contiguous();
}

// (x, p, seed, offset, residual, out_dtype) -> y
PyObject* dropout(PyObject* const* a) {
  Rows x, r;
  void* residual;
  double p;
  uint64_t seed = 0, offset;
  const uint64_t* seed_at = nullptr;
  int yd;
  if (!x.init(a[0]) || !double_arg(a[1], p) || !uint_arg(a[3], offset) || !rows_like(a[4], x.m, x.h, r, residual) ||
      !dtype_arg(a[5], residual ? r.dtype : x.dtype, yd))
    return nullptr;
  if (!uint_arg(a[2], seed)) {
    const Tensor* t = gpu_tensor(a[2]);
    if (!t || t->scalar_type() != at::kLong || t->numel() != 1) return nullptr;
    seed_at = static_cast<const uint64_t*>(t->data_ptr());
  }
  const Tensor y = buffer({x.m, x.h}, scalar(yd));
  if (!run([&] {
        return flce_dropout(x.data(), x.dtype, x.ld, residual, r.dtype, r.ld, x.m, x.h, p, seed, seed_at, offset,
                            y.data_ptr(), yd, x.h, stream());
      }))
    return nullptr;
  return wrap(y);
}

// (X, W, bias, activation, residual, out_dtype, keep_pre) -> out, or (out, pre)
PyObject* linear_forward(PyObject* const* a) {
  Rows X, W, r;
  const Tensor *bias, *none;
  void* residual;
  int64_t act, keep;
  int bd, od;
  size_t bytes = 0;
  if (!X.init(a[0]) || !W.init(a[1]) || X.dtype != FLCE_BF16 || W.dtype != FLCE_BF16 || W.h != X.h ||
      !params(Py_None, a[2], W.m, none, bias, bd) || !int_arg(a[3], act) || !rows_like(a[4], X.m, W.m, r, residual) ||
      !dtype_arg(a[5], FLCE_BF16, od) || !int_arg(a[6], keep) ||
      flce_linear_workspace(X.m, W.m, X.h, &bytes, nullptr) != FLCE_OK)
    return nullptr;
  const Tensor out = buffer({X.m, W.m}, scalar(od));
  Tensor ws, pre;
  if (bytes) ws = workspace(bytes);
  if (keep) pre = buffer({X.m, W.m}, at::kBFloat16);
  if (!run([&] {
        return flce_linear_forward(X.data(), X.ld, W.data(), W.ld, data(bias), bd, int(act), residual, r.dtype, r.ld,
                                   X.m, W.m, X.h, out.data_ptr(), od, W.m, keep ? pre.data_ptr() : nullptr, W.m,
                                   bytes ? ws.data_ptr() : nullptr, bytes ? ws.nbytes() : 0, stream());
      }))
    return nullptr;
  return keep ? tuple({wrap(out), wrap(pre)}) : wrap(out);
}

// (dy, X, W, pre, activation, need_dx, need_dw, bias_dtype) -> (dX, dW, dbias)
PyObject* linear_backward(PyObject* const* a) {
  Rows dy, X, W, pre;
  void* kept;
  int64_t act, need_dx, need_dw;
  int bd = FLCE_BF16;
  size_t bytes = 0;
  if (!dy.init(a[0]) || !X.init(a[1]) || !W.init(a[2]) || X.dtype != FLCE_BF16 || W.dtype != FLCE_BF16 ||
      X.m != dy.m || W.m != dy.h || X.h != W.h || !int_arg(a[4], act) || !int_arg(a[5], need_dx) ||
      !int_arg(a[6], need_dw) || (a[7] != Py_None && !dtype_arg(a[7], FLCE_BF16, bd)))
    return nullptr;
  if (!rows_like(act ? a[3] : Py_None, dy.m, dy.h, pre, kept) || pre.dtype != FLCE_BF16 || (act && !kept) ||
      flce_linear_workspace(dy.m, dy.h, X.h, nullptr, &bytes) != FLCE_OK)
    return nullptr;
  const Tensor ws = workspace(bytes);
  Tensor dx, dw, db;
  if (need_dx) dx = buffer({X.m, X.h}, at::kBFloat16);
  if (need_dw) dw = buffer({W.m, W.h}, at::kBFloat16);
  if (a[7] != Py_None) db = buffer({W.m}, scalar(bd));
  auto at_of = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  if (!run([&] {
        return flce_linear_backward(dy.data(), dy.dtype, dy.ld, kept, pre.ld, int(act), X.data(), X.ld, W.data(), W.ld,
                                    dy.m, dy.h, X.h, at_of(dx), X.h, at_of(dw), X.h, at_of(db), bd, ws.data_ptr(),
                                    ws.nbytes(), stream());
      }))
    return nullptr;
  return tuple({wrap_or_none(dx), wrap_or_none(dw), wrap_or_none(db)});
}

// Given tokens [m] or [m, n], or None.
bool token_block(PyObject* o, int64_t m, const Tensor*& t, int64_t& n) {
  t = nullptr;
  n = 0;
  if (o == Py_None) return true;
  t = gpu_tensor(o);
  if (!t || t->scalar_type() != at::kLong || t->dim() < 1 || t->dim() > 2 || t->size(0) != m || !t->is_contiguous())
    return false;
  n = t->dim() == 1 ? 1 : t->size(1);
  return true;
}

// (logits, tokens, ignore_index, scale, n_top, compute_entropy)
// -> (logprob, lse, entropy, top_ids, top_logprob, stats)
PyObject* token_logprobs(PyObject* const* a) {
  Rows x;
  const Tensor* tokens;
  int64_t n, ignore, k, ent;
  float scale;
  size_t bytes = 0;
  if (!x.init(a[0]) || !token_block(a[1], x.m, tokens, n) || !int_arg(a[2], ignore) || !float_arg(a[3], scale) ||
      !int_arg(a[4], k) || !int_arg(a[5], ent) || k < 0 ||
      flce_token_logprobs_workspace(x.m, x.h, k, &bytes) != FLCE_OK)
    return nullptr;
  const Tensor lp = tokens ? buffer(tokens->sizes(), at::kFloat) : buffer({x.m, 0}, at::kFloat),
               lse = buffer({x.m}, at::kFloat), stats = buffer({x.m, 2}, at::kFloat);
  Tensor ws, en, ids, top;
  if (bytes) ws = workspace(bytes);
  if (ent) en = buffer({x.m}, at::kFloat);
  if (k) {
    ids = buffer({x.m, k}, at::kLong);
    top = buffer({x.m, k}, at::kFloat);
  }
  if (!run([&] {
        return flce_token_logprobs(x.data(), x.dtype, x.ld, x.m, x.h, data_of<int64_t>(tokens), n, ignore, scale, k,
                                   lp.data_ptr<float>(), lse.data_ptr<float>(), ent ? en.data_ptr<float>() : nullptr,
                                   stats.data_ptr<float>(), k ? ids.data_ptr<int64_t>() : nullptr,
                                   k ? top.data_ptr<float>() : nullptr, bytes ? ws.data_ptr() : nullptr,
                                   bytes ? ws.nbytes() : 0, stream());
      }))
    return nullptr;
  return tuple({wrap(lp), wrap(lse), wrap_or_none(en), wrap_or_none(ids), wrap_or_none(top), wrap(stats)});
}

// (logits, tokens, stats, entropy, top_ids, grad_logprob, grad_top, grad_entropy, grad_lse,
// ignore_index, scale) -> dlogits
PyObject* token_logprobs_backward(PyObject* const* a) {
  Rows x;
  const Tensor *tokens, *stats, *entropy = nullptr, *ids = nullptr, *g, *gt = nullptr, *ge, *gl;
  int64_t n, ignore, k = 0;
  float scale;
  if (!x.init(a[0]) || !token_block(a[1], x.m, tokens, n)) return nullptr;
  const int64_t no_tokens[2] = {x.m, 0};
  if (a[2] == Py_None || !block(a[2], at::kFloat, {x.m, 2}, stats) ||
      !block(a[5], at::kFloat, tokens ? tokens->sizes() : at::IntArrayRef(no_tokens, 2), g) ||
      !block(a[7], at::kFloat, {x.m}, ge) || !block(a[8], at::kFloat, {x.m}, gl) || !int_arg(a[9], ignore) ||
      !float_arg(a[10], scale))
    return nullptr;
  if (ge && (a[3] == Py_None || !block(a[3], at::kFloat, {x.m}, entropy))) return nullptr;
  if (a[6] != Py_None) {
    const Tensor* t = gpu_tensor(a[4]);
    if (!t || t->dim() != 2) return nullptr;
    k = t->size(1);
    if (!block(a[4], at::kLong, {x.m, k}, ids) || !block(a[6], at::kFloat, {x.m, k}, gt)) return nullptr;
  }
  const Tensor d = buffer({x.m, x.h}, scalar(x.dtype));
  if (!run([&] {
        return flce_token_logprobs_backward(
            x.data(), x.dtype, x.ld, x.m, x.h, data_of<int64_t>(tokens), n, ignore, scale, data_of<float>(stats),
            data_of<float>(entropy), k ? data_of<int64_t>(ids) : nullptr, k, data_of<float>(g),
            k ? data_of<float>(gt) : nullptr, data_of<float>(ge), data_of<float>(gl), d.data_ptr(), x.h, stream());
      }))
    return nullptr;
  return wrap(d);
}

// nullptr from a function means "not this way": None.  Nothing that C++ throws (memory that
// cannot be had) leaves the entry; the long way then raises it.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  PyObject* r = nullptr;
  try {
    if (n == N) r = F(args);
  } catch (...) {
    r = nullptr;
  }
  return r || PyErr_Occurred() ? r : Py_NewRef(Py_None);
}
template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<layer_norm_forward, 6>("layer_norm_forward"),
                         method<layer_norm_backward, 11>("layer_norm_backward"),
                         method<mx_quantize, 2>("mx_quantize"),
                         method<mx_dequantize, 5>("mx_dequantize"),
                         method<mxfp4_logits, 5>("mxfp4_logits"),
                         method<mxfp4_forward, 7>("mxfp4_forward"),
                         method<dropout, 6>("dropout"),
                         method<linear_forward, 7>("linear_forward"),
                         method<linear_backward, 8>("linear_backward"),
                         method<token_logprobs, 6>("token_logprobs"),
                         method<token_logprobs_backward, 11>("token_logprobs_backward"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
