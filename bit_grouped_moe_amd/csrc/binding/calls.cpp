// Short calls of the Python binding: for decode-time operators, whose kernels
// take 2 to 20 us, argument checks, output allocation and ctypes marshalling
// in Python took 8 to 30 us.  Each function here does them for the ordinary
// call of one entry point (plain device tensors on the current device, no
// buffers passed in) and launches; for anything else it returns None, and
// the binding's Python code checks, explains and calls as before.  So every
// refusal has one wording and one place.
//
// A function returns its outputs, None (not an ordinary call), or the
// library's nonzero status as an int.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../../include/gq.h"

namespace {

struct Library {
  decltype(&gq_mxfp4_quantize) quantize;
  decltype(&gq_moe_topk) topk;
  decltype(&gq_moe_topk_backward) topk_backward;
  decltype(&gq_moe_decode) decode;
  decltype(&gq_mxfp4_grouped_gemv_fp4) gemv;
  decltype(&gq_mxfp4_grouped_gemv_fp4_swiglu) gemv_unit;
  decltype(&gq_mxfp4_grouped_gemm_fp4) gemm;
  decltype(&gq_mxfp4_grouped_gemm_fp4_swiglu) gemm_unit;
  decltype(&gq_route_sort) route_sort;
  decltype(&gq_route_max_tiles) max_tiles;
  decltype(&gq_mxfp8_quantize) quantize8;
  decltype(&gq_mxfp4_grouped_gemv_fp8) gemv8;
  decltype(&gq_mxfp4_grouped_gemv_fp8_swiglu) gemv8_unit;
  decltype(&gq_mxfp4_grouped_gemm_fp8) gemm8;
  decltype(&gq_mxfp4_grouped_gemm_fp8_swiglu) gemm8_unit;
  decltype(&gq_rms_norm) norm;
  decltype(&gq_rms_norm_backward) norm_backward;
  decltype(&gq_rms_norm_backward_workspace) norm_workspace;
  decltype(&gq_moe_route) route;
  decltype(&gq_moe_route_backward) route_backward;
} lib{};
PyObject* current_device = nullptr;          // torch's callables
PyObject* raw_stream = nullptr;

using at::Tensor;

// A plain (not subclassed) device tensor, or null.  (A tensor inside a function
// transform, torch.func.vmap for one, has the plain type and no storage.)
const Tensor* device_tensor(PyObject* o) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.layout() == at::kStrided && t.has_storage() ? &t : nullptr;
}
const Tensor* contiguous(PyObject* o, at::ScalarType type, int64_t dim) {
  const Tensor* t = device_tensor(o);
  return t && t->scalar_type() == type && t->dim() == dim && t->is_contiguous() ? t : nullptr;
}
int float_code(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return GQ_F32;
    case at::kBFloat16: return GQ_BF16;
    case at::kHalf: return GQ_F16;
    default: return -1;
  }
}
int64_t whole(PyObject* o) { return PyLong_AsLongLong(o); }

// The current stream of device `index`, if that device is current.  1: yes,
// 0: another device, -1: a Python error.
int stream_of(int64_t index, hipStream_t& stream) {
  PyObject* d = PyObject_CallNoArgs(current_device);
  if (!d) return -1;
  const int64_t now = whole(d);
  Py_DECREF(d);
  if (now != index) return 0;
  PyObject* i = PyLong_FromLongLong(index);
  if (!i) return -1;
  PyObject* s = PyObject_CallOneArg(raw_stream, i);
  Py_DECREF(i);
  if (!s) return -1;
  stream = static_cast<hipStream_t>(PyLong_AsVoidPtr(s));
  Py_DECREF(s);
  return PyErr_Occurred() ? -1 : 1;
}

bool together(const Tensor& a) { return true; }
template <typename... Rest>
bool together(const Tensor& a, const Tensor& b, const Rest&... rest) {
  return a.get_device() == b.get_device() && together(a, rest...);
}

// Launch with the interpreter free (a full queue may hold the call).  The
// arguments are made before, by the caller: a tensor's accessors may throw (an
// output made inside torch.func.grad has no storage), and an error is a Python
// error only while this thread holds the interpreter.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename Fn, typename... Args>
int launch(Fn* fn, Args... args) {
  Unlocked free;
  return fn(args...);
}

PyObject* wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* pack(std::initializer_list<Tensor> ts) {
  PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = wrap(t);
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

template <typename T>
T* data(const Tensor& t) { return static_cast<T*>(t.data_ptr()); }

// An output on the device of `like`, which is the current one: a tensor of its
// own, as at::empty makes it.  Where no mode or transform of this thread asks to
// see the allocation (dispatch keys beyond the two that are always there), it
// comes from the same allocator without a way through the dispatcher (an output
// 0.5 to 0.7 us of a call of 5: quantise 5.76 -> 4.85 us, route sort 7.9 -> 6.3).
Tensor output(const Tensor& like, at::ScalarType type, at::IntArrayRef sizes) {
  const auto options = like.options().requires_grad(false).dtype(type);
  const c10::DispatchKeySet always(
      {c10::DispatchKey::BackendSelect, c10::DispatchKey::ADInplaceOrView});
  if (!(c10::impl::tls_local_dispatch_key_set().included_ - always).empty())
    return at::empty(sizes, options);
  static c10::Allocator* from = nullptr;               // (under the interpreter's lock)
  if (!from) from = at::empty({1}, options).storage().allocator();
  return Tensor(at::detail::empty_generic(
      sizes, from, c10::DispatchKeySet(c10::DispatchKey::CUDA), type, c10::nullopt));
}

#define GQ_ARGS(count) \
  if (n != (count)) {  \
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments"); \
    return nullptr;    \
  }
#define GQ_STREAM(t)                                              \
  hipStream_t stream{};                                           \
  {                                                               \
    const int ok = stream_of((t).get_device(), stream);           \
    if (ok < 0) return nullptr;                                   \
    if (!ok) Py_RETURN_NONE;                                      \
  }

// rows, width and row stride of a tensor [..., width] without a gap between its
// leading dimensions, or of two dimensions at any stride; false: neither
bool value_rows(const Tensor& x, int64_t& rows, int64_t& K, int64_t& stride) {
  if (x.dim() < 1 || x.numel() == 0) return false;
  K = x.size(-1);
  rows = x.numel() / K;
  stride = K;
  if (!x.is_contiguous()) {
    if (x.dim() != 2 || x.stride(1) != 1) return false;
    if (rows > 1) stride = x.stride(0);
  }
  return K <= INT32_MAX;
}

// quantize(x, want_values) -> (blocks, scales[, values]); quantize8: codes for blocks
template <bool k8>
PyObject* quantize_call(PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GQ_ARGS(2)
  const Tensor* x = device_tensor(a[0]);
  const int code = x ? float_code(*x) : -1;
  int64_t rows, K, stride;
  if (code < 0 || !value_rows(*x, rows, K, stride) || K % 32) Py_RETURN_NONE;
  GQ_STREAM(*x)
  const bool want = a[1] == Py_True;
  auto shape = x->sizes().vec();
  shape.back() = K / 32;
  Tensor scales = output(*x, at::kByte, shape);
  shape.push_back(16);
  Tensor codes = output(*x, at::kByte, k8 ? x->sizes() : at::IntArrayRef(shape));
  Tensor values;
  if (want) values = output(*x, at::kBFloat16, x->sizes());
  const int st = launch(k8 ? lib.quantize8 : lib.quantize, x->data_ptr(), code, rows, (int32_t)K,
                        stride, data<uint8_t>(codes), data<uint8_t>(scales),
                        want ? data<uint16_t>(values) : nullptr, stream);
  if (st) return PyLong_FromLong(st);
  return want ? pack({codes, scales, values}) : pack({codes, scales});
  END_HANDLE_TH_ERRORS
}
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return quantize_call<false>(a, n);
}
PyObject* quantize8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return quantize_call<true>(a, n);
}

// A norm's gain [H], of the rows' type or float32: its type code, -1 where it is none.
int gain(PyObject* o, const Tensor& x, int64_t H) {
  const Tensor* w = device_tensor(o);
  if (!w || w->dim() != 1 || w->size(0) != H || !w->is_contiguous() || !(
          w->scalar_type() == x.scalar_type() || w->scalar_type() == at::kFloat) ||
      w->get_device() != x.get_device())
    return -1;
  return float_code(*w);
}
// An optional tensor of x's shape, type and device: false where it is not one.
bool same_rows(PyObject* o, const Tensor& x, const Tensor*& t, int64_t& stride) {
  t = nullptr;
  stride = 0;
  if (o == Py_None) return true;
  t = device_tensor(o);
  int64_t rows, K;
  return t && t->scalar_type() == x.scalar_type() && t->sizes() == x.sizes() &&
         t->get_device() == x.get_device() && value_rows(*t, rows, K, stride);
}
// A number as a double; false (and no error) where it is none.
bool number(PyObject* o, double& v) {
  v = PyFloat_AsDouble(o);
  if (!PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}

// rms_norm(x, weight, eps, residual, want_mxfp8, want_values)
//   -> (y, sum or None, codes or None, scales or None, values or None)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GQ_ARGS(6)
  const Tensor* x = device_tensor(a[0]);
  const int code = x ? float_code(*x) : -1;
  int64_t rows, H, stride, rstride;
  const Tensor* res;
  double eps;
  if (code < 0 || !value_rows(*x, rows, H, stride)) Py_RETURN_NONE;
  const int wcode = gain(a[1], *x, H);
  const bool eight = a[4] == Py_True, want = a[5] == Py_True;
  if (wcode < 0 || !number(a[2], eps) || !same_rows(a[3], *x, res, rstride) || (eight && H % 32) ||
      (want && !eight))
    Py_RETURN_NONE;
  GQ_STREAM(*x)
  Tensor y = output(*x, x->scalar_type(), x->sizes()), sum, codes, scales, values;
  if (res) sum = output(*x, x->scalar_type(), x->sizes());
  if (eight) {
    auto shape = x->sizes().vec();
    shape.back() = H / 32;
    codes = output(*x, at::kByte, x->sizes());
    scales = output(*x, at::kByte, shape);
    if (want) values = output(*x, at::kBFloat16, x->sizes());
  }
  const int st = launch(lib.norm, x->data_ptr(), stride, res ? res->data_ptr() : nullptr, rstride,
                        code, rows, (int32_t)H, THPVariable_Unpack(a[1]).data_ptr(), wcode,
                        (float)eps, res ? sum.data_ptr() : nullptr, y.data_ptr(),
                        eight ? data<uint8_t>(codes) : nullptr,
                        eight ? data<uint8_t>(scales) : nullptr,
                        want ? data<uint16_t>(values) : nullptr, stream);
  if (st) return PyLong_FromLong(st);
  return pack({y, sum, codes, scales, values});
  END_HANDLE_TH_ERRORS
}

// rms_norm_backward(d_y, h, weight, eps, d_residual, want_d_weight) -> (d_x, d_weight or None)
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GQ_ARGS(6)
  const Tensor* h = device_tensor(a[1]);
  const int code = h ? float_code(*h) : -1;
  int64_t rows, H, stride, dstride, rstride;
  const Tensor *dy, *res;
  double eps;
  if (code < 0 || !value_rows(*h, rows, H, stride)) Py_RETURN_NONE;
  const int wcode = gain(a[2], *h, H);
  if (wcode < 0 || !number(a[3], eps) || !same_rows(a[0], *h, dy, dstride) || !dy ||
      !same_rows(a[4], *h, res, rstride))
    Py_RETURN_NONE;
  const int64_t need = lib.norm_workspace(rows, (int32_t)H);
  if (need < 0) Py_RETURN_NONE;
  GQ_STREAM(*h)
  const Tensor& w = THPVariable_Unpack(a[2]);
  const bool want = a[5] == Py_True;
  Tensor dx = output(*h, h->scalar_type(), h->sizes()), dw, space;
  if (want) {
    dw = output(*h, w.scalar_type(), w.sizes());
    space = output(*h, at::kByte, {need});
  }
  const int st = launch(lib.norm_backward, dy->data_ptr(), dstride, h->data_ptr(), stride,
                        res ? res->data_ptr() : nullptr, rstride, code, rows, (int32_t)H,
                        w.data_ptr(), wcode, (float)eps, dx.data_ptr(),
                        want ? dw.data_ptr() : nullptr, want ? space.data_ptr() : nullptr, need,
                        stream);
  if (st) return PyLong_FromLong(st);
  return pack({dx, dw});
  END_HANDLE_TH_ERRORS
}

// rows, E and row stride of logits [rows, E]
bool logit_rows(const Tensor& z, int64_t& rows, int64_t& E, int64_t& stride) {
  if (z.dim() != 2 || z.numel() == 0 || (z.size(1) > 1 && z.stride(1) != 1)) return false;
  rows = z.size(0);
  E = z.size(1);
  stride = rows > 1 ? z.stride(0) : E;
  return E <= INT32_MAX;
}

// moe_topk(logits, topk, renormalize) -> (ids, weights)
PyObject* moe_topk(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GQ_ARGS(3)
  const Tensor* z = device_tensor(a[0]);
  const int code = z ? float_code(*z) : -1;
  int64_t rows, E, stride;
  if (code < 0 || !logit_rows(*z, rows, E, stride) || !PyLong_Check(a[1])) Py_RETURN_NONE;
  const int64_t k = whole(a[1]);
  if (k < 1 || k > E) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  GQ_STREAM(*z)
  const int renorm = PyObject_IsTrue(a[2]);
  Tensor ids = output(*z, at::kInt, {rows, k});
  Tensor w = output(*z, at::kFloat, {rows, k});
  const int st = launch(lib.topk, z->data_ptr(), code, rows, (int32_t)E, stride, (int32_t)k,
                        renorm, data<int32_t>(ids), data<float>(w), stream);
  if (st) return PyLong_FromLong(st);
  return pack({ids, w});
  END_HANDLE_TH_ERRORS
}

// moe_topk_backward(d_weights, logits, ids, renormalize) -> d_logits
PyObject* moe_topk_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GQ_ARGS(4)
  const Tensor* dw = contiguous(a[0], at::kFloat, 2);
  const Tensor* z = device_tensor(a[1]);
  const Tensor* ids = contiguous(a[2], at::kInt, 2);
  const int code = z ? float_code(*z) : -1;
  int64_t rows, E, stride;
  if (code < 0 || !dw || !ids || !logit_rows(*z, rows, E, stride) || ids->size(0) != rows ||
      dw->sizes() != ids->sizes() || ids->size(1) > INT32_MAX || !together(*z, *dw, *ids))
    Py_RETURN_NONE;
  GQ_STREAM(*z)
  const int renorm = PyObject_IsTrue(a[3]);
  Tensor dz = output(*z, z->scalar_type(), {rows, E});
  const int st = launch(lib.topk_backward, data<float>(*dw), z->data_ptr(), code, rows,
                        (int32_t)E, stride, data<int32_t>(*ids), (int32_t)ids->size(1), renorm,
                        dz.data_ptr(), stream);
  if (st) return PyLong_FromLong(st);
  return wrap(dz);
  END_HANDLE_TH_ERRORS
}

// moe_route(logits, topk, score, bias, groups, topk_groups, group_top, renormalize, scale)
//   -> (ids, weights)
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GQ_ARGS(9)
  const Tensor* z = device_tensor(a[0]);
  const int code = z ? float_code(*z) : -1;
  int64_t rows, E, stride, v[5];
  double scale;
  if (code < 0 || !logit_rows(*z, rows, E, stride) || !number(a[8], scale)) Py_RETURN_NONE;
  const int at[5] = {1, 2, 4, 5, 6};                   // topk, score, groups, topk_groups, group_top
  for (int i = 0; i < 5; ++i) {
    if (!PyLong_Check(a[at[i]])) Py_RETURN_NONE;
    v[i] = whole(a[at[i]]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    if (v[i] < 0 || v[i] > INT32_MAX) Py_RETURN_NONE;
  }
  if (v[0] < 1 || v[0] > E || v[2] < 1 || E % v[2]) Py_RETURN_NONE;
  const Tensor* bias = nullptr;
  if (a[3] != Py_None) {
    bias = contiguous(a[3], at::kFloat, 1);
    if (!bias || bias->size(0) != E || !together(*z, *bias)) Py_RETURN_NONE;
  }
  GQ_STREAM(*z)
  const int renorm = PyObject_IsTrue(a[7]);
  Tensor ids = output(*z, at::kInt, {rows, v[0]});
  Tensor w = output(*z, at::kFloat, {rows, v[0]});
  const int st = launch(lib.route, z->data_ptr(), code, rows, (int32_t)E, stride,
                        bias ? data<float>(*bias) : nullptr, (int32_t)v[0], (int32_t)v[1],
                        (int32_t)v[2], (int32_t)v[3], (int32_t)v[4], renorm, (float)scale,
                        data<int32_t>(ids), data<float>(w), stream);
  if (st) return PyLong_FromLong(st);
  return pack({ids, w});
  END_HANDLE_TH_ERRORS
}

// moe_route_backward(d_weights, logits, ids, score, renormalize, scale) -> d_logits
PyObject* moe_route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GQ_ARGS(6)
  const Tensor* dw = contiguous(a[0], at::kFloat, 2);
  const Tensor* z = device_tensor(a[1]);
  const Tensor* ids = contiguous(a[2], at::kInt, 2);
  const int code = z ? float_code(*z) : -1;
  int64_t rows, E, stride;
  double scale;
  if (code < 0 || !dw || !ids || !logit_rows(*z, rows, E, stride) || ids->size(0) != rows ||
      dw->sizes() != ids->sizes() || ids->size(1) > INT32_MAX || !together(*z, *dw, *ids) ||
      !PyLong_Check(a[3]) || !number(a[5], scale))
    Py_RETURN_NONE;
  const int64_t score = whole(a[3]);
  if (PyErr_Occurred()) return nullptr;
  GQ_STREAM(*z)
  const int renorm = PyObject_IsTrue(a[4]);
  Tensor dz = output(*z, z->scalar_type(), {rows, E});
  const int st = launch(lib.route_backward, data<float>(*dw), z->data_ptr(), code, rows,
                        (int32_t)E, stride, data<int32_t>(*ids), (int32_t)ids->size(1),
                        (int32_t)score, renorm, (float)scale, dz.data_ptr(), stream);
  if (st) return PyLong_FromLong(st);
  return wrap(dz);
  END_HANDLE_TH_ERRORS
}

// moe_decode(layer struct address, device, workspace bytes, x) -> y
PyObject* moe_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GQ_ARGS(4)
  const auto* layer = static_cast<const gq_moe_layer*>(PyLong_AsVoidPtr(a[0]));
  const int64_t index = whole(a[1]), need = whole(a[2]);
  const Tensor* x = device_tensor(a[3]);
  if (PyErr_Occurred()) return nullptr;
  if (!layer || need <= 0 || !x || x->scalar_type() != at::kBFloat16 || x->dim() != 2 ||
      x->size(1) != layer->hidden || x->stride(1) != 1 || x->size(0) < 1 ||
      x->get_device() != index)
    Py_RETURN_NONE;
  GQ_STREAM(*x)
  const int64_t rows = x->size(0);
  Tensor space = output(*x, at::kByte, {need});
  Tensor y = output(*x, at::kBFloat16, {rows, layer->hidden});
  const int st = launch(lib.decode, layer, data<uint16_t>(*x), (int32_t)rows,
                        rows > 1 ? x->stride(0) : layer->hidden, space.data_ptr(), need,
                        data<uint16_t>(y), stream);
  if (st) return PyLong_FromLong(st);
  return wrap(y);
  END_HANDLE_TH_ERRORS
}

// The operands of a product of MXFP4 or (k8) MXFP8 activations with MXFP4 weights.
struct Pair {
  const Tensor *xb, *xs, *blocks, *scales;
  int64_t rows, E, N, K;
};
template <bool k8>
bool mx_pair(PyObject* const* a, Pair& p) {
  p.xb = contiguous(a[0], at::kByte, k8 ? 2 : 3);
  p.xs = contiguous(a[1], at::kByte, 2);
  p.blocks = contiguous(a[2], at::kByte, 4);
  p.scales = contiguous(a[3], at::kByte, 3);
  if (!p.xb || !p.xs || !p.blocks || !p.scales) return false;
  const int64_t nb = p.blocks->size(2);
  p.rows = p.xb->size(0);
  p.E = p.blocks->size(0);
  p.N = p.blocks->size(1);
  p.K = nb * 32;
  return p.blocks->size(3) == 16 && p.scales->size(0) == p.E && p.scales->size(1) == p.N &&
         p.scales->size(2) == nb &&
         (k8 ? p.xb->size(1) == p.K : p.xb->size(1) == nb && p.xb->size(2) == 16) &&
         p.xs->size(0) == p.rows && p.xs->size(1) == nb && p.rows >= 1 && p.rows <= INT32_MAX &&
         p.E <= INT32_MAX && p.N <= INT32_MAX && p.K <= INT32_MAX &&
         together(*p.xb, *p.xs, *p.blocks, *p.scales);
}
// An optional float per pair: false where it is not one.
bool pair_weights(PyObject* o, int64_t P, const Tensor& beside, const float*& w) {
  w = nullptr;
  if (o == Py_None) return true;
  const Tensor* t = device_tensor(o);
  if (!t || t->scalar_type() != at::kFloat || !t->is_contiguous() || t->numel() != P ||
      !together(beside, *t))
    return false;
  w = data<float>(*t);
  return true;
}

// fp4_gemv(x blocks, x scales, blocks, scales, ids, pair_scale, unit, alpha, limit)
template <bool k8>
PyObject* gemv_call(PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GQ_ARGS(9)
  Pair p;
  const Tensor* ids = contiguous(a[4], at::kInt, 2);
  const bool unit = a[6] == Py_True;
  if (!mx_pair<k8>(a, p) || !ids || ids->size(0) != p.rows || ids->size(1) < 1 ||
      !together(*p.xb, *ids) || (unit && p.N % 2))
    Py_RETURN_NONE;
  const int64_t P = p.rows * ids->size(1);
  const float* ps;
  if (!pair_weights(a[5], P, *p.xb, ps) || ids->size(1) > INT32_MAX) Py_RETURN_NONE;
  const double alpha = PyFloat_AsDouble(a[7]), limit = PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred()) return nullptr;
  GQ_STREAM(*p.xb)
  Tensor out = output(*p.xb, at::kBFloat16, {P, unit ? p.N / 2 : p.N});
  const auto *xb = data<uint8_t>(*p.xb), *xs = data<uint8_t>(*p.xs);
  const auto *b = data<uint8_t>(*p.blocks), *s = data<uint8_t>(*p.scales);
  const auto* id = data<int32_t>(*ids);
  const int32_t k = (int32_t)ids->size(1);
  uint16_t* o = data<uint16_t>(out);
  const int st = unit ? launch(k8 ? lib.gemv8_unit : lib.gemv_unit, xb, xs, p.rows, p.K, b, s, p.E, p.N, id, k,
                               (float)alpha, (float)limit, o, stream)
                      : launch(k8 ? lib.gemv8 : lib.gemv, xb, xs, p.rows, p.K, b, s, p.E, p.N, id, k, ps,
                               o, stream);
  if (st) return PyLong_FromLong(st);
  return wrap(out);
  END_HANDLE_TH_ERRORS
}
PyObject* fp4_gemv(PyObject*, PyObject* const* a, Py_ssize_t n) { return gemv_call<false>(a, n); }
PyObject* fp8_gemv(PyObject*, PyObject* const* a, Py_ssize_t n) { return gemv_call<true>(a, n); }

// fp4_gemm(x blocks, x scales, blocks, scales, route, pair_scale, unit, alpha, limit)
template <bool k8>
PyObject* gemm_call(PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GQ_ARGS(9)
  Pair p;
  const bool unit = a[6] == Py_True;
  // expert_offsets, sorted_pairs, tiles, num_tiles, max_tiles, tile_m, rows, topk, num_experts
  if (!mx_pair<k8>(a, p) || !PyTuple_Check(a[4]) || PyTuple_GET_SIZE(a[4]) != 9 || (unit && p.N % 2))
    Py_RETURN_NONE;
  const Tensor* r[4];
  int64_t v[5];
  for (int i = 0; i < 4; ++i) {
    r[i] = device_tensor(PyTuple_GET_ITEM(a[4], i));
    if (!r[i] || r[i]->scalar_type() != at::kInt || !r[i]->is_contiguous() ||
        !together(*p.xb, *r[i]))
      Py_RETURN_NONE;
  }
  for (int i = 0; i < 5; ++i) v[i] = whole(PyTuple_GET_ITEM(a[4], 4 + i));
  const double alpha = PyFloat_AsDouble(a[7]), limit = PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred()) return nullptr;
  const int64_t k = v[3], P = p.rows * k;
  if (v[2] != p.rows || v[4] != p.E || k < 1 || k > INT32_MAX || v[0] < 0 || v[0] > INT32_MAX ||
      v[1] < 0 || v[1] > INT32_MAX || r[0]->numel() <= p.E || r[1]->numel() < P || r[2]->numel() < 2 * v[0] ||
      r[3]->numel() < 1)
    Py_RETURN_NONE;
  const float* ps;
  if (!pair_weights(a[5], P, *p.xb, ps)) Py_RETURN_NONE;
  GQ_STREAM(*p.xb)
  Tensor out = output(*p.xb, at::kBFloat16, {P, unit ? p.N / 2 : p.N});
  const auto *xb = data<uint8_t>(*p.xb), *xs = data<uint8_t>(*p.xs);
  const auto *b = data<uint8_t>(*p.blocks), *s = data<uint8_t>(*p.scales);
  const auto *off = data<int32_t>(*r[0]), *sp = data<int32_t>(*r[1]), *tl = data<int32_t>(*r[2]),
             *nt = data<int32_t>(*r[3]);
  uint16_t* o = data<uint16_t>(out);
  const int st = unit ? launch(k8 ? lib.gemm8_unit : lib.gemm_unit, xb, xs, p.rows, p.K, b, s, p.E, p.N, k, (float)alpha,
                               (float)limit, off, sp, tl, nt, v[0], v[1], o, stream)
                      : launch(k8 ? lib.gemm8 : lib.gemm, xb, xs, p.rows, p.K, b, s, p.E, p.N, k, ps, off,
                               sp, tl, nt, v[0], v[1], o, stream);
  if (st) return PyLong_FromLong(st);
  return wrap(out);
  END_HANDLE_TH_ERRORS
}
PyObject* fp4_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) { return gemm_call<false>(a, n); }
PyObject* fp8_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) { return gemm_call<true>(a, n); }

// route_sort(ids, num_experts, tile_m) -> (offsets, sorted, tiles, num_tiles)
PyObject* route_sort(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GQ_ARGS(3)
  const Tensor* ids = contiguous(a[0], at::kInt, 2);
  if (!ids || !PyLong_Check(a[1]) || !PyLong_Check(a[2])) Py_RETURN_NONE;
  const int64_t E = whole(a[1]), tm = whole(a[2]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const int64_t rows = ids->size(0), k = ids->size(1);
  if (rows < 1 || k < 1 || rows > INT32_MAX || k > INT32_MAX || E < 1 || E > INT32_MAX || tm < 1 ||
      tm > INT32_MAX)
    Py_RETURN_NONE;
  const int32_t most = lib.max_tiles((int32_t)rows, (int32_t)k, (int32_t)E, (int32_t)tm);
  if (most < 0) Py_RETURN_NONE;
  GQ_STREAM(*ids)
  Tensor off = output(*ids, at::kInt, {E + 1}), sp = output(*ids, at::kInt, {rows * k});
  Tensor tiles = output(*ids, at::kInt, {most, 2}), nt = output(*ids, at::kInt, {1});
  const int st = launch(lib.route_sort, data<int32_t>(*ids), rows, k, E, tm, data<int32_t>(off),
                        data<int32_t>(sp), data<int32_t>(tiles), most, data<int32_t>(nt), stream);
  if (st) return PyLong_FromLong(st);
  return pack({off, sp, tiles, nt});
  END_HANDLE_TH_ERRORS
}

// bind(addresses by name, current_device, raw_stream): the library's entry
// points and torch's two callables; all of them or, with an error, none
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  GQ_ARGS(3)
  if (!PyDict_Check(a[0])) {
    PyErr_SetString(PyExc_TypeError, "addresses by name expected");
    return nullptr;
  }
  auto get = [&](const char* name) -> void* {
    PyObject* o = PyDict_GetItemString(a[0], name);        // borrowed
    void* p = o ? PyLong_AsVoidPtr(o) : nullptr;
    if (!p && !PyErr_Occurred()) PyErr_SetString(PyExc_KeyError, name);
    return p;
  };
  Library l{};
#define GQ_BIND(field, name)                                                    \
  if (!(l.field = reinterpret_cast<decltype(l.field)>(get(#name)))) return nullptr;
  GQ_BIND(quantize, gq_mxfp4_quantize)
  GQ_BIND(topk, gq_moe_topk)
  GQ_BIND(topk_backward, gq_moe_topk_backward)
  GQ_BIND(decode, gq_moe_decode)
  GQ_BIND(gemv, gq_mxfp4_grouped_gemv_fp4)
  GQ_BIND(gemv_unit, gq_mxfp4_grouped_gemv_fp4_swiglu)
  GQ_BIND(gemm, gq_mxfp4_grouped_gemm_fp4)
  GQ_BIND(gemm_unit, gq_mxfp4_grouped_gemm_fp4_swiglu)
  GQ_BIND(route_sort, gq_route_sort)
  GQ_BIND(max_tiles, gq_route_max_tiles)
  GQ_BIND(quantize8, gq_mxfp8_quantize)
  GQ_BIND(gemv8, gq_mxfp4_grouped_gemv_fp8)
  GQ_BIND(gemv8_unit, gq_mxfp4_grouped_gemv_fp8_swiglu)
  GQ_BIND(gemm8, gq_mxfp4_grouped_gemm_fp8)
  GQ_BIND(gemm8_unit, gq_mxfp4_grouped_gemm_fp8_swiglu)
  GQ_BIND(norm, gq_rms_norm)
  GQ_BIND(norm_backward, gq_rms_norm_backward)
  GQ_BIND(norm_workspace, gq_rms_norm_backward_workspace)
  GQ_BIND(route, gq_moe_route)
  GQ_BIND(route_backward, gq_moe_route_backward)
  lib = l;
  Py_XINCREF(a[1]);
  Py_XINCREF(a[2]);
  Py_XDECREF(current_device);
  Py_XDECREF(raw_stream);
  current_device = a[1];
  raw_stream = a[2];
  Py_RETURN_NONE;
}

#define GQ_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GQ_METHOD(bind),       GQ_METHOD(quantize),
                         GQ_METHOD(moe_topk),   GQ_METHOD(moe_topk_backward),
                         GQ_METHOD(moe_decode), GQ_METHOD(fp4_gemv),
                         GQ_METHOD(fp4_gemm),   GQ_METHOD(route_sort),
                         GQ_METHOD(quantize8),  GQ_METHOD(rms_norm),
                         GQ_METHOD(fp8_gemv),   GQ_METHOD(rms_norm_backward),
                         GQ_METHOD(fp8_gemm),   GQ_METHOD(moe_route),
                         GQ_METHOD(moe_route_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) {
  PyObject* m = PyModule_Create(&module);
  // built against this torch; another one's tensors may be laid out otherwise
  // nor does another header's library take these arguments
  if (m && (PyModule_AddStringConstant(m, "torch_version", GQ_TORCH_VERSION) < 0 ||
            PyModule_AddStringConstant(m, "header_id", GQ_HEADER_ID) < 0)) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
