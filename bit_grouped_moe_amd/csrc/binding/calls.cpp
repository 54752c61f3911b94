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

// quantize(x, want_values) -> (blocks, scales[, values])
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GQ_ARGS(2)
  const Tensor* x = device_tensor(a[0]);
  const int code = x ? float_code(*x) : -1;
  if (code < 0 || x->dim() < 1) Py_RETURN_NONE;
  const int64_t K = x->size(-1);
  if (K <= 0 || K % 32 || K > INT32_MAX || x->numel() == 0) Py_RETURN_NONE;
  const int64_t rows = x->numel() / K;
  int64_t stride = K;
  if (!x->is_contiguous()) {
    if (x->dim() != 2 || x->stride(1) != 1) Py_RETURN_NONE;
    if (rows > 1) stride = x->stride(0);
  }
  GQ_STREAM(*x)
  const bool want = a[1] == Py_True;
  auto shape = x->sizes().vec();
  shape.back() = K / 32;
  Tensor scales = output(*x, at::kByte, shape);
  shape.push_back(16);
  Tensor blocks = output(*x, at::kByte, shape);
  Tensor values;
  if (want) values = output(*x, at::kBFloat16, x->sizes());
  const int st = launch(lib.quantize, x->data_ptr(), code, rows, (int32_t)K, stride,
                        data<uint8_t>(blocks), data<uint8_t>(scales),
                        want ? data<uint16_t>(values) : nullptr, stream);
  if (st) return PyLong_FromLong(st);
  return want ? pack({blocks, scales, values}) : pack({blocks, scales});
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

// The operands of an MXFP4 x MXFP4 product.
struct Pair {
  const Tensor *xb, *xs, *blocks, *scales;
  int64_t rows, E, N, K;
};
bool mx_pair(PyObject* const* a, Pair& p) {
  p.xb = contiguous(a[0], at::kByte, 3);
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
         p.scales->size(2) == nb && p.xb->size(1) == nb && p.xb->size(2) == 16 &&
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
PyObject* fp4_gemv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GQ_ARGS(9)
  Pair p;
  const Tensor* ids = contiguous(a[4], at::kInt, 2);
  const bool unit = a[6] == Py_True;
  if (!mx_pair(a, p) || !ids || ids->size(0) != p.rows || ids->size(1) < 1 ||
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
  const int st = unit ? launch(lib.gemv_unit, xb, xs, p.rows, p.K, b, s, p.E, p.N, id, k,
                               (float)alpha, (float)limit, o, stream)
                      : launch(lib.gemv, xb, xs, p.rows, p.K, b, s, p.E, p.N, id, k, ps, o, stream);
  if (st) return PyLong_FromLong(st);
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// fp4_gemm(x blocks, x scales, blocks, scales, route, pair_scale, unit, alpha, limit)
PyObject* fp4_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GQ_ARGS(9)
  Pair p;
  const bool unit = a[6] == Py_True;
  // expert_offsets, sorted_pairs, tiles, num_tiles, max_tiles, tile_m, rows, topk, num_experts
  if (!mx_pair(a, p) || !PyTuple_Check(a[4]) || PyTuple_GET_SIZE(a[4]) != 9 || (unit && p.N % 2))
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
  const int st = unit ? launch(lib.gemm_unit, xb, xs, p.rows, p.K, b, s, p.E, p.N, k, (float)alpha,
                               (float)limit, off, sp, tl, nt, v[0], v[1], o, stream)
                      : launch(lib.gemm, xb, xs, p.rows, p.K, b, s, p.E, p.N, k, ps, off, sp, tl,
                               nt, v[0], v[1], o, stream);
  if (st) return PyLong_FromLong(st);
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

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
