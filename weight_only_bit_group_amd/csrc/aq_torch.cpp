// The MXFP4, FP8 and routing calls of the torch binding on their common path, as a CPython module: arguments
// looked over, outputs allocated and the C entry point called without a step of Python (a call
// on a few rows is bound by the host: 7.6 us from Python through ctypes, 4.1 here, 3.3 of them the launch).
//
// Every function takes the binding function's arguments in order and returns its result, or
// None for whatever it does not do itself: an argument that fails a check, tensors on another
// device than the current one, an empty product, a status other than AQ_OK.  binding.py then
// goes through the same call step by step and names what is wrong.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/functions/accumulate_grad.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/saved_variable.h>

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <unordered_set>
#include <vector>

#include "aq.h"

namespace {

constexpr auto F32 = at::kFloat, BF16 = at::kBFloat16, U8 = at::kByte, I32 = at::kInt;

// the current device, or -1 unless the first argument is a GPU tensor (no device is asked for then)
int device_for(PyObject* first) {
  return THPVariable_CheckExact(first) && THPVariable_Unpack(first).is_cuda() ? c10::hip::current_device() : -1;
}

// a plain tensor on the current device with this type and these dimensions, or null
const at::Tensor* tensor(PyObject* o, int dims, int device) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.get_device() == device && t.dim() == dims ? &t : nullptr;
}

const at::Tensor* dense(PyObject* o, int dims, int device, at::ScalarType type) {
  const at::Tensor* t = tensor(o, dims, device);
  return t && t->scalar_type() == type && t->is_contiguous() ? t : nullptr;
}

// A matrix whose rows are dense: bf16 (or fp32), or MXFP4 codes with their scale bytes.
struct Rows {
  const at::Tensor* x = nullptr;
  const at::Tensor* scales = nullptr;
  int64_t m = 0, k = 0, ld = 0;
};

bool rows_of(PyObject* o, int device, bool or_f32, Rows& r) {
  r.x = tensor(o, 2, device);
  if (!r.x || !(r.x->scalar_type() == BF16 || (or_f32 && r.x->scalar_type() == F32))) return false;
  r.m = r.x->size(0);
  r.k = r.x->size(1);
  r.ld = r.m > 1 ? r.x->stride(0) : r.k;   // (the stride of a single row says nothing)
  return r.m > 0 && r.k > 0 && r.k % 32 == 0 && r.x->stride(1) == 1 && r.ld >= r.k;
}

bool codes_of(PyObject* codes, PyObject* scales, int device, Rows& r) {
  r.x = dense(codes, 2, device, U8);
  r.scales = dense(scales, 2, device, U8);
  if (!r.x || !r.scales) return false;
  r.m = r.x->size(0);
  r.k = 2 * r.x->size(1);
  return r.m > 0 && r.k > 0 && r.k % 32 == 0 && r.scales->size(0) == r.m && r.scales->size(1) == r.k / 32;
}

// weights [(E,) N, K/2] and [(E,) N, K/32]
struct Weights {
  const at::Tensor *codes = nullptr, *scales = nullptr;
  int64_t e = 1, n = 0;
};

bool weights_of(PyObject* codes, PyObject* scales, int dims, int device, int64_t k, Weights& w) {
  w.codes = dense(codes, dims, device, U8);
  w.scales = dense(scales, dims, device, U8);
  if (!w.codes || !w.scales) return false;
  if (dims == 3) w.e = w.codes->size(0);
  w.n = w.codes->size(dims - 2);
  return w.n > 0 && w.codes->size(dims - 1) * 2 == k && w.scales->size(dims - 1) == k / 32 &&
         w.scales->size(dims - 2) == w.n && (dims == 2 || w.scales->size(0) == w.e);
}

// The output [m, n]: `given`, or a new tensor of the type that out_dtype names (fp32 without one).
struct Output {
  at::Tensor fresh;
  const at::Tensor* y = nullptr;
  PyObject* given = nullptr;
  int32_t dtype = AQ_F32;

  bool make(PyObject* out_dtype, PyObject* out, int64_t m, int64_t n, int device) {
    at::ScalarType type = F32;
    if (out_dtype != Py_None) {
      if (!THPDtype_Check(out_dtype)) return false;
      type = reinterpret_cast<THPDtype*>(out_dtype)->scalar_type;
    }
    if (out != Py_None) {
      y = tensor(out, 2, device);
      if (!y || !y->is_contiguous() || y->size(0) != m || y->size(1) != n) return false;
      if (out_dtype != Py_None && type != y->scalar_type()) return false;
      type = y->scalar_type();
      given = out;
    }
    if (type != F32 && type != BF16) return false;
    dtype = type == F32 ? AQ_F32 : AQ_BF16;
    if (!given) {
      fresh = at::empty({m, n}, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)device));
      y = &fresh;
    }
    return true;
  }
  PyObject* result() {
    if (!given) return THPVariable_Wrap(std::move(fresh));
    Py_INCREF(given);
    return given;
  }
};

void* stream_of(int device) { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream(); }

const uint8_t* bytes(const at::Tensor* t) { return static_cast<const uint8_t*>(t->const_data_ptr()); }

// the call without the interpreter lock, as through ctypes
template <class F>
bool succeeds(F call) {
  aq_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = call();
  Py_END_ALLOW_THREADS;
  return st == AQ_OK;
}

// X, [x_scales,] codes, scales, [offsets, rows,] out_dtype, out
template <bool A4, bool GROUPED>
PyObject* product(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 5 + A4 + 2 * GROUPED) Py_RETURN_NONE;
  const int device = device_for(args[0]);
  if (device < 0) Py_RETURN_NONE;
  PyObject* const* rest = args + 1 + A4;
  Rows x;
  if (!(A4 ? codes_of(args[0], args[A4], device, x) : rows_of(args[0], device, false, x))) Py_RETURN_NONE;
  Weights w;
  if (!weights_of(rest[0], rest[1], GROUPED ? 3 : 2, device, x.k, w)) Py_RETURN_NONE;
  int64_t m = x.m;
  const int32_t *offsets = nullptr, *rows = nullptr;
  if constexpr (GROUPED) {
    const at::Tensor* o = dense(rest[2], 1, device, I32);
    if (!o || o->size(0) != w.e + 1) Py_RETURN_NONE;
    offsets = o->const_data_ptr<int32_t>();
    if (rest[3] != Py_None) {
      const at::Tensor* r = dense(rest[3], 1, device, I32);
      if (!r || r->size(0) == 0) Py_RETURN_NONE;
      rows = r->const_data_ptr<int32_t>();
      m = r->size(0);
    }
    rest += 2;
  }
  Output y;
  if (!y.make(rest[2], rest[3], m, w.n, device)) Py_RETURN_NONE;
  void* const stream = stream_of(device);
  void* const to = y.y->data_ptr();
  const bool ok = succeeds([&] {
    if constexpr (GROUPED && A4)
      return aq_mxfp4_grouped_gemm_a4(bytes(x.x), bytes(x.scales), x.m, x.k, bytes(w.codes), bytes(w.scales), w.e, w.n,
                                      offsets, rows, m, to, y.dtype, stream);
    else if constexpr (GROUPED)
      return aq_mxfp4_grouped_gemm(static_cast<const uint16_t*>(x.x->const_data_ptr()), x.m, x.k, x.ld, bytes(w.codes),
                                   bytes(w.scales), w.e, w.n, offsets, rows, m, to, y.dtype, stream);
    else if constexpr (A4)
      return aq_mxfp4_gemm_a4(bytes(x.x), bytes(x.scales), m, x.k, bytes(w.codes), bytes(w.scales), w.n, to, y.dtype,
                              stream);
    else
      return aq_mxfp4_gemm(static_cast<const uint16_t*>(x.x->const_data_ptr()), m, x.k, x.ld, bytes(w.codes),
                           bytes(w.scales), w.n, to, y.dtype, stream);
  });
  if (!ok) Py_RETURN_NONE;
  return y.result();
  END_HANDLE_TH_ERRORS
}

// X -> (codes, scales)
PyObject* quantize(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 1) Py_RETURN_NONE;
  const int device = device_for(args[0]);
  if (device < 0) Py_RETURN_NONE;
  Rows x;
  if (!rows_of(args[0], device, true, x)) Py_RETURN_NONE;
  const auto options = at::TensorOptions().dtype(U8).device(at::kCUDA, (c10::DeviceIndex)device);
  at::Tensor codes = at::empty({x.m, x.k / 2}, options), scales = at::empty({x.m, x.k / 32}, options);
  void* const stream = stream_of(device);
  auto* c = static_cast<uint8_t*>(codes.data_ptr());
  auto* s = static_cast<uint8_t*>(scales.data_ptr());
  const bool ok = succeeds([&] {
    return aq_mxfp4_quantize(x.x->const_data_ptr(), x.x->scalar_type() == F32 ? AQ_F32 : AQ_BF16, x.m, x.k, x.ld, c, s,
                             stream);
  });
  if (!ok) Py_RETURN_NONE;
  PyObject* pair = PyTuple_New(2);
  if (!pair) return nullptr;
  PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(std::move(codes)));
  PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(std::move(scales)));
  return pair;
  END_HANDLE_TH_ERRORS
}

// codes, scales, out_dtype, out
PyObject* dequantize(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 4) Py_RETURN_NONE;
  const int device = device_for(args[0]);
  if (device < 0) Py_RETURN_NONE;
  Rows x;
  if (!codes_of(args[0], args[1], device, x)) Py_RETURN_NONE;
  Output y;
  if (!y.make(args[2], args[3], x.m, x.k, device)) Py_RETURN_NONE;
  void* const stream = stream_of(device);
  void* const to = y.y->data_ptr();
  if (!succeeds([&] { return aq_mxfp4_dequantize(bytes(x.x), bytes(x.scales), x.m, x.k, to, y.dtype, stream); }))
    Py_RETURN_NONE;
  return y.result();
  END_HANDLE_TH_ERRORS
}

// ---- FP8 ------------------------------------------------------------------------------------

constexpr auto F8 = at::kFloat8_e4m3fn;

int64_t blocks(int64_t n) { return (n + 127) / 128; }

const at::Tensor* dense_of(PyObject* o, int device, at::ScalarType type, at::IntArrayRef shape) {
  const at::Tensor* t = dense(o, (int)shape.size(), device, type);
  return t && t->sizes() == shape ? t : nullptr;
}

// FP8 codes (or the same bytes as uint8)
const at::Tensor* f8_codes(PyObject* o, int dims, int device) {
  const at::Tensor* t = tensor(o, dims, device);
  return t && (t->scalar_type() == F8 || t->scalar_type() == U8) && t->is_contiguous() ? t : nullptr;
}

int32_t code_of(const at::Tensor* t) { return t->scalar_type() == F32 ? AQ_F32 : AQ_BF16; }

// a matrix [M, K] of fp32 or bf16 values whose rows are dense
bool f8_rows(PyObject* o, int device, Rows& r) {
  r.x = tensor(o, 2, device);
  if (!r.x || !(r.x->scalar_type() == BF16 || r.x->scalar_type() == F32)) return false;
  r.m = r.x->size(0);
  r.k = r.x->size(1);
  r.ld = r.m > 1 ? r.x->stride(0) : r.k;
  return r.m > 0 && r.k > 0 && r.k % 16 == 0 && r.x->stride(1) == 1 && r.ld >= r.k;
}

// codes [M, K], scales [M, blocks of K]
bool f8_pair(PyObject* codes, PyObject* scales, int device, Rows& r) {
  r.x = f8_codes(codes, 2, device);
  if (!r.x) return false;
  r.m = r.x->size(0);
  r.k = r.x->size(1);
  r.scales = dense_of(scales, device, F32, {r.m, blocks(r.k)});
  return r.scales && r.m > 0 && r.k > 0 && r.k % 16 == 0;
}

// weights [(E,) N, K] in blocks of 128 x 128
bool f8_weights(PyObject* codes, PyObject* scales, int dims, int device, int64_t k, Weights& w) {
  w.codes = f8_codes(codes, dims, device);
  if (!w.codes) return false;
  if (dims == 3) w.e = w.codes->size(0);
  w.n = w.codes->size(dims - 2);
  w.scales = dims == 3 ? dense_of(scales, device, F32, {w.e, blocks(w.n), blocks(k)})
                       : dense_of(scales, device, F32, {blocks(w.n), blocks(k)});
  return w.scales && w.e > 0 && w.n > 0 && w.codes->size(dims - 1) == k;
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int device) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)device));
}

template <class... T>
PyObject* tuple_of(T&&... t) {
  PyObject* o = PyTuple_New(sizeof...(T));
  if (!o) return nullptr;
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(o, i++, THPVariable_Wrap(std::move(t))), ...);
  return o;
}

const float* floats(const at::Tensor* t) { return static_cast<const float*>(t->const_data_ptr()); }
const int32_t* ints(const at::Tensor* t) { return static_cast<const int32_t*>(t->const_data_ptr()); }

// X, block_rows -> (codes, scales)
PyObject* f8_quantize(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 2 || !PyLong_CheckExact(args[1])) Py_RETURN_NONE;
  const int device = device_for(args[0]);
  if (device < 0) Py_RETURN_NONE;
  Rows x;
  const long rows = PyLong_AsLong(args[1]);
  if (rows == -1 && PyErr_Occurred()) PyErr_Clear();
  if ((rows != 1 && rows != 128) || !f8_rows(args[0], device, x)) Py_RETURN_NONE;
  at::Tensor codes = fresh({x.m, x.k}, F8, device), scales = fresh({rows == 1 ? x.m : blocks(x.m), blocks(x.k)}, F32, device);
  void* const stream = stream_of(device);
  auto* c = static_cast<uint8_t*>(codes.data_ptr());
  auto* s = static_cast<float*>(scales.data_ptr());
  if (!succeeds([&] {
        return aq_fp8_quantize(x.x->const_data_ptr(), code_of(x.x), 1, x.m, x.k, x.ld, (int32_t)rows, c, s, stream);
      }))
    Py_RETURN_NONE;
  return tuple_of(codes, scales);
  END_HANDLE_TH_ERRORS
}

// codes [N, K], scales, block_rows, out_dtype, out
PyObject* f8_dequantize(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 5 || !PyLong_CheckExact(args[2])) Py_RETURN_NONE;
  const int device = device_for(args[0]);
  if (device < 0) Py_RETURN_NONE;
  const at::Tensor* codes = f8_codes(args[0], 2, device);
  const long rows = PyLong_AsLong(args[2]);
  if (rows == -1 && PyErr_Occurred()) PyErr_Clear();
  if (!codes || (rows != 1 && rows != 128)) Py_RETURN_NONE;
  const int64_t n = codes->size(0), k = codes->size(1);
  const at::Tensor* scales = dense_of(args[1], device, F32, {rows == 1 ? n : blocks(n), blocks(k)});
  if (!scales || n == 0 || k == 0 || k % 16) Py_RETURN_NONE;
  Output y;
  if (!y.make(args[3], args[4], n, k, device)) Py_RETURN_NONE;
  void* const stream = stream_of(device);
  void* const to = y.y->data_ptr();
  if (!succeeds([&] { return aq_fp8_dequantize(bytes(codes), floats(scales), 1, n, k, (int32_t)rows, to, y.dtype, stream); }))
    Py_RETURN_NONE;
  return y.result();
  END_HANDLE_TH_ERRORS
}

// X_codes, X_scales, codes, scales, [offsets, rows,] out_dtype, out
template <bool GROUPED>
PyObject* f8_product(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 6 + 2 * GROUPED) Py_RETURN_NONE;
  const int device = device_for(args[0]);
  if (device < 0) Py_RETURN_NONE;
  Rows x;
  if (!f8_pair(args[0], args[1], device, x)) Py_RETURN_NONE;
  Weights w;
  if (!f8_weights(args[2], args[3], GROUPED ? 3 : 2, device, x.k, w)) Py_RETURN_NONE;
  int64_t m = x.m;
  const int32_t *offsets = nullptr, *rows = nullptr;
  if constexpr (GROUPED) {
    const at::Tensor* o = dense_of(args[4], device, I32, {w.e + 1});
    if (!o) Py_RETURN_NONE;
    offsets = ints(o);
    if (args[5] != Py_None) {
      const at::Tensor* r = dense(args[5], 1, device, I32);
      if (!r || r->size(0) == 0) Py_RETURN_NONE;
      rows = ints(r);
      m = r->size(0);
    }
  }
  Output y;
  if (!y.make(args[nargs - 2], args[nargs - 1], m, w.n, device)) Py_RETURN_NONE;
  void* const stream = stream_of(device);
  void* const to = y.y->data_ptr();
  const bool ok = succeeds([&] {
    if constexpr (GROUPED)
      return aq_fp8_grouped_gemm(bytes(x.x), floats(x.scales), x.m, x.k, bytes(w.codes), floats(w.scales), w.e, w.n, offsets,
                                 rows, m, to, y.dtype, stream);
    else
      return aq_fp8_gemm(bytes(x.x), floats(x.scales), m, x.k, bytes(w.codes), floats(w.scales), w.n, to, y.dtype, stream);
  });
  if (!ok) Py_RETURN_NONE;
  return y.result();
  END_HANDLE_TH_ERRORS
}

// X, codes, scales, out_dtype, out
PyObject* f8_linear(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 5) Py_RETURN_NONE;
  const int device = device_for(args[0]);
  if (device < 0) Py_RETURN_NONE;
  Rows x;
  if (!f8_rows(args[0], device, x)) Py_RETURN_NONE;
  Weights w;
  if (!f8_weights(args[1], args[2], 2, device, x.k, w)) Py_RETURN_NONE;
  Output y;
  if (!y.make(args[3], args[4], x.m, w.n, device)) Py_RETURN_NONE;
  const size_t need = aq_fp8_linear_workspace(x.m, x.k);
  at::Tensor workspace = fresh({(int64_t)need}, U8, device);
  void* const stream = stream_of(device);
  void* const to = y.y->data_ptr();
  void* const work = workspace.data_ptr();
  if (!succeeds([&] {
        return aq_fp8_linear(x.x->const_data_ptr(), code_of(x.x), x.m, x.k, x.ld, bytes(w.codes), floats(w.scales), w.n, to,
                             y.dtype, work, need, stream);
      }))
    Py_RETURN_NONE;
  return y.result();
  END_HANDLE_TH_ERRORS
}

// ---- routing --------------------------------------------------------------------------------

bool integer(PyObject* o, int64_t& v) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  v = PyLong_AsLongLongAndOverflow(o, &over);
  return !over;
}

bool number(PyObject* o, float& v) {
  if (!PyFloat_CheckExact(o) && !PyLong_CheckExact(o)) return false;
  const double d = PyFloat_AsDouble(o);
  if (d == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  v = (float)d;
  return true;
}

bool score_of(PyObject* o, int32_t& score) {
  if (!PyUnicode_CheckExact(o)) return false;
  if (PyUnicode_CompareWithASCIIString(o, "softmax") == 0) score = AQ_SOFTMAX;
  else if (PyUnicode_CompareWithASCIIString(o, "sigmoid") == 0) score = AQ_SIGMOID;
  else return false;
  return true;
}

// logits [T, E] with dense rows
bool logits_of(PyObject* o, int device, Rows& r) {
  r.x = tensor(o, 2, device);
  if (!r.x || !(r.x->scalar_type() == BF16 || r.x->scalar_type() == F32)) return false;
  r.m = r.x->size(0);
  r.k = r.x->size(1);
  r.ld = r.m > 1 ? r.x->stride(0) : r.k;
  return r.m > 0 && r.k > 0 && (r.k == 1 || r.x->stride(1) == 1) && r.ld >= r.k;
}

// logits [T, E], top, score, bias, groups, top_groups, renormalize, scale, as the binding takes them
struct Routing {
  Rows l;
  int64_t top = 0, groups = 0, top_groups = 0;
  int32_t score = 0;
  bool renormalize = false;
  float scale = 0;
  const at::Tensor* bias = nullptr;
  at::Tensor ids, weights;

  bool read(PyObject* const* args, int device) {
    if (!logits_of(args[0], device, l) || !integer(args[1], top) || !score_of(args[2], score) || !integer(args[4], groups) ||
        !(args[5] == Py_None || integer(args[5], top_groups)) || !PyBool_Check(args[6]) || !number(args[7], scale))
      return false;
    if (args[5] == Py_None) top_groups = groups;
    renormalize = args[6] == Py_True;
    if (top <= 0 || top > std::min<int64_t>(l.k, 64) || groups <= 0 || groups > 64 || top_groups <= 0 || top_groups > 64)
      return false;
    return args[3] == Py_None || (bias = dense_of(args[3], device, F32, {l.k}));
  }
  bool run(int device) {
    ids = fresh({l.m, top}, I32, device);
    weights = fresh({l.m, top}, F32, device);
    void* const stream = stream_of(device);
    auto* i = static_cast<int32_t*>(ids.data_ptr());
    auto* w = static_cast<float*>(weights.data_ptr());
    return succeeds([&] {
      return aq_moe_route(l.x->const_data_ptr(), code_of(l.x), l.m, l.k, l.ld, top, score, bias ? floats(bias) : nullptr,
                          (int32_t)groups, (int32_t)top_groups, renormalize, scale, i, w, stream);
    });
  }
};

// -> (ids, weights)
PyObject* route(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 8) Py_RETURN_NONE;
  const int device = device_for(args[0]);
  if (device < 0) Py_RETURN_NONE;
  Routing r;
  if (!r.read(args, device) || !r.run(device)) Py_RETURN_NONE;
  return tuple_of(r.ids, r.weights);
  END_HANDLE_TH_ERRORS
}

// Whether the current stream is being captured while a leaf that t was computed from belongs to a graph of an earlier
// call on another stream.  Its node accumulates on that stream: a captured backward pass would send work there, which
// breaks the capture in a thread of torch's engine.
bool capture_conflict(const at::Tensor& t, int device) {
  if (!at::GradMode::is_enabled() || !t.requires_grad()) return false;
  hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
  const auto stream = c10::hip::getCurrentHIPStream((c10::DeviceIndex)device);
  if (hipStreamIsCapturing(stream.stream(), &status) != hipSuccess || status == hipStreamCaptureStatusNone) return false;
  std::vector<std::shared_ptr<torch::autograd::Node>> open;
  if (auto leaf = t.grad_fn() ? t.grad_fn() : torch::autograd::impl::try_get_grad_accumulator(t)) open.push_back(leaf);
  std::unordered_set<torch::autograd::Node*> seen;
  while (!open.empty()) {
    const auto node = open.back();
    open.pop_back();
    if (!seen.insert(node.get()).second) continue;
    if (dynamic_cast<torch::autograd::AccumulateGrad*>(node.get())) {
      const auto on = node->stream();
      if (on && on->id() != stream.id()) return true;   // (the device type's name differs: only the numbers compare)
    }
    for (const auto& edge : node->next_edges())
      if (edge.function) open.push_back(edge.function);
  }
  return false;
}

// tensor -> bool
PyObject* conflict(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  const int device = nargs == 1 ? device_for(args[0]) : -1;
  return PyBool_FromLong(device >= 0 && capture_conflict(THPVariable_Unpack(args[0]), device));
  END_HANDLE_TH_ERRORS
}

// The gradient of route's weights with respect to the logits, as a node of torch's graph (from Python, applying the
// function and going back through it take 30 us of the host more).
struct RouteBackward : public torch::autograd::Node {
  torch::autograd::SavedVariable logits, ids, weights;
  int32_t score = 0;
  bool renormalize = false;
  float scale = 0;

  torch::autograd::variable_list apply(torch::autograd::variable_list&& grads) override {
    std::lock_guard<std::mutex> lock(mutex_);
    torch::autograd::variable_list out(1);
    if (!grads[0].defined() || !task_should_compute_output(0)) return out;
    const bool again = at::GradMode::is_enabled();   // (create_graph)
    {
      at::NoGradGuard no_grad;
      const at::Tensor l = logits.unpack(), i = ids.unpack(), w = weights.unpack(shared_from_this());
      const at::Tensor d = grads[0].to(F32).contiguous();
      const c10::OptionalDeviceGuard guard(l.device());
      out[0] = fresh({l.size(0), l.size(1)}, l.scalar_type(), l.get_device());
      const int64_t ld = l.size(0) > 1 ? l.stride(0) : l.size(1);
      const aq_status st = aq_moe_route_backward(l.const_data_ptr(), code_of(&l), l.size(0), l.size(1), ld, i.size(1), score,
                                                 renormalize, scale, ints(&i), floats(&w), floats(&d), out[0].data_ptr(),
                                                 stream_of(l.get_device()));
      TORCH_CHECK(st == AQ_OK, "aq_moe_route_backward: ", aq_last_error());
    }
    // The gradient is a function of the logits, whatever the gradient that came in, and not differentiable itself: asking
    // for its gradient is an error.
    if (again) {
      torch::autograd::DelayedError error("trying to differentiate the gradient of route", 1);
      out = error.apply({out[0].requires_grad_(true)});
    }
    return out;
  }
  void release_variables() override {
    std::lock_guard<std::mutex> lock(mutex_);
    logits.reset_data();
    ids.reset_data();
    weights.reset_data();
  }
  std::string name() const override { return "RouteBackward"; }
};

// -> (ids, weights), weights part of the graph where the logits are
PyObject* route_graph(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 8) Py_RETURN_NONE;
  const int device = device_for(args[0]);
  if (device < 0) Py_RETURN_NONE;
  Routing r;
  // (a conflict, or a tangent, is the caller's to report)
  if (!r.read(args, device) || r.l.x->_fw_grad(0).defined() || capture_conflict(*r.l.x, device) || !r.run(device)) Py_RETURN_NONE;
  if (at::GradMode::is_enabled() && r.l.x->requires_grad()) {
    auto node = std::shared_ptr<RouteBackward>(new RouteBackward(), torch::autograd::deleteNode);
    node->set_next_edges(torch::autograd::collect_next_edges(*r.l.x));
    node->score = r.score;
    node->renormalize = r.renormalize;
    node->scale = r.scale;
    torch::autograd::set_history(r.weights, node);
    node->logits = torch::autograd::SavedVariable(*r.l.x, false);
    node->ids = torch::autograd::SavedVariable(r.ids, false);
    node->weights = torch::autograd::SavedVariable(r.weights, true);
  }
  return tuple_of(r.ids, r.weights);
  END_HANDLE_TH_ERRORS
}

// logits, ids, weights, dweights, score, renormalize, scale -> dlogits
PyObject* route_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 7) Py_RETURN_NONE;
  const int device = device_for(args[0]);
  if (device < 0) Py_RETURN_NONE;
  Rows l;
  int32_t score = 0;
  float scale = 0;
  const at::Tensor* ids = dense(args[1], 2, device, I32);
  if (!ids || !logits_of(args[0], device, l) || !score_of(args[4], score) || !PyBool_Check(args[5]) || !number(args[6], scale))
    Py_RETURN_NONE;
  const int64_t top = ids->size(1);
  const at::Tensor *weights = dense_of(args[2], device, F32, {l.m, top}), *grad = dense_of(args[3], device, F32, {l.m, top});
  if (ids->size(0) != l.m || top == 0 || !weights || !grad) Py_RETURN_NONE;
  at::Tensor out = fresh({l.m, l.k}, l.x->scalar_type(), device);
  void* const stream = stream_of(device);
  void* const to = out.data_ptr();
  if (!succeeds([&] {
        return aq_moe_route_backward(l.x->const_data_ptr(), code_of(l.x), l.m, l.k, l.ld, top, score, args[5] == Py_True,
                                     scale, ints(ids), floats(weights), floats(grad), to, stream);
      }))
    Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// X, gate_up codes, scales, down codes, scales, ids [T, top], weights, out_dtype -> (out, products, slots)
PyObject* experts(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 8) Py_RETURN_NONE;
  const int device = device_for(args[0]);
  if (device < 0) Py_RETURN_NONE;
  Rows x;
  Weights up, down;
  if (!f8_rows(args[0], device, x) || !f8_weights(args[1], args[2], 3, device, x.k, up) || up.n % 2 ||
      !f8_weights(args[3], args[4], 3, device, up.n / 2, down) || down.e != up.e || down.n != x.k)
    Py_RETURN_NONE;
  const at::Tensor* ids = dense(args[5], 2, device, I32);
  if (!ids || ids->size(0) != x.m || ids->size(1) == 0) Py_RETURN_NONE;
  const int64_t top = ids->size(1), inner = up.n / 2;
  const at::Tensor* weights = dense_of(args[6], device, F32, {x.m, top});
  if (!weights) Py_RETURN_NONE;
  Output y;
  if (!y.make(args[7], Py_None, x.m, x.k, device)) Py_RETURN_NONE;
  const size_t need = aq_fp8_experts_workspace(x.m, top, x.k, up.e, inner);
  if (need == 0) Py_RETURN_NONE;
  at::Tensor products = fresh({x.m * top, x.k}, F32, device), slots = fresh({x.m, top}, I32, device);
  at::Tensor workspace = fresh({(int64_t)need}, U8, device);
  void* const stream = stream_of(device);
  void* const to = y.y->data_ptr();
  auto* p = static_cast<float*>(products.data_ptr());
  auto* s = static_cast<int32_t*>(slots.data_ptr());
  void* const work = workspace.data_ptr();
  if (!succeeds([&] {
        return aq_fp8_experts(x.x->const_data_ptr(), code_of(x.x), x.m, x.k, x.ld, bytes(up.codes), floats(up.scales),
                              bytes(down.codes), floats(down.scales), up.e, inner, ints(ids), floats(weights), top, p, s, to,
                              y.dtype, work, need, stream);
      }))
    Py_RETURN_NONE;
  return tuple_of(y.fresh, products, slots);
  END_HANDLE_TH_ERRORS
}

#define AQ_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr

PyMethodDef methods[] = {{"quantize", AQ_FAST(quantize)},
                         {"dequantize", AQ_FAST(dequantize)},
                         {"gemm", AQ_FAST((product<false, false>))},
                         {"gemm_a4", AQ_FAST((product<true, false>))},
                         {"grouped_gemm", AQ_FAST((product<false, true>))},
                         {"grouped_gemm_a4", AQ_FAST((product<true, true>))},
                         {"fp8_quantize", AQ_FAST(f8_quantize)},
                         {"fp8_dequantize", AQ_FAST(f8_dequantize)},
                         {"fp8_gemm", AQ_FAST(f8_product<false>)},
                         {"fp8_grouped_gemm", AQ_FAST(f8_product<true>)},
                         {"fp8_linear", AQ_FAST(f8_linear)},
                         {"fp8_experts", AQ_FAST(experts)},
                         {"route", AQ_FAST(route)},
                         {"route_graph", AQ_FAST(route_graph)},
                         {"capture_conflict", AQ_FAST(conflict)},
                         {"route_backward", AQ_FAST(route_backward)},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_aq_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__aq_torch() { return PyModule_Create(&module); }
