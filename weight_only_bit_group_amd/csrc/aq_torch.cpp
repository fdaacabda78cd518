// The MXFP4 calls of the torch binding on their common path, as a CPython module: arguments
// looked over, outputs allocated and the C entry point called without a step of Python (a call
// on a few rows is bound by the host: 7.6 us from Python through ctypes, 4.1 here, 3.3 of them the launch).
//
// Every function takes the binding function's arguments in order and returns its result, or
// None for whatever it does not do itself: an argument that fails a check, tensors on another
// device than the current one, an empty product, a status other than AQ_OK.  binding.py then
// goes through the same call step by step and names what is wrong.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

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

#define AQ_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr

PyMethodDef methods[] = {{"quantize", AQ_FAST(quantize)},
                         {"dequantize", AQ_FAST(dequantize)},
                         {"gemm", AQ_FAST((product<false, false>))},
                         {"gemm_a4", AQ_FAST((product<true, false>))},
                         {"grouped_gemm", AQ_FAST((product<false, true>))},
                         {"grouped_gemm_a4", AQ_FAST((product<true, true>))},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_aq_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__aq_torch() { return PyModule_Create(&module); }
