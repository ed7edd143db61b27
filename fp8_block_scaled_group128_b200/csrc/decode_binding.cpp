// Python binding of the calls that a decode step makes back to back on little
// data (norm and quantization, router, expert MLP): argument checks, output and
// workspace allocation and the C call in one native function each. The same in
// Python around ctypes takes 14 us for the norm's four outputs, most of the
// call; here it takes 6.
//
// Every function returns its outputs, or the FP8BS_ERR_* code (an int) that the
// C call gave; wrong types raise TypeError, wrong shapes, layouts and devices
// ValueError. The call is made with the operands' device current, on its current
// stream; outputs and workspaces that it allocates belong to that stream.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fp8bs.h"

namespace {

using at::Tensor;
using c10::IntArrayRef;
using c10::ScalarType;

const Tensor& cuda_tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda(), name,
                   " must be a CUDA tensor");
  return THPVariable_Unpack(o);
}

// A contiguous tensor of the given type, shape and device.
const Tensor& operand(PyObject* o, ScalarType type, IntArrayRef shape, c10::Device device,
                      const char* name) {
  const Tensor& t = cuda_tensor(o, name);
  TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", got ", t.sizes());
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
  TORCH_CHECK_VALUE(t.device() == device, name, " is on another device than the first operand");
  return t;
}

void* address(PyObject* o, ScalarType type, IntArrayRef shape, c10::Device device,
              const char* name) {
  return operand(o, type, shape, device, name).data_ptr();
}

IntArrayRef matrix(const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.dim() == 2, name, " must have two dimensions, got ", t.sizes());
  return t.sizes();
}

// A given output (checked), or a new one.
struct Output {
  PyObject* object = nullptr;   // owned
  void* data = nullptr;
  Output(PyObject* given, ScalarType type, IntArrayRef shape, c10::Device device, const char* name) {
    if (given != Py_None) {
      data = address(given, type, shape, device, name);
      Py_INCREF(given);
      object = given;
    } else {
      Tensor t = at::empty(shape, at::TensorOptions().dtype(type).device(device));
      data = t.data_ptr();
      object = THPVariable_Wrap(std::move(t));
      if (object == nullptr) throw python_error();
    }
  }
  Output() = default;
  Output(Output&& o) noexcept : object(o.object), data(o.data) { o.object = nullptr; }
  Output& operator=(Output&& o) noexcept {
    std::swap(object, o.object);
    data = o.data;
    return *this;
  }
  ~Output() { Py_XDECREF(object); }
  PyObject* release() {   // None where there is no output
    PyObject* o = object;
    object = nullptr;
    if (o == nullptr) Py_RETURN_NONE;
    return o;
  }
};

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(v);
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

void count(Py_ssize_t given, Py_ssize_t wanted) {
  TORCH_CHECK_TYPE(given == wanted, "expected ", wanted, " arguments, got ", given);
}

// The operands' device, current for the life of the object, and its stream.
struct Place {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;
  explicit Place(c10::Device device) {
    if (c10::cuda::current_device() != device.index()) guard.set_device(device);
    stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
  }
};

// (ue8m0, x, residual, weight, eps, q, s, y, residual_out, want_y)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const bool ue8m0 = truth(a[0]);
  const auto bf16 = c10::kBFloat16;
  const Tensor& x = cuda_tensor(a[1], "x");
  const IntArrayRef shape = matrix(x, "x");
  const c10::Device device = x.device();
  const int64_t M = shape[0], K = shape[1];
  const int64_t row[1] = {K}, groups[2] = {M, K / 128};
  const void* xp = address(a[1], bf16, shape, device, "x");
  const void* rp = a[2] == Py_None ? nullptr : address(a[2], bf16, shape, device, "residual");
  const void* wp = a[3] == Py_None ? nullptr : address(a[3], bf16, row, device, "weight");
  const float eps = number(a[4]);
  TORCH_CHECK_VALUE(rp != nullptr || a[8] == Py_None,
                    "residual_out without a residual would be a copy of x");
  const Place place(device);
  Output r, y;
  if (rp != nullptr) r = Output(a[8], bf16, shape, device, "residual_out");
  if (a[7] != Py_None || truth(a[9])) y = Output(a[7], bf16, shape, device, "y");
  Output q(a[5], c10::kByte, shape, device, "q");
  Output s(a[6], ue8m0 ? c10::kByte : c10::kFloat, groups, device, ue8m0 ? "s8" : "s");
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = ue8m0 ? fp8_add_rmsnorm_quant_ue8m0(xp, rp, wp, eps, M, K, r.data, y.data, q.data,
                                               static_cast<uint8_t*>(s.data), place.stream)
                 : fp8_add_rmsnorm_quant(xp, rp, wp, eps, M, K, r.data, y.data, q.data,
                                         static_cast<float*>(s.data), place.stream);
  Py_END_ALLOW_THREADS
  if (status != FP8BS_OK) return PyLong_FromLong(status);
  PyObject* out = PyTuple_New(4);
  if (out == nullptr) throw python_error();
  PyTuple_SET_ITEM(out, 0, q.release());
  PyTuple_SET_ITEM(out, 1, s.release());
  PyTuple_SET_ITEM(out, 2, y.release());
  PyTuple_SET_ITEM(out, 3, r.release());
  return out;
  END_HANDLE_TH_ERRORS
}

// (logits, top_k, scoring, bias, n_group, topk_group, renormalize, scale, ids, weights)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const Tensor& logits = cuda_tensor(a[0], "logits");
  const IntArrayRef shape = matrix(logits, "logits");
  const c10::Device device = logits.device();
  const ScalarType type = logits.scalar_type();
  TORCH_CHECK_TYPE(type == c10::kFloat || type == c10::kBFloat16,
                   "logits must be float32 or bfloat16, got ", type);
  const int64_t M = shape[0], E = shape[1], top_k = integer(a[1]), row[1] = {E};
  const void* lp = address(a[0], type, shape, device, "logits");
  const void* bp = a[3] == Py_None ? nullptr : address(a[3], c10::kFloat, row, device, "bias");
  const int scoring = static_cast<int>(integer(a[2]));
  const int64_t n_group = integer(a[4]), topk_group = integer(a[5]);
  const int renormalize = truth(a[6]);
  const float scale = number(a[7]);
  const int64_t out_shape[2] = {M, top_k < 0 ? 0 : top_k};
  const Place place(device);
  Output ids(a[8], c10::kInt, out_shape, device, "ids");
  Output weights(a[9], c10::kFloat, out_shape, device, "weights");
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = moe_route_topk(lp, type == c10::kBFloat16, static_cast<const float*>(bp), scoring, M, E,
                          top_k, n_group, topk_group, renormalize, scale,
                          static_cast<int32_t*>(ids.data), static_cast<float*>(weights.data),
                          place.stream);
  Py_END_ALLOW_THREADS
  if (status != FP8BS_OK) return PyLong_FromLong(status);
  PyObject* out = PyTuple_New(2);
  if (out == nullptr) throw python_error();
  PyTuple_SET_ITEM(out, 0, ids.release());
  PyTuple_SET_ITEM(out, 1, weights.release());
  return out;
  END_HANDLE_TH_ERRORS
}

// (ue8m0, qa, sa, ids, weights, qw_gate_up, sw_gate_up, qw_down, sw_down, first_expert, y,
//  workspace)
PyObject* mlp(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 12);
  const bool ue8m0 = truth(a[0]);
  const auto u8 = c10::kByte, f32 = c10::kFloat;
  const auto scales = ue8m0 ? u8 : f32;
  const Tensor& qa = cuda_tensor(a[1], "qa");
  const IntArrayRef shape = matrix(qa, "qa");
  const c10::Device device = qa.device();
  const int64_t M = shape[0], K = shape[1], top_k = matrix(cuda_tensor(a[3], "ids"), "ids")[1];
  const Tensor& down = cuda_tensor(a[7], "qw_down");
  TORCH_CHECK_VALUE(down.dim() == 3, "qw_down must have three dimensions, got ", down.sizes());
  const int64_t E = down.size(0), I = down.size(2), KB = K / 128, IB = I / 128;
  const int64_t pairs[2] = {M, top_k}, rows[2] = {M, KB};
  const int64_t gu[3] = {E, 2 * I, K}, gu_blocks[3] = {E, 2 * IB, KB};
  const int64_t dn[3] = {E, K, I}, dn_blocks[3] = {E, KB, IB};
  const void* qp = address(a[1], u8, shape, device, "qa");
  const void* sp = address(a[2], scales, rows, device, "sa");
  const void* ip = address(a[3], c10::kInt, pairs, device, "ids");
  const void* wp = address(a[4], f32, pairs, device, "weights");
  const void* qg = address(a[5], u8, gu, device, "qw_gate_up");
  const void* sg = address(a[6], scales, gu_blocks, device, "sw_gate_up");
  const void* qd = address(a[7], u8, dn, device, "qw_down");
  const void* sd = address(a[8], scales, dn_blocks, device, "sw_down");
  const int64_t first_expert = integer(a[9]);
  const Place place(device);
  Output y(a[10], c10::kBFloat16, shape, device, "y");
  Tensor own;
  void* workspace;
  size_t bytes;
  if (a[11] == Py_None) {
    bytes = fp8bs_moe_workspace_bytes(M, K, I, E, top_k);
    own = at::empty({static_cast<int64_t>(bytes)}, at::TensorOptions().dtype(u8).device(device));
    workspace = own.data_ptr();
  } else {
    const Tensor& w = cuda_tensor(a[11], "workspace");
    TORCH_CHECK_VALUE(w.device() == device && w.is_contiguous(),
                      "workspace must be a contiguous tensor on the operands' device");
    workspace = w.data_ptr();
    bytes = w.nbytes();
  }
  const int32_t* ids = static_cast<const int32_t*>(ip);
  const float* weights = static_cast<const float*>(wp);
  int status;
  Py_BEGIN_ALLOW_THREADS
  if (ue8m0) {
    status = fp8_moe_mlp_ue8m0(qp, static_cast<const uint8_t*>(sp), ids, weights, qg,
                               static_cast<const uint8_t*>(sg), qd,
                               static_cast<const uint8_t*>(sd), y.data, M, K, I, E, top_k,
                               first_expert, workspace, bytes, place.stream);
  } else {
    status = fp8_moe_mlp(qp, static_cast<const float*>(sp), ids, weights, qg,
                         static_cast<const float*>(sg), qd, static_cast<const float*>(sd), y.data,
                         M, K, I, E, top_k, first_expert, workspace, bytes, place.stream);
  }
  Py_END_ALLOW_THREADS
  if (status != FP8BS_OK) return PyLong_FromLong(status);
  return y.release();
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm)), METH_FASTCALL,
     nullptr},
    {"route", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(route)), METH_FASTCALL,
     nullptr},
    {"mlp", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(mlp)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decode", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode() { return PyModule_Create(&module); }
