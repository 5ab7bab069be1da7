// mrr_torch.cpp -- the short way from torch tensors to the experts' operators:
// their plain calls (outputs allocated by the call, tensors of the current
// device), of which the Python binding's checks and ctypes are most of the time
// when the work is small (quantising a row: 8.6 us of host time from Python, of
// which the launch is 2.8). Every function returns None for a call that is not
// of that kind or that the library refuses, without having launched anything;
// experts.py then makes the call itself and raises what there is to raise.
#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe_rerouting_v2.h"

namespace {

int wide_code(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return MRR_F16;
    case at::kBFloat16: return MRR_BF16;
    case at::kFloat: return MRR_F32;
    default: return -1;
  }
}

bool is_packed(const at::Tensor& t) {
  return t.scalar_type() == at::kFloat4_e2m1fn_x2 || t.scalar_type() == at::kByte;
}

// The tensors of one call: all plain, dense and on the current device.
struct Call {
  c10::Device device{c10::DeviceType::CPU};
  bool ok = true;

  const at::Tensor* take(PyObject* o) {
    if (!ok || !THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || !t.is_contiguous()) {
      ok = false;
    } else if (device.type() == c10::DeviceType::CPU) {
      device = t.device();
      ok = device.index() == c10::hip::current_device();
    } else {
      ok = t.device() == device;
    }
    return &t;
  }
  const at::Tensor* take_optional(PyObject* o) { return o == Py_None ? nullptr : take(o); }

  // A pair of packed rows and scales; the values of a row.
  int64_t rows(const at::Tensor* packed, const at::Tensor* scales, int64_t dims) {
    if (!ok || !is_packed(*packed) ||
        (scales->scalar_type() != at::kFloat8_e8m0fnu && scales->scalar_type() != at::kByte) ||
        packed->dim() < 1 || (dims >= 0 && packed->dim() != dims) || scales->dim() != packed->dim() + 1) {
      ok = false;
      return 0;
    }
    const int64_t n = packed->dim(), values = 2 * packed->size(n - 1);
    for (int64_t i = 0; i + 1 < n; ++i) ok = ok && scales->size(i) == packed->size(i);
    ok = ok && scales->size(n - 1) == (values + 63) / 64 && scales->size(n) == 2;
    return values;
  }

  at::Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
    return at::detail::empty_cuda(shape, t, device, std::nullopt);  // what at::empty comes to, without its dispatch
  }
  ihipStream_t* stream() const { return c10::hip::getCurrentHIPStream(device.index()).stream(); }
};

PyObject* none() { Py_RETURN_NONE; }

template <typename F>
mrr_status unlocked(F&& f) {
  mrr_status st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS return st;
}

void* ptr(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }

// quantize(x)
PyObject* quantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  const at::Tensor* x = n == 1 ? c.take(args[0]) : nullptr;
  if (x == nullptr || !c.ok || wide_code(x->scalar_type()) < 0 || x->dim() < 1) return none();
  const int64_t H = x->size(-1);
  if (H == 0 || H % 2 != 0) return none();
  c10::SmallVector<int64_t, 6> shape(x->sizes().begin(), x->sizes().end());
  shape.back() = H / 2;
  at::Tensor packed = c.empty(shape, at::kFloat4_e2m1fn_x2);
  shape.back() = (H + 63) / 64;
  shape.push_back(2);
  at::Tensor scales = c.empty(shape, at::kFloat8_e8m0fnu);
  mrr_mx_args a{x->data_ptr(), wide_code(x->scalar_type()), x->numel() / H, H, packed.data_ptr(), scales.data_ptr()};
  if (unlocked([&] { return mrr_mx_quantize(&a, c.stream()); }) != MRR_SUCCESS) return none();
  PyObject* p = THPVariable_Wrap(std::move(packed));
  PyObject* s = THPVariable_Wrap(std::move(scales));
  PyObject* r = PyTuple_Pack(2, p, s);
  Py_DECREF(p);
  Py_DECREF(s);
  return r;
  END_HANDLE_TH_ERRORS
}

// dequantize(packed, scales, dtype)
PyObject* dequantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 3 || !THPDtype_Check(args[2])) return none();
  const at::ScalarType dtype = reinterpret_cast<THPDtype*>(args[2])->scalar_type;
  Call c;
  const at::Tensor* packed = c.take(args[0]);
  const at::Tensor* scales = c.take(args[1]);
  if (!c.ok || wide_code(dtype) < 0) return none();
  const int64_t H = c.rows(packed, scales, -1);
  if (!c.ok || H == 0) return none();
  c10::SmallVector<int64_t, 6> shape(packed->sizes().begin(), packed->sizes().end());
  shape.back() = H;
  at::Tensor out = c.empty(shape, dtype);
  mrr_mx_args a{out.data_ptr(), wide_code(dtype), out.numel() / H, H, packed->data_ptr(), scales->data_ptr()};
  if (unlocked([&] { return mrr_mx_dequantize(&a, c.stream()); }) != MRR_SUCCESS) return none();
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// grouped_mm(tokens, scales, weight, weight_scales, expert_token_num, gated, row_weight, expert_token_num_type, dtype)
PyObject* grouped_mm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9 || !PyBool_Check(args[5]) || !PyLong_CheckExact(args[7]) || !THPDtype_Check(args[8])) return none();
  const bool gated = args[5] == Py_True;
  const at::ScalarType dtype = reinterpret_cast<THPDtype*>(args[8])->scalar_type;
  Call c;
  const at::Tensor* tokens = c.take(args[0]);
  const at::Tensor* scales = c.take(args[1]);
  const at::Tensor* weight = c.take(args[2]);
  const at::Tensor* weight_scales = c.take(args[3]);
  const at::Tensor* num = c.take(args[4]);
  const at::Tensor* row_weight = c.take_optional(args[6]);
  if (!c.ok || wide_code(dtype) < 0) return none();
  const int64_t K = c.rows(tokens, scales, 2), wk = c.rows(weight, weight_scales, 3);
  if (!c.ok || K != wk) return none();
  const int64_t A = tokens->size(0), E = weight->size(0), N = weight->size(1);
  const at::ScalarType counts = num->scalar_type();
  if ((counts != at::kInt && counts != at::kLong) || num->dim() != 1 || num->size(0) != E) return none();
  if (row_weight != nullptr &&
      (row_weight->scalar_type() != at::kFloat || row_weight->dim() > 2 || row_weight->numel() != A))
    return none();
  const int64_t type = PyLong_AsLongLong(args[7]);
  if (type == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return none();
  }
  at::Tensor out = c.empty({A, gated ? N / 2 : N}, dtype);
  const mrr_grouped_mm_args a{tokens->data_ptr(), scales->data_ptr(), A, K, weight->data_ptr(),
                              weight_scales->data_ptr(), E, N, num->data_ptr(),
                              counts == at::kLong ? MRR_I64 : MRR_I32, type, gated,
                              static_cast<const float*>(ptr(row_weight)), out.data_ptr(), wide_code(dtype)};
  if (unlocked([&] { return mrr_mx_grouped_mm(&a, nullptr, 0, c.stream()); }) != MRR_SUCCESS) return none();
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// few_tokens(x, gate_up, down, router_logits, top_k, renormalize, expert_ids, expert_weight, gate_up_scales, down_scales)
PyObject* few_tokens(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 10 || !PyBool_Check(args[5])) return none();
  Call c;
  const at::Tensor* x = c.take(args[0]);
  const at::Tensor* gate_up = c.take(args[1]);
  const at::Tensor* down = c.take(args[2]);
  const at::Tensor* logits = c.take_optional(args[3]);
  const at::Tensor* ids = c.take_optional(args[6]);
  const at::Tensor* weight = c.take_optional(args[7]);
  const at::Tensor* gate_up_scales = c.take_optional(args[8]);
  const at::Tensor* down_scales = c.take_optional(args[9]);
  if (!c.ok || x->dim() != 2 || gate_up->dim() != 3 || down->dim() != 3) return none();
  const at::ScalarType dtype = x->scalar_type();
  if (dtype != at::kHalf && dtype != at::kBFloat16) return none();
  const bool mx = gate_up_scales != nullptr;
  if (mx != (down_scales != nullptr) || (logits != nullptr) == (ids != nullptr) ||
      (ids != nullptr) != (weight != nullptr))
    return none();
  const int64_t T = x->size(0), H = x->size(1), E = gate_up->size(0);
  int64_t h = gate_up->size(2), I = down->size(2);
  if (mx) {
    h = c.rows(gate_up, gate_up_scales, 3);
    I = c.rows(down, down_scales, 3);
    if (!c.ok) return none();
  } else if (gate_up->scalar_type() != dtype || down->scalar_type() != dtype) {
    return none();
  }
  if (h != H || gate_up->size(1) != 2 * I || down->size(0) != E || down->size(1) != H) return none();
  int64_t k;
  if (logits != nullptr) {
    if (logits->scalar_type() != at::kFloat || logits->dim() != 2 || logits->size(0) != T || logits->size(1) != E ||
        !PyLong_CheckExact(args[4]))
      return none();
    k = PyLong_AsLongLong(args[4]);
    if (k == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      return none();
    }
    if (k > E) return none();
  } else {
    if (ids->scalar_type() != at::kInt || weight->scalar_type() != at::kFloat || ids->dim() != 2 ||
        ids->size(0) != T || weight->sizes() != ids->sizes() || args[4] != Py_None)
      return none();
    k = ids->size(1);
  }
  const int64_t bytes = static_cast<int64_t>(mrr_few_tokens_workspace_size(T, k, I));
  if (bytes == 0) return none();
  at::Tensor y = c.empty({T, H}, dtype), ws = c.empty({bytes}, at::kByte);
  const int code = wide_code(dtype);
  const mrr_few_tokens_args a{x->data_ptr(), code, T, H, E, I, k, static_cast<const float*>(ptr(logits)),
                              args[5] == Py_True, static_cast<const int32_t*>(ptr(ids)),
                              static_cast<const float*>(ptr(weight)), mx ? MRR_F4_E2M1 : code, gate_up->data_ptr(),
                              ptr(gate_up_scales), down->data_ptr(), ptr(down_scales), y.data_ptr()};
  if (unlocked([&] { return mrr_few_tokens(&a, ws.data_ptr(), static_cast<size_t>(bytes), c.stream()); }) != MRR_SUCCESS)
    return none();
  return THPVariable_Wrap(std::move(y));
  END_HANDLE_TH_ERRORS
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"quantize", fast(quantize), METH_FASTCALL, nullptr},
                         {"dequantize", fast(dequantize), METH_FASTCALL, nullptr},
                         {"grouped_mm", fast(grouped_mm), METH_FASTCALL, nullptr},
                         {"few_tokens", fast(few_tokens), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mrr_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mrr_torch() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "source_hash", MRR_SOURCE_HASH) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
