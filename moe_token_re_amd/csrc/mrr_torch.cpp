// mrr_torch.cpp -- the short way from torch tensors to the experts' operators and
// the ones around a layer: their plain calls (outputs allocated by the call, tensors of the current
// device), of which the Python binding's checks and ctypes are most of the time
// when the work is small (quantising a row: 8.6 us of host time from Python, of
// which the launch is 2.8). Every function returns None for a call that is not
// of that kind or that the library refuses, without having launched anything;
// experts.py or layer.py then makes the call itself and raises what there is to raise.
#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/GradMode.h>
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

// Whether autograd would have to record a call with these inputs, which no operator does.
bool recorded(std::initializer_list<const at::Tensor*> inputs) {
  if (!c10::GradMode::is_enabled()) return false;
  for (const at::Tensor* t : inputs)
    if (t != nullptr && t->requires_grad()) return true;
  return false;
}

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

// A result of several parts, None for those that are not there.
PyObject* result(std::initializer_list<at::Tensor*> parts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(parts.size()));
  Py_ssize_t i = 0;
  for (at::Tensor* t : parts) {
    PyObject* o = Py_None;
    if (t != nullptr && t->defined())
      o = THPVariable_Wrap(std::move(*t));
    else
      Py_INCREF(o);
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

bool same_shape(const at::Tensor* t, const at::Tensor* like) {
  return t == nullptr || (t->scalar_type() == like->scalar_type() && t->sizes() == like->sizes());
}

bool norm_weight(const at::Tensor* w, const at::Tensor* x) {
  return w->dim() == 1 && w->size(0) == x->size(-1) &&
         (w->scalar_type() == x->scalar_type() || w->scalar_type() == at::kFloat);
}

bool real(PyObject* o, double* v) {
  if (!PyFloat_CheckExact(o)) return false;
  *v = PyFloat_AS_DOUBLE(o);
  return true;
}

bool whole(PyObject* o, int64_t* v) {
  if (!PyLong_CheckExact(o)) return false;
  *v = PyLong_AsLongLong(o);
  if (*v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

// rms_norm(x, weight, residual, eps, quantize)
PyObject* rms_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  double eps;
  if (n != 5 || !real(args[3], &eps)) return none();
  Call c;
  const at::Tensor* x = c.take(args[0]);
  const at::Tensor* weight = c.take(args[1]);
  const at::Tensor* residual = c.take_optional(args[2]);
  if (!c.ok || recorded({x, weight, residual}) || wide_code(x->scalar_type()) < 0 || x->dim() < 1) return none();
  const int64_t H = x->size(-1);
  if (H == 0 || !norm_weight(weight, x) || !same_shape(residual, x)) return none();
  const at::ScalarType dtype = x->scalar_type();
  at::Tensor y, scales, sum;
  int32_t code = wide_code(dtype), scales_code = MRR_F32;
  if (args[4] == Py_None) {
    y = c.empty(x->sizes(), dtype);
  } else {
    if (!PyUnicode_CheckExact(args[4])) return none();
    const auto is = [&](const char* what) { return PyUnicode_CompareWithASCIIString(args[4], what) == 0; };
    const bool fp4 = is("mxfp4"), mx = fp4 || is("mxfp8"), i8 = is("int8");
    if ((!mx && !i8 && !is("fp8")) || (fp4 && H % 2 != 0)) return none();
    c10::SmallVector<int64_t, 6> shape(x->sizes().begin(), x->sizes().end());
    shape.back() = fp4 ? H / 2 : H;
    y = c.empty(shape, i8 ? at::kChar : fp4 ? at::kFloat4_e2m1fn_x2 : at::kFloat8_e4m3fn);
    code = i8 ? MRR_I8 : fp4 ? MRR_F4_E2M1 : MRR_F8_E4M3FN;
    if (mx) {
      shape.back() = (H + 63) / 64;
      shape.push_back(2);
      scales_code = MRR_F8_E8M0;
    } else {
      shape.pop_back();
    }
    scales = c.empty(shape, mx ? at::kFloat8_e8m0fnu : at::kFloat);
  }
  if (residual != nullptr) sum = c.empty(x->sizes(), dtype);
  const mrr_rms_norm_args a{x->data_ptr(), wide_code(dtype), x->numel() / H, H, ptr(residual), weight->data_ptr(),
                            wide_code(weight->scalar_type()), eps, y.data_ptr(), code,
                            scales.defined() ? scales.data_ptr() : nullptr, scales_code,
                            sum.defined() ? sum.data_ptr() : nullptr};
  if (unlocked([&] { return mrr_rms_norm(&a, c.stream()); }) != MRR_SUCCESS) return none();
  return result({&y, &scales, &sum});
  END_HANDLE_TH_ERRORS
}

// rms_norm_backward(grad, x, weight, grad_residual, eps)
PyObject* rms_norm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  double eps;
  if (n != 5 || !real(args[4], &eps)) return none();
  Call c;
  const at::Tensor* grad = c.take(args[0]);
  const at::Tensor* x = c.take(args[1]);
  const at::Tensor* weight = c.take(args[2]);
  const at::Tensor* grad_sum = c.take_optional(args[3]);
  if (!c.ok || wide_code(x->scalar_type()) < 0 || x->dim() < 1) return none();
  const int64_t H = x->size(-1);
  if (H == 0 || !norm_weight(weight, x) || !same_shape(grad, x) || !same_shape(grad_sum, x)) return none();
  const int64_t rows = x->numel() / H;
  const size_t bytes = mrr_rms_norm_backward_workspace_size(rows, H);
  if (bytes == 0) return none();
  at::Tensor grad_x = c.empty(x->sizes(), x->scalar_type()), grad_weight = c.empty({H}, weight->scalar_type());
  at::Tensor ws = c.empty({static_cast<int64_t>(bytes)}, at::kByte);
  const mrr_rms_norm_backward_args a{grad->data_ptr(), x->data_ptr(), wide_code(x->scalar_type()), rows, H,
                                     weight->data_ptr(), wide_code(weight->scalar_type()), eps, ptr(grad_sum),
                                     grad_x.data_ptr(), grad_weight.data_ptr()};
  if (unlocked([&] { return mrr_rms_norm_backward(&a, ws.data_ptr(), bytes, c.stream()); }) != MRR_SUCCESS) return none();
  return result({&grad_x, &grad_weight});
  END_HANDLE_TH_ERRORS
}

// router(logits, top_k, renormalize)
PyObject* router(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t k;
  if (n != 3 || !whole(args[1], &k) || !PyBool_Check(args[2])) return none();
  Call c;
  const at::Tensor* logits = c.take(args[0]);
  if (!c.ok || recorded({logits}) || wide_code(logits->scalar_type()) < 0 || logits->dim() != 2) return none();
  const int64_t T = logits->size(0), E = logits->size(1);
  if (k < 1 || k > E || k > 16) return none();
  at::Tensor weight = c.empty({T, k}, at::kFloat), ids = c.empty({T, k}, at::kInt);
  const mrr_router_args a{logits->data_ptr(), wide_code(logits->scalar_type()), T, E, k, args[2] == Py_True,
                          static_cast<float*>(weight.data_ptr()), static_cast<int32_t*>(ids.data_ptr())};
  if (unlocked([&] { return mrr_router(&a, c.stream()); }) != MRR_SUCCESS) return none();
  return result({&weight, &ids});
  END_HANDLE_TH_ERRORS
}

bool choices(const at::Tensor* t, at::ScalarType dtype, int64_t T, int64_t k) {
  return t == nullptr || (t->scalar_type() == dtype && t->dim() == 2 && t->size(0) == T && t->size(1) == k);
}

// router_backward(grad_weight, logits, expert_weight, expert_ids, renormalize)
PyObject* router_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 5 || !PyBool_Check(args[4])) return none();
  Call c;
  const at::Tensor* grad = c.take(args[0]);
  const at::Tensor* logits = c.take(args[1]);
  const at::Tensor* weight = c.take(args[2]);
  const at::Tensor* ids = c.take(args[3]);
  if (!c.ok || wide_code(logits->scalar_type()) < 0 || logits->dim() != 2 || ids->dim() != 2) return none();
  const int64_t T = logits->size(0), E = logits->size(1), k = ids->size(1);
  if (!choices(ids, at::kInt, T, k) || !choices(weight, at::kFloat, T, k) || !choices(grad, at::kFloat, T, k))
    return none();
  at::Tensor out = c.empty({T, E}, logits->scalar_type());
  const mrr_router_backward_args a{static_cast<const float*>(grad->data_ptr()), logits->data_ptr(),
                                   wide_code(logits->scalar_type()), T, E, k, args[4] == Py_True,
                                   static_cast<const float*>(weight->data_ptr()),
                                   static_cast<const int32_t*>(ids->data_ptr()), out.data_ptr()};
  if (unlocked([&] { return mrr_router_backward(&a, c.stream()); }) != MRR_SUCCESS) return none();
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

int moved_code(at::ScalarType t) {
  switch (t) {
    case at::kChar: return MRR_I8;
    case at::kFloat8_e5m2: return MRR_F8_E5M2;
    case at::kFloat8_e4m3fn: return MRR_F8_E4M3FN;
    case at::kFloat4_e2m1fn_x2: return MRR_F4_E2M1;
    default: return wide_code(t);
  }
}

// permute(tokens, expert_ids, num_experts, per_token_scales, expert_weight, expert_token_num_type)
PyObject* permute(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t E, type;
  if (n != 6 || !whole(args[2], &E) || !whole(args[5], &type)) return none();
  Call c;
  const at::Tensor* tokens = c.take(args[0]);
  const at::Tensor* ids = c.take(args[1]);
  const at::Tensor* scales = c.take_optional(args[3]);
  const at::Tensor* weight = c.take_optional(args[4]);
  if (!c.ok || recorded({tokens, scales, weight}) || tokens->dim() != 2 || ids->dim() != 2) return none();
  const int code = moved_code(tokens->scalar_type());
  const int64_t T = tokens->size(0), k = ids->size(1), H = tokens->size(1) * (code == MRR_F4_E2M1 ? 2 : 1);
  if (code < 0 || H == 0 || E < 1 || !choices(ids, at::kInt, T, k) || !choices(weight, at::kFloat, T, k)) return none();
  const size_t bytes = mrr_token_permute_workspace_size(T, k, E);
  if (bytes == 0) return none();
  mrr_token_permute_args a{};
  at::Tensor out_scales, out_weight;
  if (scales != nullptr) {
    const at::ScalarType t = scales->scalar_type();
    const int64_t dims = scales->dim();
    if (dims < 1 || dims > 3 || scales->size(0) != T || (t != at::kFloat && t != at::kFloat8_e8m0fnu && t != at::kByte) ||
        (t == at::kFloat ? dims == 3 || (dims == 2 && scales->size(1) < 1)
                         : dims != 3 || scales->size(1) != (H + 63) / 64 || scales->size(2) != 2))
      return none();
    a.scales_dtype = t == at::kFloat ? MRR_F32 : MRR_F8_E8M0;
    a.scales_ndim = static_cast<int32_t>(dims);
    c10::SmallVector<int64_t, 3> shape(scales->sizes().begin(), scales->sizes().end());
    for (int64_t i = 0; i < dims; ++i) a.scales_dims[i] = shape[i];
    shape[0] = T * k;
    out_scales = c.empty(shape, t);
    a.per_token_scales = scales->data_ptr();
    a.permute_per_token_scales = out_scales.data_ptr();
  }
  if (weight != nullptr) {
    out_weight = c.empty({T * k, 1}, at::kFloat);
    a.expert_weight = static_cast<const float*>(weight->data_ptr());
    a.permute_topk_weight = static_cast<float*>(out_weight.data_ptr());
  }
  at::Tensor rows = c.empty({T * k, tokens->size(1)}, tokens->scalar_type()), idx = c.empty({T, k}, at::kInt);
  at::Tensor num = c.empty({E}, at::kInt), ws;
  if (T * k > MRR_TOKEN_PERMUTE_ALONE) ws = c.empty({static_cast<int64_t>(bytes)}, at::kByte);
  a.tokens = tokens->data_ptr();
  a.tokens_dtype = code;
  a.T = T;
  a.H = H;
  a.expert_ids = static_cast<const int32_t*>(ids->data_ptr());
  a.top_k = k;
  a.E = E;
  a.permute_tokens = rows.data_ptr();
  a.permute_token_idx = static_cast<int32_t*>(idx.data_ptr());
  a.expert_token_num = static_cast<int32_t*>(num.data_ptr());
  a.expert_token_num_type = type;
  if (unlocked([&] { return mrr_token_permute(&a, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? bytes : 0, c.stream()); }) != MRR_SUCCESS) return none();
  return result({&rows, &out_scales, &idx, &num, &out_weight});
  END_HANDLE_TH_ERRORS
}

bool sum_sizes(const at::Tensor* rows, const at::Tensor* idx, const at::Tensor* weight) {
  return wide_code(rows->scalar_type()) >= 0 && rows->dim() == 2 && rows->size(1) > 0 && idx->dim() == 2 &&
         idx->scalar_type() == at::kInt && idx->size(1) >= 1 && idx->size(1) <= 16 &&
         choices(weight, at::kFloat, idx->size(0), idx->size(1));
}

// unpermute(rows, permute_token_idx, expert_weight)
PyObject* unpermute(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 3) return none();
  Call c;
  const at::Tensor* rows = c.take(args[0]);
  const at::Tensor* idx = c.take(args[1]);
  const at::Tensor* weight = c.take_optional(args[2]);
  if (!c.ok || recorded({rows, weight}) || !sum_sizes(rows, idx, weight)) return none();
  at::Tensor y = c.empty({idx->size(0), rows->size(1)}, rows->scalar_type());
  const mrr_token_unpermute_args a{rows->data_ptr(), wide_code(rows->scalar_type()), rows->size(0), rows->size(1),
                                   static_cast<const int32_t*>(idx->data_ptr()), idx->size(0), idx->size(1),
                                   static_cast<const float*>(ptr(weight)), y.data_ptr(), nullptr, nullptr};
  if (unlocked([&] { return mrr_token_unpermute(&a, c.stream()); }) != MRR_SUCCESS) return none();
  return THPVariable_Wrap(std::move(y));
  END_HANDLE_TH_ERRORS
}

// permute_backward(grad_rows, permute_token_idx, grad_topk_weight)
PyObject* permute_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 3) return none();
  Call c;
  const at::Tensor* rows = c.take(args[0]);
  const at::Tensor* idx = c.take(args[1]);
  const at::Tensor* weight = c.take_optional(args[2]);
  if (!c.ok || !sum_sizes(rows, idx, nullptr)) return none();
  if (weight != nullptr && (weight->scalar_type() != at::kFloat || weight->dim() < 1 || weight->dim() > 2 ||
                            weight->size(0) != rows->size(0) || weight->numel() != rows->size(0)))
    return none();
  at::Tensor grad = c.empty({idx->size(0), rows->size(1)}, rows->scalar_type()), grad_weight;
  if (weight != nullptr) grad_weight = c.empty(idx->sizes(), at::kFloat);
  const mrr_token_unpermute_args a{rows->data_ptr(), wide_code(rows->scalar_type()), rows->size(0), rows->size(1),
                                   static_cast<const int32_t*>(idx->data_ptr()), idx->size(0), idx->size(1), nullptr,
                                   grad.data_ptr(), static_cast<const float*>(ptr(weight)),
                                   weight == nullptr ? nullptr : static_cast<float*>(grad_weight.data_ptr())};
  if (unlocked([&] { return mrr_token_unpermute(&a, c.stream()); }) != MRR_SUCCESS) return none();
  return result({&grad, &grad_weight});
  END_HANDLE_TH_ERRORS
}

// unpermute_backward(grad, rows, permute_token_idx, expert_weight)
PyObject* unpermute_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) return none();
  Call c;
  const at::Tensor* grad = c.take(args[0]);
  const at::Tensor* rows = c.take(args[1]);
  const at::Tensor* idx = c.take(args[2]);
  const at::Tensor* weight = c.take_optional(args[3]);
  if (!c.ok || !sum_sizes(rows, idx, weight) || grad->scalar_type() != rows->scalar_type() || grad->dim() != 2 ||
      grad->size(0) != idx->size(0) || grad->size(1) != rows->size(1))
    return none();
  at::Tensor grad_rows = c.empty(rows->sizes(), rows->scalar_type()), grad_weight;
  if (weight != nullptr) grad_weight = c.empty(idx->sizes(), at::kFloat);
  const mrr_token_unpermute_backward_args a{
      grad->data_ptr(), rows->data_ptr(), wide_code(rows->scalar_type()), rows->size(0), rows->size(1),
      static_cast<const int32_t*>(idx->data_ptr()), idx->size(0), idx->size(1), static_cast<const float*>(ptr(weight)),
      grad_rows.data_ptr(), weight == nullptr ? nullptr : static_cast<float*>(grad_weight.data_ptr())};
  if (unlocked([&] { return mrr_token_unpermute_backward(&a, c.stream()); }) != MRR_SUCCESS) return none();
  return result({&grad_rows, &grad_weight});
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
                         {"rms_norm", fast(rms_norm), METH_FASTCALL, nullptr},
                         {"rms_norm_backward", fast(rms_norm_backward), METH_FASTCALL, nullptr},
                         {"router", fast(router), METH_FASTCALL, nullptr},
                         {"router_backward", fast(router_backward), METH_FASTCALL, nullptr},
                         {"permute", fast(permute), METH_FASTCALL, nullptr},
                         {"unpermute", fast(unpermute), METH_FASTCALL, nullptr},
                         {"permute_backward", fast(permute_backward), METH_FASTCALL, nullptr},
                         {"unpermute_backward", fast(unpermute_backward), METH_FASTCALL, nullptr},
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
