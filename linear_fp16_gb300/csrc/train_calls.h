// The tensor-level calls of the training operators (see ffn_torch.cpp, which
// lists them): the vocabulary head's loss and its gradients, the AdamW step.
#pragma once

#include <vector>

#include "poot_train.h"
#include "tensor_call.h"

namespace {

using namespace poot_torch;

// A one-dimensional tensor of M elements of `dtype`, unit stride unless `strided`
// (then *stride is what it has: 0 in an expanded one).
void* vector(PyObject* o, const char* name, const char* what, at::ScalarType dtype, int64_t M, int64_t device,
             int64_t* stride = nullptr) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != dtype) refuse(PyExc_TypeError, what, name);
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
  if (t.get_device() != device) refuse(PyExc_ValueError, "%s must be on the same device as the other tensors", name);
  if (t.dim() != 1 || t.size(0) != M) refuse(PyExc_ValueError, "%s must have one element for each row of x", name);
  if (stride != nullptr) *stride = M > 1 ? t.stride(0) : 0;
  else if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  return t.data_ptr();
}
constexpr const char* kInt64 = "%s must be int64";
constexpr const char* kFloat32 = "%s must be float32";

int64_t whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}

// (x, w, target, bias, ignore_index, save, stream)
PyObject* linear_cross_entropy(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 7);
  Common c;
  poot_linear_cross_entropy_args p{};
  const at::Tensor& x = first(a[0], &c, &p.M, &p.K, &p.ldx);
  p.V = rows_of(a[1], "w");
  p.x = x.data_ptr();
  p.w = dense(a[1], "w", c, {p.V, p.K});
  p.target = static_cast<const int64_t*>(vector(a[2], "target", kInt64, at::kLong, p.M, c.device));
  if (a[3] != Py_None) p.b = dense(a[3], "bias", c, {p.V});
  p.ignore_index = whole(a[4]);
  p.dtype = c.code;
  const bool save = truth(a[5]);
  Run run(c.device, a[6]);
  const at::Tensor loss = run.empty({p.M}, at::kFloat);
  at::Tensor lse;
  if (save) lse = run.empty({p.M}, at::kFloat);
  p.loss = static_cast<float*>(loss.data_ptr());
  p.lse = static_cast<float*>(ptr(lse));
  run.uses(a, 4);
  const int rc = run.call([&](poot_stream_t s) { return poot_linear_cross_entropy(&p, s); });
  if (rc != POOT_OK) return PyLong_FromLong(rc);
  return save ? wrap_all({&loss, &lse}) : wrap(loss);
}

// (dloss, x, w, target, lse, bias, ignore_index, need_dx, need_dw, need_db, stream)
PyObject* linear_cross_entropy_backward(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 11);
  Common c;
  poot_linear_cross_entropy_backward_args p{};
  const at::Tensor& x = first(a[1], &c, &p.M, &p.K, &p.ldx);
  p.V = rows_of(a[2], "w");
  p.x = x.data_ptr();
  p.w = dense(a[2], "w", c, {p.V, p.K});
  p.dloss = static_cast<const float*>(vector(a[0], "dloss", kFloat32, at::kFloat, p.M, c.device, &p.dloss_stride));
  p.target = static_cast<const int64_t*>(vector(a[3], "target", kInt64, at::kLong, p.M, c.device));
  p.lse = static_cast<const float*>(vector(a[4], "lse", kFloat32, at::kFloat, p.M, c.device));
  if (a[5] != Py_None) p.b = dense(a[5], "bias", c, {p.V});
  p.ignore_index = whole(a[6]);
  p.dtype = c.code;
  Run run(c.device, a[10]);
  at::Tensor dx, dw, db;
  if (truth(a[7])) dx = run.empty({p.M, p.K}, c.dtype);
  if (truth(a[8])) dw = run.empty({p.V, p.K}, c.dtype);
  if (truth(a[9])) db = run.empty({p.V}, c.dtype);
  p.dx = ptr(dx);
  p.dw = ptr(dw);
  p.db = ptr(db);
  run.uses(a, 6);
  const int rc = run.call([&](poot_stream_t s) { return poot_linear_cross_entropy_backward(&p, s); });
  return rc != POOT_OK ? PyLong_FromLong(rc) : wrap_all({&dx, &dw, &db});
}

// ---- the AdamW step -------------------------------------------------------------
// A list argument of `count` tensors (count < 0: any number), or nullptr for None.
PyObject* tensor_list(PyObject* o, const char* name, Py_ssize_t count, bool optional) {
  if (optional && o == Py_None) return nullptr;
  if (!PyList_Check(o)) refuse(PyExc_TypeError, "%s must be a sequence of tensors", name);
  if (count >= 0 && PyList_GET_SIZE(o) != count) refuse(PyExc_ValueError, "%s must hold as many tensors as params", name);
  return o;
}

int64_t scale_blocks(int64_t n) { return (n + POOT_ADAMW_BLOCK - 1) / POOT_ADAMW_BLOCK; }

// The tensors of one call's lists: contiguous, on one device.
class OnDevice {
 public:
  const at::Tensor& get(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda() || (device_ >= 0 && t.get_device() != device_) || !t.is_contiguous())
      refuse(PyExc_ValueError, "every tensor of %s must be a contiguous CUDA tensor, all on one device", name);
    device_ = t.get_device();
    return t;
  }
  // one of `dtype` with the elements of a parameter
  void* like(PyObject* o, const char* name, at::ScalarType dtype, const at::Tensor& p) {
    const at::Tensor& t = get(o, name);
    if (t.scalar_type() != dtype) refuse(PyExc_TypeError, "a tensor of %s does not have the dtype of its kind of state", name);
    if (t.sizes() != p.sizes()) refuse(PyExc_ValueError, "every tensor of %s must have the shape of its parameter", name);
    return t.data_ptr();
  }
  float* scales(PyObject* o, const char* name, int64_t n) {
    const at::Tensor& t = get(o, name);
    if (t.scalar_type() != at::kFloat) refuse(PyExc_TypeError, "every tensor of %s must be float32", name);
    if (t.dim() != 1 || t.size(0) != scale_blocks(n))
      refuse(PyExc_ValueError, "every tensor of %s must have one element for each 256 of its parameter", name);
    return static_cast<float*>(t.data_ptr());
  }
  int64_t device() const { return device_; }

 private:
  int64_t device_ = -1;
};

int element_type(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kHalf: return POOT_GRAD_F16;
    case at::kBFloat16: return POOT_GRAD_BF16;
    case at::kFloat: return POOT_GRAD_F32;
    default: refuse(PyExc_TypeError, "every tensor of %s must be float16, bfloat16 or float32", name);
  }
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}

// A number, or a CUDA tensor of one element read when the step runs.
template <typename T>
const T* on_device(PyObject* o, const char* name, at::ScalarType dtype, int64_t device) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != dtype)
    refuse(PyExc_TypeError, dtype == at::kLong ? "%s as a tensor must be int64" : "%s as a tensor must be float32", name);
  if (!t.is_cuda() || t.get_device() != device || t.numel() != 1)
    refuse(PyExc_ValueError, "%s as a tensor must have one element, on the parameters' device", name);
  return static_cast<const T*>(t.data_ptr());
}

// (params, grads, m, v, m_scale or None, v_scale or None, copies or None, weight_decay: number or list,
//  step, lr, grad_scale, beta1, beta2, eps, stream)
PyObject* adamw_step(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 15);
  PyObject* const params = tensor_list(a[0], "params", -1, false);
  const Py_ssize_t count = PyList_GET_SIZE(params);
  if (count == 0) refuse(PyExc_ValueError, "%s must hold at least one tensor", "params");
  PyObject* const grads = tensor_list(a[1], "grads", count, false);
  PyObject* const ms = tensor_list(a[2], "state.m", count, false);
  PyObject* const vs = tensor_list(a[3], "state.v", count, false);
  PyObject* const sms = tensor_list(a[4], "state.m_scale", count, true);
  PyObject* const svs = tensor_list(a[5], "state.v_scale", count, true);
  PyObject* const copies = tensor_list(a[6], "copies", count, true);
  const bool small = sms != nullptr;
  if (small != (svs != nullptr)) refuse(PyExc_ValueError, "%s must be there both or neither", "state.m_scale and state.v_scale");
  PyObject* const decays = PyList_Check(a[7]) ? a[7] : nullptr;
  if (decays != nullptr && PyList_GET_SIZE(decays) != count)
    refuse(PyExc_ValueError, "%s must hold as many numbers as params tensors", "weight_decay");
  const double decay = decays == nullptr ? real(a[7]) : 0.0;
  std::vector<poot_adamw_tensor> table(static_cast<size_t>(count));
  OnDevice on;
  for (Py_ssize_t i = 0; i < count; ++i) {
    poot_adamw_tensor& e = table[static_cast<size_t>(i)];
    const at::Tensor& p = on.get(PyList_GET_ITEM(params, i), "params");
    const at::Tensor& g = on.get(PyList_GET_ITEM(grads, i), "grads");
    if (g.sizes() != p.sizes()) refuse(PyExc_ValueError, "every tensor of %s must have the shape of its parameter", "grads");
    e.param = p.data_ptr();
    e.grad = g.data_ptr();
    e.param_dtype = element_type(p, "params");
    e.grad_dtype = element_type(g, "grads");
    e.n = p.numel();
    e.m = on.like(PyList_GET_ITEM(ms, i), "state.m", small ? at::kChar : at::kFloat, p);
    e.v = on.like(PyList_GET_ITEM(vs, i), "state.v", small ? at::kByte : at::kFloat, p);
    if (small) {
      e.m_scale = on.scales(PyList_GET_ITEM(sms, i), "state.m_scale", e.n);
      e.v_scale = on.scales(PyList_GET_ITEM(svs, i), "state.v_scale", e.n);
    }
    if (copies != nullptr && PyList_GET_ITEM(copies, i) != Py_None) {
      const at::Tensor& c = on.get(PyList_GET_ITEM(copies, i), "copies");
      e.copy_dtype = element_type(c, "copies");
      if (e.copy_dtype == POOT_GRAD_F32 || e.param_dtype != POOT_GRAD_F32)
        refuse(PyExc_TypeError, "every tensor of %s must be float16 or bfloat16, beside a float32 parameter", "copies");
      if (c.sizes() != p.sizes()) refuse(PyExc_ValueError, "every tensor of %s must have the shape of its parameter", "copies");
      e.copy = c.data_ptr();
    }
    e.weight_decay = decays == nullptr ? decay : real(PyList_GET_ITEM(decays, i));
  }
  poot_adamw_args p{};
  p.tensors = table.data();
  p.count = count;
  p.bits = small ? 8 : 32;
  p.step_device = on_device<int64_t>(a[8], "step", at::kLong, on.device());
  p.lr_device = on_device<float>(a[9], "lr", at::kFloat, on.device());
  p.grad_scale_device = on_device<float>(a[10], "grad_scale", at::kFloat, on.device());
  if (p.step_device == nullptr) p.step = whole(a[8]);
  if (p.lr_device == nullptr) p.lr = real(a[9]);
  if (p.grad_scale_device == nullptr) p.grad_scale = real(a[10]);
  p.beta1 = real(a[11]);
  p.beta2 = real(a[12]);
  p.eps = real(a[13]);
  Run run(on.device(), a[14]);
  PyObject* const lists[] = {params, ms, vs, sms, svs, copies};
  for (PyObject* list : lists)
    if (list != nullptr)
      for (Py_ssize_t i = 0; i < count; ++i) run.uses(PyList_GET_ITEM(list, i));
  for (Py_ssize_t i = 0; i < count; ++i) run.uses(PyList_GET_ITEM(grads, i));
  for (int i = 8; i < 11; ++i)
    if (THPVariable_Check(a[i])) run.uses(a[i]);
  const int rc = run.call([&](poot_stream_t s) { return poot_adamw_step(&p, s); });
  if (rc != POOT_OK) return PyLong_FromLong(rc);
  for (PyObject* list : lists)
    if (list != nullptr)
      for (Py_ssize_t i = 0; i < count; ++i)
        if (PyList_GET_ITEM(list, i) != Py_None) written(PyList_GET_ITEM(list, i));
  Py_RETURN_NONE;
}

// (m, v, m_scale, v_scale, stream) -> ([m], [v]) in FP32
PyObject* adamw_values(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 5);
  PyObject* const ms = tensor_list(a[0], "state.m", -1, false);
  const Py_ssize_t count = PyList_GET_SIZE(ms);
  PyObject* const vs = tensor_list(a[1], "state.v", count, false);
  PyObject* const sms = tensor_list(a[2], "state.m_scale", count, false);
  PyObject* const svs = tensor_list(a[3], "state.v_scale", count, false);
  if (count == 0) refuse(PyExc_ValueError, "%s must hold at least one tensor", "state.m");
  std::vector<poot_adamw_codes> table(static_cast<size_t>(count));
  std::vector<at::Tensor> outs;
  outs.reserve(2 * static_cast<size_t>(count));
  OnDevice on;
  const int64_t device = on.get(PyList_GET_ITEM(ms, 0), "state.m").get_device();
  Run run(device, a[4]);
  for (Py_ssize_t i = 0; i < count; ++i) {
    poot_adamw_codes& e = table[static_cast<size_t>(i)];
    const at::Tensor& m = on.get(PyList_GET_ITEM(ms, i), "state.m");
    e.m = on.like(PyList_GET_ITEM(ms, i), "state.m", at::kChar, m);
    e.v = on.like(PyList_GET_ITEM(vs, i), "state.v", at::kByte, m);
    e.n = m.numel();
    e.m_scale = on.scales(PyList_GET_ITEM(sms, i), "state.m_scale", e.n);
    e.v_scale = on.scales(PyList_GET_ITEM(svs, i), "state.v_scale", e.n);
    for (float** out : {&e.m_out, &e.v_out}) {
      outs.push_back(run.empty(m.sizes(), at::kFloat));
      *out = static_cast<float*>(outs.back().data_ptr());
    }
  }
  for (PyObject* list : {ms, vs, sms, svs})
    for (Py_ssize_t i = 0; i < count; ++i) run.uses(PyList_GET_ITEM(list, i));
  const int rc = run.call([&](poot_stream_t s) { return poot_adamw_values(table.data(), count, s); });
  if (rc != POOT_OK) return PyLong_FromLong(rc);
  PyObject* const m = PyList_New(count);
  PyObject* const v = PyList_New(count);
  PyObject* const r = m != nullptr && v != nullptr ? PyTuple_Pack(2, m, v) : nullptr;
  Py_XDECREF(m);
  Py_XDECREF(v);
  if (r == nullptr) return nullptr;
  for (Py_ssize_t i = 0; i < count; ++i) {
    for (int k = 0; k < 2; ++k) {
      PyObject* const o = wrap(outs[2 * static_cast<size_t>(i) + k]);
      if (o == nullptr) {
        Py_DECREF(r);
        return nullptr;
      }
      PyList_SET_ITEM(k == 0 ? m : v, i, o);
    }
  }
  return r;
}

}  // namespace
