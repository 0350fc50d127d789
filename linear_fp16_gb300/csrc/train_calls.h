// The tensor-level calls of the training operators (see ffn_torch.cpp, which
// lists them): the vocabulary head's loss and its gradients.
#pragma once

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

}  // namespace
