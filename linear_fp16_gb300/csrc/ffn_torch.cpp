// The tensor-level calls of the feed-forward and the training operators:
// argument checks on torch tensors, allocation of the results, and the call of
// the C entry point (include/poot_ffn.h, include/poot_train.h) on a stream.  No
// computation.
//
// A decode step or a small model's gradients take ten microseconds on the
// GPU; the same checks and allocations in Python took 15 - 25 (GB300 host,
// 1024 x 1024 x 768 gradients: 28 us a call against 17.6).  ffn.py and train.py hold the
// documented functions, which pass their arguments through.
//
// A function returns its result, or the status code (an int) that is not
// POOT_OK, or raises TypeError / ValueError for arguments it cannot take.
#include "tensor_call.h"
#include "train_calls.h"

#include <vector>

#include "poot_ffn.h"

namespace {

using namespace poot_torch;

// (x, wg, wu, bg, bu, out, activation, save, stream)
PyObject* gated_linear(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 9);
  Common c;
  poot_gated_linear_args p{};
  const at::Tensor& x = first(a[0], &c, &p.M, &p.K, &p.ldx);
  p.N = rows_of(a[1], "wg");
  p.x = x.data_ptr();
  p.wg = dense(a[1], "wg", c, {p.N, p.K});
  p.wu = dense(a[2], "wu", c, {p.N, p.K});
  if (a[3] != Py_None) p.bg = dense(a[3], "bg", c, {p.N});
  if (a[4] != Py_None) p.bu = dense(a[4], "bu", c, {p.N});
  p.dtype = c.code;
  p.activation = static_cast<int>(PyLong_AsLong(a[6]));
  const bool save = truth(a[7]);
  Run run(c.device, a[8]);
  at::Tensor h, g, u;
  if (a[5] != Py_None) {
    p.h = dense(a[5], "out", c, {p.M, p.N});
  } else {
    h = run.empty({p.M, p.N}, c.dtype);
    p.h = h.data_ptr();
  }
  if (save) {
    g = run.empty({p.M, p.N}, c.dtype);
    u = run.empty({p.M, p.N}, c.dtype);
    p.g = ptr(g);
    p.u = ptr(u);
  }
  run.uses(a, 6);
  const int rc = run.call([&](poot_stream_t s) { return poot_gated_linear(&p, s); });
  if (rc != POOT_OK) return PyLong_FromLong(rc);
  if (a[5] != Py_None) written(a[5]);
  if (!save && a[5] != Py_None) {
    Py_INCREF(a[5]);
    return a[5];
  }
  if (!save) return wrap(h);
  if (a[5] != Py_None) h = THPVariable_Unpack(a[5]);
  return wrap_all({&h, &g, &u});
}

// (dh, x, wg, wu, g, u, activation, need_dx, need_dw, need_db, stream)
PyObject* gated_linear_backward(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 11);
  Common c;
  poot_gated_linear_backward_args p{};
  const at::Tensor& x = first(a[1], &c, &p.M, &p.K, &p.ldx);
  p.N = rows_of(a[2], "wg");
  p.x = x.data_ptr();
  p.wg = dense(a[2], "wg", c, {p.N, p.K});
  p.wu = dense(a[3], "wu", c, {p.N, p.K});
  p.dh = rows(a[0], "dh", c, p.M, p.N, &p.ld_dh);
  p.g = rows(a[4], "g", c, p.M, p.N, &p.ld_g);
  p.u = rows(a[5], "u", c, p.M, p.N, &p.ld_u);
  p.dtype = c.code;
  p.activation = static_cast<int>(PyLong_AsLong(a[6]));
  Run run(c.device, a[10]);
  at::Tensor dx, dwg, dwu, dbg, dbu;
  if (truth(a[7])) dx = run.empty({p.M, p.K}, c.dtype);
  if (truth(a[8])) {
    dwg = run.empty({p.N, p.K}, c.dtype);
    dwu = run.empty({p.N, p.K}, c.dtype);
  }
  if (truth(a[9])) {
    dbg = run.empty({p.N}, c.dtype);
    dbu = run.empty({p.N}, c.dtype);
  }
  p.dx = ptr(dx);
  p.dwg = ptr(dwg);
  p.dwu = ptr(dwu);
  p.dbg = ptr(dbg);
  p.dbu = ptr(dbu);
  run.uses(a, 6);
  const int rc = run.call([&](poot_stream_t s) { return poot_gated_linear_backward(&p, s); });
  return rc != POOT_OK ? PyLong_FromLong(rc) : wrap_all({&dx, &dwg, &dwu, &dbg, &dbu});
}

// (dy, x, w, need_dx, need_dw, need_db, stream)
PyObject* linear_backward(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 7);
  Common c;
  poot_linear_backward_args p{};
  const at::Tensor& x = first(a[1], &c, &p.M, &p.K, &p.ldx);
  p.N = rows_of(a[2], "w");
  p.x = x.data_ptr();
  p.w = dense(a[2], "w", c, {p.N, p.K});
  p.dy = rows(a[0], "dy", c, p.M, p.N, &p.ld_dy);
  p.dtype = c.code;
  Run run(c.device, a[6]);
  at::Tensor dx, dw, db;
  if (truth(a[3])) dx = run.empty({p.M, p.K}, c.dtype);
  if (truth(a[4])) dw = run.empty({p.N, p.K}, c.dtype);
  if (truth(a[5])) db = run.empty({p.N}, c.dtype);
  p.dx = ptr(dx);
  p.dw = ptr(dw);
  p.db = ptr(db);
  run.uses(a, 3);
  const int rc = run.call([&](poot_stream_t s) { return poot_linear_backward(&p, s); });
  return rc != POOT_OK ? PyLong_FromLong(rc) : wrap_all({&dx, &dw, &db});
}

// (grads: list, out: list or None, max_norm, stream)
PyObject* clip_grad_norm(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 4);
  if (!PyList_Check(a[0]) || (a[1] != Py_None && !PyList_Check(a[1])))
    refuse(PyExc_TypeError, "%s must be lists", "grads and out");
  const Py_ssize_t count = PyList_GET_SIZE(a[0]);
  if (count == 0) refuse(PyExc_ValueError, "%s must hold at least one tensor", "grads");
  if (a[1] != Py_None && PyList_GET_SIZE(a[1]) != count)
    refuse(PyExc_ValueError, "%s must hold as many tensors as grads", "out");
  const double max_norm = PyFloat_AsDouble(a[2]);
  if (max_norm == -1.0 && PyErr_Occurred()) throw Refused{};
  std::vector<poot_grad_tensor> table(static_cast<size_t>(count));
  int64_t device = -1;
  auto grad = [&](PyObject* o, const char* name) -> const at::Tensor& {
    const at::Tensor& t = tensor(o, name);
    const at::ScalarType s = t.scalar_type();
    if (s != at::kHalf && s != at::kBFloat16 && s != at::kFloat)
      refuse(PyExc_TypeError, "every tensor of %s must be float16, bfloat16 or float32", name);
    if (!t.is_cuda() || (device >= 0 && t.get_device() != device) || !t.is_contiguous())
      refuse(PyExc_ValueError, "every tensor of %s must be a contiguous CUDA tensor, all on one device", name);
    device = t.get_device();
    return t;
  };
  for (Py_ssize_t i = 0; i < count; ++i) {
    const at::Tensor& g = grad(PyList_GET_ITEM(a[0], i), "grads");
    poot_grad_tensor& e = table[static_cast<size_t>(i)];
    e.src = e.dst = g.data_ptr();
    e.n = g.numel();
    e.dtype = g.scalar_type() == at::kHalf ? POOT_GRAD_F16 : (g.scalar_type() == at::kBFloat16 ? POOT_GRAD_BF16 : POOT_GRAD_F32);
    if (a[1] != Py_None) {
      const at::Tensor& d = grad(PyList_GET_ITEM(a[1], i), "out");
      if (d.scalar_type() != g.scalar_type() || d.sizes() != g.sizes())
        refuse(PyExc_ValueError, "every tensor of %s must have the shape and dtype of its gradient", "out");
      e.dst = d.data_ptr();
    }
  }
  Run run(device, a[3]);
  at::Tensor norm = run.empty({}, at::kFloat);
  float* const out = static_cast<float*>(norm.data_ptr());
  for (Py_ssize_t i = 0; i < count; ++i) {
    run.uses(PyList_GET_ITEM(a[0], i));
    if (a[1] != Py_None) run.uses(PyList_GET_ITEM(a[1], i));
  }
  const int rc = run.call(
      [&](poot_stream_t s) { return poot_clip_grad_norm(table.data(), count, static_cast<float>(max_norm), out, s); });
  if (rc != POOT_OK) return PyLong_FromLong(rc);
  PyObject* const results = a[1] != Py_None ? a[1] : a[0];
  for (Py_ssize_t i = 0; i < count; ++i) written(PyList_GET_ITEM(results, i));
  return wrap(norm);
}

PyMethodDef g_methods[] = {method<gated_linear>("gated_linear"),
                           method<gated_linear_backward>("gated_linear_backward"),
                           method<linear_backward>("linear_backward"),
                           method<clip_grad_norm>("clip_grad_norm"),
                           method<linear_cross_entropy>("linear_cross_entropy"),
                           method<linear_cross_entropy_backward>("linear_cross_entropy_backward"),
                           method<adamw_step>("adamw_step"),
                           method<adamw_values>("adamw_values"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ffn_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ffn_torch() { return PyModule_Create(&g_module); }
