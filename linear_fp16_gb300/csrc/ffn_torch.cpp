// The tensor-level calls of the feed-forward operators: argument checks on
// torch tensors, allocation of the results, and the call of the C entry point
// (include/poot_ffn.h) on a stream.  No computation.
//
// A decode step or a small model's gradients take ten microseconds on the
// GPU; the same checks and allocations in Python took 15 - 25 (GB300 host,
// 1024 x 1024 x 768 gradients: 28 us a call against 17.6).  ffn.py holds the
// documented functions, which pass their arguments through.
//
// A function returns its result, or the status code (an int) that is not
// POOT_OK, or raises TypeError / ValueError for arguments it cannot take.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cuda_runtime_api.h>

#include <cstdint>
#include <cstring>
#include <vector>

#include "poot_ffn.h"

namespace {

// A Python error is set; unwinds to the entry point.
struct Refused {};

[[noreturn]] void refuse(PyObject* type, const char* format, const char* name) {
  PyErr_Format(type, format, name);
  throw Refused{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

// What all tensors of a call share.
struct Common {
  at::ScalarType dtype;
  int code;
  int64_t device;
};

const at::Tensor& check(PyObject* o, const char* name, const Common& c, std::initializer_list<int64_t> shape) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != c.dtype)
    refuse(PyExc_TypeError, "%s must be float16 or bfloat16, one dtype for all tensors", name);
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
  if (t.get_device() != c.device) refuse(PyExc_ValueError, "%s must be on the same device as the other tensors", name);
  if (t.sizes() != at::IntArrayRef(shape)) refuse(PyExc_ValueError, "%s does not have the shape the other tensors give it", name);
  return t;
}

void* dense(PyObject* o, const char* name, const Common& c, std::initializer_list<int64_t> shape) {
  const at::Tensor& t = check(o, name, c, shape);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  return t.data_ptr();
}

// Row pitch of a matrix whose rows may be further apart than its columns.
int64_t pitch(const at::Tensor& t, const char* name) {
  const int64_t rows = t.size(0), cols = t.size(1);
  if (t.is_contiguous()) return cols;
  if ((cols > 1 && t.stride(1) != 1) || (rows > 1 && t.stride(0) < cols))
    refuse(PyExc_ValueError, "%s must have unit column stride and rows that do not overlap", name);
  return rows > 1 ? t.stride(0) : cols;
}

void* rows(PyObject* o, const char* name, const Common& c, int64_t m, int64_t n, int64_t* ld) {
  const at::Tensor& t = check(o, name, c, {m, n});
  *ld = pitch(t, name);
  return t.data_ptr();
}

// x [M, K]: gives the call its dtype, device and two of its sizes.
const at::Tensor& first(PyObject* o, Common* c, int64_t* M, int64_t* K, int64_t* ld) {
  const at::Tensor& t = tensor(o, "x");
  c->dtype = t.scalar_type();
  if (c->dtype == at::kHalf) c->code = POOT_DTYPE_F16;
  else if (c->dtype == at::kBFloat16) c->code = POOT_DTYPE_BF16;
  else refuse(PyExc_TypeError, "%s must be float16 or bfloat16", "x");
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", "x");
  if (t.dim() != 2) refuse(PyExc_ValueError, "%s must have 2 dims", "x");
  c->device = t.get_device();
  *M = t.size(0);
  *K = t.size(1);
  *ld = pitch(t, "x");
  return t;
}

int64_t rows_of(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 2) refuse(PyExc_ValueError, "%s must have 2 dims", name);
  return t.size(0);
}

// Without the interpreter's lock while it lives.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

// The stream of a call and the tensors it allocates: from that stream's
// memory, and kept from reuse while the caller's current stream may still
// read them.  The caller's tensors are kept from reuse while that stream may
// still use them, whatever becomes of them meanwhile.
class Run {
 public:
  // stream: None (the current one) or (stream_id, device_index, device_type)
  Run(int64_t device, PyObject* stream)
      : device_(static_cast<c10::DeviceIndex>(device)), current_(c10::cuda::getCurrentCUDAStream(device_)), stream_(current_) {
    if (stream == Py_None) return;
    long long id = 0;
    int index = 0, type = 0;
    if (!PyArg_ParseTuple(stream, "Lii", &id, &index, &type)) throw Refused{};
    if (index != device) refuse(PyExc_ValueError, "%s must be one of the tensors' device", "stream");
    stream_ = c10::cuda::CUDAStream::unpack3(id, static_cast<c10::DeviceIndex>(index), static_cast<c10::DeviceType>(type));
  }
  at::Tensor empty(std::initializer_list<int64_t> shape, at::ScalarType dtype) {
    const auto options = at::TensorOptions().dtype(dtype).device(at::kCUDA, device_);
    if (stream_ == current_) return at::empty(at::IntArrayRef(shape), options);
    c10::cuda::CUDAStreamGuard guard(stream_);
    at::Tensor t = at::empty(at::IntArrayRef(shape), options);
    c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), current_);
    return t;
  }
  void uses(PyObject* o) const {  // a tensor of the caller's, or None
    if (o != Py_None && !(stream_ == current_))
      c10::cuda::CUDACachingAllocator::recordStream(THPVariable_Unpack(o).storage().data_ptr(), stream_);
  }
  void uses(PyObject* const* a, int n) const {
    for (int i = 0; i < n; ++i) uses(a[i]);
  }
  // Runs f(stream) with the device current and without the interpreter's lock.
  // The library takes its workspace from the device, where torch's cache may
  // hold all of it: a call that found none queued nothing, and is made again
  // when torch has given back what it does not use (not under capture, where the
  // workspace is the graph's and the cache may not be touched).
  template <typename F>
  int call(F&& f) {
    const c10::cuda::CUDAGuard guard(device_);
    const auto s = reinterpret_cast<poot_stream_t>(stream_.stream());
    const Unlocked unlocked;
    const int rc = f(s);
    if (rc != POOT_ERR_CUDA || std::strcmp(poot_linear_last_cuda_error(), "cudaErrorMemoryAllocation") != 0) return rc;
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(stream_.stream(), &capture) != cudaSuccess || capture != cudaStreamCaptureStatusNone)
      return rc;
    c10::cuda::CUDACachingAllocator::emptyCache();
    return f(s);
  }

 private:
  c10::DeviceIndex device_;
  c10::cuda::CUDAStream current_, stream_;
};

// The call has written to a tensor of the caller's: a graph that saved its former
// values finds out (inference tensors carry no version).
void written(PyObject* o) {
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

PyObject* wrap_all(std::initializer_list<const at::Tensor*> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (r == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor* t : ts) {
    PyObject* o = wrap(*t);
    if (o == nullptr) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{};
  return v != 0;
}

void count_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(PyExc_TypeError, "%s", "wrong number of arguments");
}

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

// C++ exceptions end here: torch's become its Python errors.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<gated_linear>("gated_linear"),
                           method<gated_linear_backward>("gated_linear_backward"),
                           method<linear_backward>("linear_backward"),
                           method<clip_grad_norm>("clip_grad_norm"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ffn_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ffn_torch() { return PyModule_Create(&g_module); }
