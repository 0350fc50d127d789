// What the tensor-level calls share: checks of torch tensors, the stream and
// the tensors of a call, the entry points' error handling.
#pragma once

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

#include "poot_linear.h"

namespace poot_torch {

// A Python error is set; unwinds to the entry point.
struct Refused {};

[[noreturn]] inline void refuse(PyObject* type, const char* format, const char* name) {
  PyErr_Format(type, format, name);
  throw Refused{};
}

inline const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

// What all tensors of a call share.
struct Common {
  at::ScalarType dtype;
  int code;
  int64_t device;
};

inline const at::Tensor& check(PyObject* o, const char* name, const Common& c, std::initializer_list<int64_t> shape) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != c.dtype)
    refuse(PyExc_TypeError, "%s must be float16 or bfloat16, one dtype for all tensors", name);
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
  if (t.get_device() != c.device) refuse(PyExc_ValueError, "%s must be on the same device as the other tensors", name);
  if (t.sizes() != at::IntArrayRef(shape)) refuse(PyExc_ValueError, "%s does not have the shape the other tensors give it", name);
  return t;
}

inline void* dense(PyObject* o, const char* name, const Common& c, std::initializer_list<int64_t> shape) {
  const at::Tensor& t = check(o, name, c, shape);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  return t.data_ptr();
}

// Row pitch of a matrix whose rows may be further apart than its columns.
inline int64_t pitch(const at::Tensor& t, const char* name) {
  const int64_t rows = t.size(0), cols = t.size(1);
  if (t.is_contiguous()) return cols;
  if ((cols > 1 && t.stride(1) != 1) || (rows > 1 && t.stride(0) < cols))
    refuse(PyExc_ValueError, "%s must have unit column stride and rows that do not overlap", name);
  return rows > 1 ? t.stride(0) : cols;
}

inline void* rows(PyObject* o, const char* name, const Common& c, int64_t m, int64_t n, int64_t* ld) {
  const at::Tensor& t = check(o, name, c, {m, n});
  *ld = pitch(t, name);
  return t.data_ptr();
}

// x [M, K]: gives the call its dtype, device and two of its sizes.
inline const at::Tensor& first(PyObject* o, Common* c, int64_t* M, int64_t* K, int64_t* ld) {
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

inline int64_t rows_of(PyObject* o, const char* name) {
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
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype) {
    const auto options = at::TensorOptions().dtype(dtype).device(at::kCUDA, device_);
    if (stream_ == current_) return at::empty(shape, options);
    c10::cuda::CUDAStreamGuard guard(stream_);
    at::Tensor t = at::empty(shape, options);
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
inline void written(PyObject* o) {
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

inline PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

inline PyObject* wrap_all(std::initializer_list<const at::Tensor*> ts) {
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

inline void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

inline bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{};
  return v != 0;
}

inline void count_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(PyExc_TypeError, "%s", "wrong number of arguments");
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

}  // namespace poot_torch
