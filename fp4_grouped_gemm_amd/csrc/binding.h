// What the compiled parts of the Python binding share: checks of tensors and
// calls of the C ABI (include/fgg.h).  Everything that they or the library
// refuse raises ValueError.
#pragma once

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>

#include <cstdint>
#include <string>

#include "fgg.h"

namespace fgg_binding {

using at::Tensor;

inline const char* type_name(at::ScalarType t) {
  return t == at::kBFloat16 ? "torch.bfloat16" : t == at::kInt ? "torch.int32" : t == at::kFloat ? "torch.float32"
                                                                                                : c10::toString(t);
}

inline const Tensor& tensor(PyObject* o, const char* name, at::ScalarType dtype, int64_t dim) {
  const bool is = THPVariable_Check(o) && THPVariable_Unpack(o).scalar_type() == dtype &&
                  THPVariable_Unpack(o).dim() == dim;
  TORCH_CHECK_VALUE(is, name, " must be a ", dim, "-D ", type_name(dtype), " tensor");
  const Tensor& t = THPVariable_Unpack(o);
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a GPU tensor");
  return t;
}

inline void on(const Tensor& t, const char* name, const Tensor& q) {
  TORCH_CHECK_VALUE(t.get_device() == q.get_device(), name, " is on ", t.device(), ", expected ", q.device());
}

// Stride of a dimension; one that holds a single entry may have any.
inline long long step(const Tensor& t, int dim) { return t.size(dim) > 1 ? t.stride(dim) : 0; }

// A contiguous vector of n values on q's device; any length if n is negative.
template <class T>
const T* vector(PyObject* o, const char* name, int64_t n, at::ScalarType dtype, const Tensor& q) {
  const Tensor& t = tensor(o, name, dtype, 1);
  on(t, name, q);
  TORCH_CHECK_VALUE(t.is_contiguous() && (n < 0 || t.size(0) == n), name, " must be a contiguous ",
                    type_name(dtype), " tensor", n < 0 ? "" : " of shape (", n < 0 ? "" : std::to_string(n),
                    n < 0 ? "" : ",)");
  return static_cast<const T*>(t.const_data_ptr());
}

// Runs a call of the library without the interpreter's lock (a launch can wait for
// room in the stream's queue).
template <class F>
void call(F f) {
  PyThreadState* const state = PyEval_SaveThread();
  const fgg_status st = f();
  PyEval_RestoreThread(state);
  if (st == FGG_OK) return;
  const char* msg = fgg_last_error();
  TORCH_CHECK_VALUE(false, msg && *msg ? msg : "fgg call failed");
}

inline int as_int(int64_t n, const char* name) {
  TORCH_CHECK_VALUE(n <= INT32_MAX, name, " passes 2^31");
  return (int)n;
}

inline bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw python_error();
  return x;
}

inline void* stream_on(const Tensor& q) { return c10::hip::getCurrentHIPStream(q.get_device()).stream(); }

inline void arity(Py_ssize_t n, Py_ssize_t want) {
  TORCH_CHECK_VALUE(n == want, "expected ", want, " arguments, got ", n);
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}

// mxfp4_binding.cpp
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n);
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n);
PyObject* product(PyObject*, PyObject* const* a, Py_ssize_t n);
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n);

}  // namespace fgg_binding
