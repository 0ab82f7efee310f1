// What the argument marshalling of the operators shares: the checks of
// PyTorch tensors (TypeError and ValueError, as the binding's other functions
// raise them) and the outputs.
#pragma once
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "fp8bs.h"

namespace marshal {

using at::Tensor;

inline const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}
inline const Tensor* optional(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }
inline int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
inline int32_t narrow(PyObject* o) {
  const int64_t v = integer(o);
  TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, "an integer argument is out of range: ", v);
  return static_cast<int32_t>(v);
}
inline double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
inline hipStream_t stream(PyObject* current) {
  THPObjectPtr handle(PyObject_CallNoArgs(current));
  if (!handle) throw python_error();
  void* p = PyLong_AsVoidPtr(handle);
  if (!p && PyErr_Occurred()) throw python_error();
  return static_cast<hipStream_t>(p);
}

inline void on_gpu(const Tensor& t) { TORCH_CHECK_VALUE(t.is_cuda(), "all tensors must be on the GPU"); }
inline void need(const Tensor& t, at::IntArrayRef shape, at::ScalarType dtype, const char* name) {
  TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", t.sizes(), ", expected ", shape);
  TORCH_CHECK_TYPE(t.scalar_type() == dtype, name, " must be ", dtype, ", got ", t.scalar_type());
}
inline void dense(const Tensor& t, at::IntArrayRef shape, at::ScalarType dtype, const char* name) {
  need(t, shape, dtype, name);
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
}
// `given` checked, or a new tensor.
inline Tensor output(const Tensor* given, const Tensor& like, at::IntArrayRef shape, at::ScalarType dtype, const char* name) {
  if (!given) return at::empty(shape, like.options().dtype(dtype).requires_grad(false));
  on_gpu(*given);
  dense(*given, shape, dtype, name);
  return *given;
}
inline int32_t dtype_code(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return FP8BS_BF16;
  TORCH_CHECK_TYPE(t.scalar_type() == at::kFloat, name, " must be bfloat16 or float32, got ", t.scalar_type());
  return FP8BS_F32;
}
// Pitch of a matrix with unit column stride.
inline int64_t pitch(const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.dim() == 2, name, " must have two dimensions");
  TORCH_CHECK_VALUE(t.size(1) <= 1 || t.stride(1) == 1, name, " must have unit column stride");
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

inline PyObject* wrap(std::initializer_list<Tensor> ts) {
  THPObjectPtr tuple(PyTuple_New(static_cast<Py_ssize_t>(ts.size())));
  if (!tuple) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(tuple.get(), i++, THPVariable_Wrap(t));
  return tuple.release();
}
inline PyObject* refused(fp8bs_status st) { return PyLong_FromLong(st); }
inline void arity(Py_ssize_t got, Py_ssize_t want) { TORCH_CHECK_TYPE(got == want, want, " arguments expected, got ", got); }


using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
inline PyMethodDef method(const char* name, Fast f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

}  // namespace marshal
