// What the compiled Python bindings share (experts_binding.cpp,
// feedforward_binding.cpp): checks of torch tensors, allocation, argument
// conversion and the form in which functions and errors reach Python.
#pragma once

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <limits>
#include <optional>
#include <string>

#include "dgt_experts.h"

namespace {

// A refused argument: the Python exception's type and text.
struct Refused {
  PyObject* type;
  std::string text;
};
[[noreturn]] void type_error(const std::string& text) { throw Refused{PyExc_TypeError, text}; }
[[noreturn]] void value_error(const std::string& text) { throw Refused{PyExc_ValueError, text}; }

using Tensor = at::Tensor;

const Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) type_error(std::string(what) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

// The library's number of an element type; -1 for another.
int kind(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kHalf: return GEMM_TYPE_F16;
    case at::kBFloat16: return GEMM_TYPE_BF16;
    case at::kFloat: return GEMM_TYPE_F32;
    case at::kFloat8_e4m3fn: return GEMM_TYPE_E4M3;
    default: return -1;
  }
}
int float_kind(const Tensor& t, const char* what) {
  const int k = kind(t);
  if (k < 0 || k == GEMM_TYPE_E4M3) type_error(std::string(what) + " must be float16, bfloat16 or float32");
  return k;
}

void same_type(const Tensor& t, at::ScalarType dt, const char* what) {
  if (t.scalar_type() != dt) type_error(std::string(what) + " must be " + c10::toString(dt));
}

// Leading dimension of a 2-D CUDA tensor with contiguous rows.
int64_t matrix(const Tensor& t, const char* what) {
  if (t.dim() != 2 || !t.is_cuda()) value_error(std::string(what) + " must be a 2-D CUDA tensor");
  const int64_t rows = t.size(0), cols = t.size(1);
  if (cols > 1 && t.stride(1) != 1) value_error(std::string(what) + " must have unit stride along its rows");
  if (rows <= 1) return cols;
  if (t.stride(0) < cols) value_error(std::string(what) + " must not have rows that overlap");
  return t.stride(0);
}
int64_t matrix(const Tensor& t, const char* what, at::ScalarType dt, int64_t rows, int64_t cols) {
  same_type(t, dt, what);
  const int64_t ld = matrix(t, what);
  if (t.size(0) != rows || t.size(1) != cols)
    value_error(std::string(what) + " must be " + std::to_string(rows) + " x " + std::to_string(cols));
  return ld;
}

// Address of a contiguous CUDA tensor of n elements.
template <class T>
T* vector(const Tensor& t, const char* what, at::ScalarType dt, int64_t n) {
  same_type(t, dt, what);
  if (t.numel() != n || !t.is_cuda() || !t.is_contiguous())
    value_error(std::string(what) + " must be a contiguous CUDA tensor of " + std::to_string(n) + " elements");
  return static_cast<T*>(t.data_ptr());
}
template <class T>
T* vector_or_null(PyObject* o, const char* what, at::ScalarType dt, int64_t n) {
  return o == Py_None ? nullptr : vector<T>(tensor(o, what), what, dt, n);
}

// groups x rows x cols with contiguous rows: leading dimension and matrix stride.
struct Stack {
  int64_t ld, stride;
};
Stack stack(const Tensor& t, const char* what) {
  if (t.dim() != 3 || !t.is_cuda()) value_error(std::string(what) + " must be a 3-D CUDA tensor");
  const int64_t g = t.size(0), r = t.size(1), c = t.size(2);
  if (c > 1 && t.stride(2) != 1) value_error(std::string(what) + " must have unit stride along its rows");
  const int64_t ld = r > 1 ? t.stride(1) : c;
  return {ld, g > 1 ? t.stride(0) : r * ld};
}

// An empty tensor on the device of `like` (a CUDA tensor), straight from the allocator: a trip through the dispatcher
// costs half as much again.
Tensor make(at::IntArrayRef size, const Tensor& like, at::ScalarType dt) {
  return at::detail::empty_cuda(size, dt, like.device(), std::nullopt);
}
[[maybe_unused]] Tensor make_strided(at::IntArrayRef size, at::IntArrayRef stride, const Tensor& like, at::ScalarType dt) {
  return at::detail::empty_strided_cuda(size, stride, dt, like.device());
}

// A scratch buffer of n bytes, or nothing.
Tensor scratch(int64_t n, const Tensor& like) { return n > 0 ? make({n}, like, at::kByte) : Tensor(); }

void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

int64_t whole(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
// A whole number that the C call takes as an int.
int whole_int(PyObject* o, const char* what) {
  const int64_t v = whole(o);
  if (v != static_cast<int>(v)) value_error(std::string(what) + " does not fit 32 bits");
  return static_cast<int>(v);
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
template <class... T>
PyObject* tuple_of(const T&... t) {
  PyObject* out = PyTuple_New(sizeof...(T));
  if (out == nullptr) throw python_error();
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(out, i++, wrap(t)), ...);
  return out;
}

// Whether bind() has been called (each binding's own).
bool is_bound();

// The Python-callable form: N arguments, and every C++ exception as a Python one.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* method(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are taken, %zd were given", N, n);
    return nullptr;
  }
  if (!is_bound()) {
    PyErr_SetString(PyExc_RuntimeError, "bind() has not given the library's entry points");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// bind({name: address}): the n entry points of the loaded library, in the order of `names`.
PyObject* bind_entries(PyObject* addresses, const char* const* names, void** to, int n) {
  for (int pass = 0; pass < 2; ++pass)  // all are found before one is kept
    for (int i = 0; i < n; ++i) {
      PyObject* v = PyDict_Check(addresses) ? PyDict_GetItemString(addresses, names[i]) : nullptr;
      void* found = v != nullptr ? PyLong_AsVoidPtr(v) : nullptr;
      if (found == nullptr) {
        if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "no address of %s", names[i]);
        return nullptr;
      }
      if (pass == 1) to[i] = found;
    }
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef def(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&method<F, N>)), METH_FASTCALL, nullptr};
}

}  // namespace
