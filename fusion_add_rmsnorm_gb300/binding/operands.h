// What the compiled wrappers share: Python arguments by position or name, the
// checks of a tensor operand, the stream, and the exception of a failed call.
#pragma once

#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>

#include "gbfuse.h"

namespace {

PyObject* g_error = nullptr;       // GbfError

// Thrown once a Python exception is set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(type, fmt, ap);
  va_end(ap);
  throw Raised();
}

// ------------------------------------------------------------- call arguments

template <int N>
struct Args {
  PyObject* at[N];

  // Positional arguments, then those by name; the first `required` must be there.
  Args(const char* fn, const char* const (&names)[N], int required, PyObject* const* args, Py_ssize_t nargs,
       PyObject* kwnames) {
    if (nargs > N) raise(PyExc_TypeError, "%s() takes at most %d arguments (%zd given)", fn, N, nargs);
    for (int i = 0; i < N; ++i) at[i] = i < nargs ? args[i] : nullptr;
    const Py_ssize_t named = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t j = 0; j < named; ++j) {
      PyObject* key = PyTuple_GET_ITEM(kwnames, j);
      int i = 0;
      while (i < N && PyUnicode_CompareWithASCIIString(key, names[i]) != 0) ++i;
      if (i == N) raise(PyExc_TypeError, "%s() got an unexpected keyword argument '%U'", fn, key);
      if (at[i]) raise(PyExc_TypeError, "%s() got multiple values for argument '%s'", fn, names[i]);
      at[i] = args[nargs + j];
    }
    for (int i = 0; i < N; ++i)
      if (!at[i]) {
        if (i < required) raise(PyExc_TypeError, "%s() missing required argument '%s'", fn, names[i]);
        at[i] = Py_None;
      }
  }
};

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    raise(PyExc_TypeError, "%s: expected an int that fits 64 bits, got %R", name, o);
  }
  return v;
}

int narrow(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v != static_cast<int>(v)) raise(PyExc_ValueError, "%s: %lld does not fit 32 bits", name, static_cast<long long>(v));
  return static_cast<int>(v);
}

double real(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    raise(PyExc_TypeError, "%s: expected a number, got %R", name, o);
  }
  return v;
}

// ------------------------------------------------------------------- operands

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s: expected a torch.Tensor, got %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// The current CUDA device, or -1 when the call's first operand is on none: the
// other operands' extents are checked all the same, and the call ends in stream().
int device_of(const at::Tensor& first) { return first.is_cuda() ? c10::cuda::current_device() : -1; }

void check_type(const at::Tensor& t, at::ScalarType type, const char* name) {
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s: expected torch.%s, got torch.%s", name,
          type == at::kInt ? "int32" : type == at::kFloat ? "float32" : type == at::kByte ? "uint8" : "bfloat16",
          c10::toString(t.scalar_type()));
}

void check_device(const at::Tensor& t, const char* name, int device) {
  if (device < 0 || t.get_device() == device) return;
  if (!t.is_cuda()) raise(PyExc_ValueError, "%s: must be on a CUDA device", name);
  raise(PyExc_ValueError, "%s: is on cuda:%d, the current device is cuda:%d", name, static_cast<int>(t.get_device()), device);
}

// Data pointer of a dense operand of n elements; None is an absent optional one.
void* operand(PyObject* o, int64_t n, at::ScalarType type, const char* name, int device) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.numel() != n)
    raise(PyExc_ValueError, "%s: holds %lld elements, the call needs %lld", name, static_cast<long long>(t.numel()),
          static_cast<long long>(n));
  check_type(t, type, name);
  if (!t.is_contiguous()) raise(PyExc_ValueError, "%s: must be contiguous", name);
  check_device(t, name, device);
  return t.data_ptr();
}

// A [batch, width] operand whose rows may be apart (a column range of a wider one).
struct Rows {
  void* at;
  int64_t batch, width, apart;
};
Rows rows(const at::Tensor& t, int64_t batch, at::ScalarType type, const char* name, int device) {
  if (t.dim() != 2 || (batch >= 0 && t.size(0) != batch))
    raise(PyExc_ValueError, "%s: expected [batch, n] with one row per request", name);
  Rows r{nullptr, t.size(0), t.size(1), t.stride(0)};
  if (r.width > 1 && t.stride(1) != 1) raise(PyExc_ValueError, "%s: the elements of a row must be contiguous", name);
  if (r.batch <= 1) r.apart = r.width;
  else if (r.apart < r.width) raise(PyExc_ValueError, "%s: rows may not overlap", name);
  check_type(t, type, name);
  check_device(t, name, device);
  r.at = t.data_ptr();
  return r;
}

// cudaStream_t of `o`, by default of the current torch stream; the last check.
void* stream(PyObject* o, int device) {
  if (device < 0) raise(PyExc_ValueError, "the operands must be on a CUDA device");
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
  if (!raw) throw Raised();
  void* s = PyLong_AsVoidPtr(raw);
  Py_DECREF(raw);
  if (!s && PyErr_Occurred()) throw Raised();
  return s;
}

PyObject* finish(int status) {
  if (status == GBF_OK) return PyLong_FromLong(0);
  PyObject* e = PyObject_CallFunction(g_error, "is", status, gbf_last_error());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

template <typename Call>
PyObject* guarded(Call call) {
  try {
    return finish(call());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define GBF_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL | METH_KEYWORDS

}  // namespace
