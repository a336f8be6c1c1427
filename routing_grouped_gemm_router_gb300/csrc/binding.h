// binding.h — what the extensions that call the training operators on torch tensors share (host code,
// internal header; each extension has its own copy): checks of tensors, output allocation from
// PyTorch's caching allocator on the current stream, C++ exceptions and statuses as Python's.
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <initializer_list>
#include <string>

#include "moe.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_moe_error = nullptr;  // _lib.MoeError

struct Refused {  // an argument that does not fit: becomes a ValueError
  std::string what;
};
struct Failed {  // a status of the C entry point: becomes a MoeError
  const char* fn;
  moe_status_t status;
};

constexpr ScalarType kAnyFloat = ScalarType::Undefined;  // bf16 or fp32
constexpr ScalarType kF32 = ScalarType::Float, kI32 = ScalarType::Int;

std::string name_of(ScalarType t) {
  switch (t) {
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Long: return "torch.int64";
    case ScalarType::Half: return "torch.float16";
    case ScalarType::Double: return "torch.float64";
    case ScalarType::Bool: return "torch.bool";
    default: return std::string("torch.") + c10::toString(t);
  }
}
template <typename R>
std::string list_of(const R& v) {
  std::string s = "(";
  for (int64_t d : v) s += (s.size() > 1 ? ", " : "") + (d < 0 ? std::string("any") : std::to_string(d));
  return s + ")";
}
bool is_float(ScalarType t) { return t == ScalarType::BFloat16 || t == ScalarType::Float; }

// The calling thread's device, where the library launches: another device's tensors are not this call's.
int current_device() {
  c10::DeviceIndex d = -1;
  return c10::cuda::GetDevice(&d) == cudaSuccess ? d : -1;
}

// A contiguous CUDA tensor of these extents (-1: any), type and device (-1: the current one, for an
// operator's first tensor). The fast way through is a handful of comparisons; only a tensor that does
// not fit is described.
const Tensor& check(const char* name, PyObject* o, std::initializer_list<int64_t> shape,
                    ScalarType type, int dev) {
  if (!THPVariable_Check(o))
    throw Refused{std::string(name) + ": a tensor is needed, got " + Py_TYPE(o)->tp_name};
  const Tensor& t = THPVariable_Unpack(o);
  const ScalarType st = t.scalar_type();
  if (type == kAnyFloat ? !is_float(st) : st != type)
    throw Refused{std::string(name) + ": dtype " + name_of(st) + ", expected " +
                  (type == kAnyFloat ? "bfloat16 or float32" : name_of(type))};
  bool fits = t.dim() == (int64_t)shape.size();
  if (fits) {
    int64_t i = 0;
    for (int64_t d : shape) {
      fits &= d < 0 || d == t.size(i);
      ++i;
    }
  }
  if (!fits)
    throw Refused{std::string(name) + ": shape " + list_of(t.sizes()) + ", expected " + list_of(shape)};
  if (!t.is_contiguous())
    throw Refused{std::string(name) + ": has to be contiguous (strides " + list_of(t.strides()) + ")"};
  if (!t.is_cuda()) throw Refused{std::string(name) + ": has to be on a CUDA device"};
  if (dev >= 0 && t.get_device() != dev)
    throw Refused{std::string(name) + ": is on another device than the other tensors"};
  if (dev < 0 && t.get_device() != current_device())
    throw Refused{std::string(name) + ": is on cuda:" + std::to_string(t.get_device()) +
                  ", which is not the current device"};
  return t;
}

Tensor empty(at::IntArrayRef shape, ScalarType type, const Tensor& like) {
  return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}
Tensor empty_as(const Tensor& like) { return empty(like.sizes(), like.scalar_type(), like); }

// Small outputs of one call in one allocation, each from a 64-byte boundary on: a tensor more of it costs
// 0.3 us, one with memory of its own 1.2.
struct Output {
  std::initializer_list<int64_t> shape;
  ScalarType type;
};
template <size_t N>
std::array<Tensor, N> empties(const Output (&outs)[N], const Tensor& like) {
  int64_t at[N], bytes = 0;
  for (size_t i = 0; i < N; ++i) {
    int64_t n = (int64_t)c10::elementSize(outs[i].type);
    for (int64_t d : outs[i].shape) n *= d;
    at[i] = bytes;
    bytes += (n + 63) / 64 * 64;
  }
  const Tensor all = empty({bytes}, ScalarType::Byte, like);
  std::array<Tensor, N> r;
  for (size_t i = 0; i < N; ++i) {
    r[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()),
                                                    c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                    c10::scalarTypeToTypeMeta(outs[i].type));
    r[i].unsafeGetTensorImpl()->set_sizes_contiguous(at::IntArrayRef(outs[i].shape.begin(), outs[i].shape.size()));
    r[i].unsafeGetTensorImpl()->set_storage_offset(at[i] / (int64_t)c10::elementSize(outs[i].type));
  }
  return r;
}

cudaStream_t stream_of(const Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
}
moe_dtype_t dtype_of(const Tensor& t) {
  return t.scalar_type() == ScalarType::BFloat16 ? MOE_BF16 : MOE_F32;
}
int narrow(const char* name, int64_t v) {  // extents beyond 32 bits are no sizes of these operators
  if (v > INT32_MAX || v < 0) throw Refused{std::string(name) + ": an extent of " + std::to_string(v)};
  return (int)v;
}
void done(const char* fn, moe_status_t st) {
  if (st != MOE_OK) throw Failed{fn, st};
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
float number(PyObject* o) { return (float)real(o); }
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}
bool given(PyObject* o) { return o != Py_None; }
void* ptr(const Tensor& t) { return t.data_ptr(); }
float* fptr(const Tensor& t) { return (float*)t.data_ptr(); }
int32_t* iptr(const Tensor& t) { return (int32_t*)t.data_ptr(); }

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
// A new tuple of tensors; undefined ones become None.
PyObject* tuple(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = t.defined() ? wrap(t) : Py_NewRef(Py_None);
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Runs an operator's body; C++ exceptions become Python's.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F body) {
  HANDLE_TH_ERRORS
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
  } catch (const Failed& f) {
    PyObject* e = g_moe_error ? PyObject_CallFunction(g_moe_error, "si", f.fn, (int)f.status) : nullptr;
    if (e) {
      PyErr_SetObject(g_moe_error, e);
      Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
      PyErr_Format(PyExc_RuntimeError, "%s failed: %d", f.fn, (int)f.status);
    }
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

void* maybe(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
float* fmaybe(const Tensor& t) { return (float*)maybe(t); }

// The type of a gradient that goes into `out`, or is a new tensor of `out_dtype` (default: like's).
ScalarType out_type(PyObject* out, PyObject* out_dtype, bool accumulate, const Tensor& like) {
  ScalarType type = given(out) ? kAnyFloat : like.scalar_type();
  if (given(out_dtype)) {
    if (!THPDtype_Check(out_dtype)) throw Refused{"out_dtype: a torch.dtype is needed"};
    type = reinterpret_cast<THPDtype*>(out_dtype)->scalar_type;
    if (!is_float(type)) throw Refused{"out_dtype: " + name_of(type) + ", expected bfloat16 or float32"};
  }
  if (accumulate && !given(out)) throw Refused{"accumulate: needs the tensor to add to (out)"};
  return type;
}

PyObject* set_error(PyObject*, PyObject* e) {  // the class that statuses raise
  Py_XSETREF(g_moe_error, Py_NewRef(e));
  Py_RETURN_NONE;
}

#define OPERATOR(name) PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n)
#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}

}  // namespace
