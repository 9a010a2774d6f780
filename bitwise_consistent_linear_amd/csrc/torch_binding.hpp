// What the Python bindings share (CPython modules over torch's tensors): checks of tensors that
// hand the ones they refuse to the Python functions that name what is wrong, outputs, workspaces,
// and the entry points' frame. Included once by each module.
#pragma once

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>

#include "gdn_cpr.h"

namespace {

const char *last_error();  // of the module's library

struct Refused {};  // a Python exception is set

// What setup() hands over: torch's functions for the current device and its raw stream, the
// functions that raise for a tensor, the error class, and tuples of dtypes for those functions.
PyObject *g_device, *g_stream, *g_refuse, *g_rows, *g_need, *g_error;
enum Types {
  kF32, kFloat, kI8, kInts, kFlags, kI32, kBytes, kBf16,
  kF8, kE4m3, kE5m2, kE8m0, kReal, kI64, kTypes
};
PyObject *g_dtypes[kTypes];

bool admits(Types types, at::ScalarType t) {
  switch (types) {
    case kF32: return t == at::kFloat;
    case kFloat: return t == at::kFloat || t == at::kBFloat16;
    case kI8: return t == at::kChar;
    case kInts: return t == at::kInt || t == at::kLong;
    case kFlags: return t == at::kBool || t == at::kByte;
    case kI32: return t == at::kInt;
    case kBytes: return t == at::kByte;
    case kF8: return t == at::kFloat8_e4m3fn || t == at::kFloat8_e5m2;
    case kE4m3: return t == at::kFloat8_e4m3fn;
    case kE5m2: return t == at::kFloat8_e5m2;
    case kE8m0: return t == at::kFloat8_e8m0fnu;
    case kReal: return t == at::kFloat || t == at::kDouble;
    case kI64: return t == at::kLong;
    default: return t == at::kBFloat16;
  }
}
Types alone(at::ScalarType t) {  // of an output
  switch (t) {
    case at::kBFloat16: return kBf16;
    case at::kChar: return kI8;
    case at::kFloat8_e4m3fn: return kE4m3;
    case at::kFloat8_e5m2: return kE5m2;
    case at::kFloat8_e8m0fnu: return kE8m0;
    case at::kInt: return kI32;
    case at::kLong: return kI64;
    default: return kF32;
  }
}
[[maybe_unused]] int32_t code(at::ScalarType t) { return t == at::kBFloat16 ? GDN_DTYPE_BF16 : GDN_DTYPE_F32; }

// `fn` is expected to raise.
[[noreturn]] void refuse(PyObject *fn, PyObject *args) {
  PyObject *r = args ? PyObject_CallObject(fn, args) : nullptr;
  Py_XDECREF(args);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an argument was refused");
  throw Refused{};
}

[[noreturn]] void value_error(const std::string &text) {
  PyErr_SetString(PyExc_ValueError, text.c_str());
  throw Refused{};
}

[[maybe_unused]] bool given(PyObject *o) { return o != Py_None; }

// A matrix on a GPU whose rows are contiguous.
struct Rows {
  const at::Tensor &t;
  int64_t stride;
};
Rows rows(PyObject *o, const char *name, Types types) {
  if (THPVariable_Check(o)) {
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.is_cuda() && admits(types, t.scalar_type()) && t.dim() == 2 &&
        (t.stride(1) == 1 || t.size(1) <= 1))
      return {t, t.size(0) > 1 ? t.stride(0) : t.size(1)};
  }
  refuse(g_rows, Py_BuildValue("(OsO)", o, name, g_dtypes[types]));
}

// A tensor of `dim` dimensions on a GPU.
const at::Tensor &need(PyObject *o, const char *name, Types types, int dim) {
  if (THPVariable_Check(o)) {
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.is_cuda() && admits(types, t.scalar_type()) && t.dim() == dim && t.is_contiguous())
      return t;
  }
  refuse(g_need, Py_BuildValue("(OsOi)", o, name, g_dtypes[types], dim));
}

// The pointer of a dense tensor of `shape` on GPU `dev`.
void *take(PyObject *o, const char *name, Types types, at::IntArrayRef shape, int dev) {
  if (THPVariable_Check(o)) {
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.is_cuda() && t.get_device() == dev && admits(types, t.scalar_type()) &&
        t.sizes() == shape && t.is_contiguous())
      return t.data_ptr();
  }
  PyObject *sizes = PyTuple_New((Py_ssize_t)shape.size());
  for (size_t i = 0; sizes && i < shape.size(); ++i)
    PyTuple_SET_ITEM(sizes, (Py_ssize_t)i, PyLong_FromLongLong(shape[i]));
  refuse(g_refuse, Py_BuildValue("(OsONi)", o, name, g_dtypes[types], sizes, dev));
}
[[maybe_unused]] void *take_if(PyObject *o, const char *name, Types types, at::IntArrayRef shape, int dev) {
  return given(o) ? take(o, name, types, shape, dev) : nullptr;
}

// The current stream of GPU `dev`, which has to be the current device: the library launches there.
void *stream_of(int dev) {
  PyObject *r = PyObject_CallNoArgs(g_device);
  const long current = r ? PyLong_AsLong(r) : -1;
  Py_XDECREF(r);
  if (PyErr_Occurred()) throw Refused{};
  if (current != dev)
    value_error("the tensors are on GPU " + std::to_string(dev) + ", the current device is " +
                std::to_string(current));
  PyObject *index = PyLong_FromLong(dev);
  r = index ? PyObject_CallOneArg(g_stream, index) : nullptr;
  Py_XDECREF(index);
  void *s = r ? PyLong_AsVoidPtr(r) : nullptr;
  Py_XDECREF(r);
  if (PyErr_Occurred()) throw Refused{};
  return s;
}

// A new dense tensor on GPU `dev`: at::empty without its way through the dispatcher (three of
// them and a launch take 5.5 us of host time against 6.1).
at::Tensor fresh(at::ScalarType type, at::IntArrayRef shape, int dev) {
  return at::Tensor(at::detail::empty_cuda(
      shape, type, c10::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt));
}

// An output: the caller's, checked, or a new one. Owns a reference until it is handed out.
class Out {
 public:
  Out() : obj_(nullptr), ptr_(nullptr) {}
  Out(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, int dev) {
    if (given(o)) {
      ptr_ = take(o, name, alone(type), shape, dev);
      Py_INCREF(o);
      obj_ = o;
    } else {
      at::Tensor t = fresh(type, shape, dev);
      ptr_ = t.data_ptr();
      obj_ = THPVariable_Wrap(std::move(t));
      if (!obj_) throw Refused{};
    }
  }
  Out(const Out &) = delete;
  Out &operator=(const Out &) = delete;
  ~Out() { Py_XDECREF(obj_); }
  template <class T = void>
  T *get() const { return static_cast<T *>(ptr_); }
  PyObject *release() {  // None where there is no output
    PyObject *o = obj_;
    obj_ = nullptr;
    if (!o) Py_INCREF(o = Py_None);
    return o;
  }

 private:
  PyObject *obj_;
  void *ptr_;
};

template <class... Outs>
PyObject *tuple(Outs &...outs) {
  PyObject *t = PyTuple_New(sizeof...(outs));
  if (!t) throw Refused{};
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(t, i++, outs.release()), ...);
  return t;
}

// A workspace: the caller's bytes, or new ones of the size that `size` reports.
struct Workspace {
  at::Tensor own;
  void *ptr;
  size_t bytes;
};
void check(gdn_status_t st) {
  if (st == GDN_OK) return;
  PyObject *e = PyObject_CallFunction(g_error, "is", (int)st, last_error());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Refused{};
}

template <class Size>
Workspace workspace(PyObject *o, int dev, Size size) {
  if (given(o)) {
    const at::Tensor &t = need(o, "workspace", kBytes, 1);
    if (t.get_device() != dev)
      value_error("workspace is on GPU " + std::to_string(t.get_device()) + ", expected GPU " +
                  std::to_string(dev));
    return {at::Tensor(), t.data_ptr(), (size_t)t.numel()};
  }
  size_t bytes = 0;
  check(size(&bytes));
  if (bytes == 0) return {at::Tensor(), nullptr, 0};
  at::Tensor t = fresh(at::kByte, {(int64_t)bytes}, dev);
  void *p = t.data_ptr();
  return {std::move(t), p, bytes};
}

[[maybe_unused]] double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}
[[maybe_unused]] bool flag(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{};
  return v != 0;
}

// One entry point of the module: the number of arguments, then the call, errors as Python's.
template <PyObject *(*Fn)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N || !g_error) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or setup() was not called");
    return nullptr;
  }
  try {
    return Fn(args);
  } catch (const Refused &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// setup(current_device, raw_stream, refuse, rows, need, error, dtypes)
PyObject *setup(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 7 || !PyTuple_Check(args[6]) || PyTuple_GET_SIZE(args[6]) != kTypes) {
    PyErr_SetString(PyExc_TypeError, "setup takes six objects and a tuple of tuples of dtypes");
    return nullptr;
  }
  PyObject **to[6] = {&g_device, &g_stream, &g_refuse, &g_rows, &g_need, &g_error};
  for (int i = 0; i < 6; ++i) {
    Py_INCREF(args[i]);
    Py_XDECREF(*to[i]);
    *to[i] = args[i];
  }
  for (int i = 0; i < kTypes; ++i) {
    PyObject *t = PyTuple_GET_ITEM(args[6], i);
    Py_INCREF(t);
    Py_XDECREF(g_dtypes[i]);
    g_dtypes[i] = t;
  }
  Py_RETURN_NONE;
}

template <PyObject *(*Fn)(PyObject *const *), int N>
PyMethodDef method(const char *name) {
  return {name, (PyCFunction)(void (*)(void))entry<Fn, N>, METH_FASTCALL, nullptr};
}

}  // namespace
