// Python binding of the policy head's calls (a CPython module over torch's tensors).
//
// The calls take a few microseconds on the GPU, and a training or decode step is a row of them:
// through ctypes, with every argument checked in Python, the layer norm of 256 rows cost 8.9 us
// of host time, of which its launch is 2.5 (its kernel runs 3.9); this way it costs 5.5. A call
// checks its tensors, allocates what it returns with torch (on the current stream) and enters the
// C ABI without a Python object in between. A check that fails hands the tensor to the Python
// function that names what is wrong; nothing has been launched by then.

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>

#include "gdn_policy.h"

namespace {

struct Refused {};  // a Python exception is set

// What setup() hands over: torch's functions for the current device and its raw stream, the
// functions that raise for a tensor, the error class, and tuples of dtypes for those functions.
PyObject *g_device, *g_stream, *g_refuse, *g_rows, *g_need, *g_error;
enum Types { kF32, kFloat, kI8, kInts, kFlags, kI32, kBytes, kBf16, kTypes };
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
    default: return t == at::kBFloat16;
  }
}
Types alone(at::ScalarType t) { return t == at::kBFloat16 ? kBf16 : kF32; }
int32_t code(at::ScalarType t) { return t == at::kBFloat16 ? GDN_DTYPE_BF16 : GDN_DTYPE_F32; }

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

bool given(PyObject *o) { return o != Py_None; }

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
void *take_if(PyObject *o, const char *name, Types types, at::IntArrayRef shape, int dev) {
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
      ptr_ = take(o, name, type == at::kChar ? kI8 : alone(type), shape, dev);
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
  PyObject *e = PyObject_CallFunction(g_error, "is", (int)st, gdn_policy_last_error());
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

double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}
bool flag(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{};
  return v != 0;
}

// norm_fwd(x, weight, bias, eps, layer, y, mean, rstd)
PyObject *norm_fwd(PyObject *const *a) {
  const Rows x = rows(a[0], "x", kFloat);
  const int64_t M = x.t.size(0), D = x.t.size(1);
  const int dev = x.t.get_device();
  void *const stream = stream_of(dev);
  const bool layer = flag(a[4]);
  const double eps = number(a[3]);
  void *w = take(a[1], "weight", kFloat, {D}, dev);
  const at::ScalarType wt = THPVariable_Unpack(a[1]).scalar_type(), xt = x.t.scalar_type();
  void *b = take_if(a[2], "bias", alone(wt), {D}, dev);
  if (!layer && given(a[6])) value_error("kind 'rms' has no mean");
  Out none, y(a[5], "y", xt, {M, D}, dev), rstd(a[7], "rstd", at::kFloat, {M}, dev);
  const gdn_norm_shape_t shape = {M, (int32_t)std::min<int64_t>(D, INT32_MAX),
                                  layer ? GDN_NORM_LAYER : GDN_NORM_RMS, code(xt), code(wt)};
  auto call = [&](Out &mean) {
    check(gdn_layer_norm_fwd(&shape, x.t.data_ptr(), x.stride, w, b, eps, y.get(),
                             mean.get<float>(), rstd.get<float>(), stream));
    return tuple(y, mean, rstd);
  };
  if (!layer) return call(none);
  Out mean(a[6], "mean", at::kFloat, {M}, dev);
  return call(mean);
}

// norm_bwd(dy, x, weight, mean, rstd, layer, bias, dx, d_weight, d_bias, workspace)
PyObject *norm_bwd(PyObject *const *a) {
  const Rows x = rows(a[1], "x", kFloat);
  const at::ScalarType xt = x.t.scalar_type();
  const Rows dy = rows(a[0], "dy", alone(xt));
  const int64_t M = x.t.size(0), D = x.t.size(1);
  const int dev = x.t.get_device();
  if (dy.t.sizes() != x.t.sizes() || dy.t.get_device() != dev)
    value_error("dy and x differ, in shape or GPU");
  void *const stream = stream_of(dev);
  const bool layer = flag(a[5]), bias = flag(a[6]);
  void *w = take(a[2], "weight", kFloat, {D}, dev);
  const at::ScalarType wt = THPVariable_Unpack(a[2]).scalar_type();
  if (!layer && given(a[3])) value_error("kind 'rms' has no mean");
  float *mean = layer ? static_cast<float *>(take(a[3], "mean", kF32, {M}, dev)) : nullptr;
  float *rstd = static_cast<float *>(take(a[4], "rstd", kF32, {M}, dev));
  if (!bias && given(a[9])) value_error("d_bias is given but bias is False");
  Out none, dx(a[7], "dx", xt, {M, D}, dev), dw(a[8], "d_weight", at::kFloat, {D}, dev);
  const gdn_norm_shape_t shape = {M, (int32_t)std::min<int64_t>(D, INT32_MAX),
                                  layer ? GDN_NORM_LAYER : GDN_NORM_RMS, code(xt), code(wt)};
  auto call = [&](Out &db) {
    const Workspace ws = workspace(
        a[10], dev, [&](size_t *n) { return gdn_layer_norm_bwd_workspace(&shape, n); });
    check(gdn_layer_norm_bwd(&shape, dy.t.data_ptr(), dy.stride, x.t.data_ptr(), x.stride, w,
                             mean, rstd, dx.get(), dw.get<float>(), db.get<float>(), ws.ptr,
                             ws.bytes, stream));
    return tuple(dx, dw, db);
  };
  if (!bias) return call(none);
  Out db(a[9], "d_bias", at::kFloat, {D}, dev);
  return call(db);
}

// quantize_rows(x, xq, scale)
PyObject *quantize_rows(PyObject *const *a) {
  const Rows x = rows(a[0], "x", kFloat);
  const int64_t M = x.t.size(0), K = x.t.size(1);
  const int dev = x.t.get_device();
  void *const stream = stream_of(dev);
  const int64_t padded = (K + GDN_I8_K_ALIGN - 1) / GDN_I8_K_ALIGN * GDN_I8_K_ALIGN;
  Out xq(a[1], "xq", at::kChar, {M, padded}, dev), scale(a[2], "scale", at::kFloat, {M}, dev);
  check(gdn_quantize_rows(x.t.data_ptr(), M, K, x.stride, code(x.t.scalar_type()),
                          xq.get<int8_t>(), scale.get<float>(), stream));
  return tuple(xq, scale);
}

// linear_i8(xq, x_scale, wq, w_scale, bf16, y, workspace)
PyObject *linear_i8(PyObject *const *a) {
  const at::Tensor &xq = need(a[0], "xq", kI8, 2), &wq = need(a[2], "wq", kI8, 2);
  const int64_t M = xq.size(0), K = xq.size(1), N = wq.size(0);
  const int dev = xq.get_device();
  void *const stream = stream_of(dev);
  if (wq.size(1) != K)
    value_error("xq has rows of " + std::to_string(K) + " values but wq is " +
                std::to_string(N) + " x " + std::to_string(wq.size(1)));
  take(a[2], "wq", kI8, {N, K}, dev);
  const void *xs = take(a[1], "x_scale", kF32, {M}, dev), *ws = take(a[3], "w_scale", kF32, {N}, dev);
  const at::ScalarType yt = flag(a[4]) ? at::kBFloat16 : at::kFloat;
  Out y(a[5], "y", yt, {M, N}, dev);
  const Workspace room = workspace(
      a[6], dev, [&](size_t *bytes) { return gdn_linear_i8_fwd_workspace(M, N, K, bytes); });
  check(gdn_linear_i8_fwd(M, N, K, static_cast<const int8_t *>(xq.data_ptr()),
                          static_cast<const float *>(xs), static_cast<const int8_t *>(wq.data_ptr()),
                          static_cast<const float *>(ws), code(yt), y.get(), room.ptr, room.bytes,
                          stream));
  return y.release();
}

struct Logits {
  Rows z;
  const void *ids;
  int dev;
  gdn_logprob_shape_t shape;
};
Logits logits_of(PyObject *logits, PyObject *ids, PyObject *scale) {
  const Rows z = rows(logits, "logits", kFloat);
  const int64_t M = z.t.size(0);
  const int dev = z.t.get_device();
  const void *p = take(ids, "ids", kInts, {M}, dev);
  return {z, p, dev, {M, z.t.size(1), z.stride, code(z.t.scalar_type()),
                      (int32_t)THPVariable_Unpack(ids).element_size(), number(scale)}};
}

// logprob_fwd(logits, ids, scale, entropy, logp, lse, workspace)
PyObject *logprob_fwd(PyObject *const *a) {
  const Logits g = logits_of(a[0], a[1], a[2]);
  void *const stream = stream_of(g.dev);
  const int64_t M = g.shape.rows;
  Out none, logp(a[4], "logp", at::kFloat, {M}, g.dev), lse(a[5], "lse", at::kFloat, {M}, g.dev);
  const Workspace ws = workspace(
      a[6], g.dev, [&](size_t *n) { return gdn_token_logprob_fwd_workspace(&g.shape, n); });
  auto call = [&](Out &ent) {
    check(gdn_token_logprob_fwd(&g.shape, g.z.t.data_ptr(), g.ids, logp.get<float>(),
                                lse.get<float>(), ent.get<float>(), ws.ptr, ws.bytes,
                                stream));
    return tuple(logp, lse, ent);
  };
  if (!flag(a[3])) return call(none);
  Out ent(Py_None, "entropy", at::kFloat, {M}, g.dev);
  return call(ent);
}

// logprob_bwd(logits, ids, lse, d_logp, scale, entropy, d_entropy, d_logits)
PyObject *logprob_bwd(PyObject *const *a) {
  const Logits g = logits_of(a[0], a[1], a[4]);
  void *const stream = stream_of(g.dev);
  const int64_t M = g.shape.rows;
  auto row = [&](PyObject *o, const char *name) {
    return static_cast<const float *>(take(o, name, kF32, {M}, g.dev));
  };
  const float *lse = row(a[2], "lse"), *d_logp = row(a[3], "d_logp"), *ent = nullptr,
              *d_ent = nullptr;
  if (given(a[6])) {
    if (!given(a[5])) value_error("d_entropy needs the entropy that token_logprob_fwd returned");
    ent = row(a[5], "entropy");
    d_ent = row(a[6], "d_entropy");
  }
  Out d(a[7], "d_logits", g.z.t.scalar_type(), g.z.t.sizes(), g.dev);
  check(gdn_token_logprob_bwd(&g.shape, g.z.t.data_ptr(), g.ids, lse, d_logp, ent, d_ent, d.get(),
                              stream));
  return d.release();
}

// The arguments that both directions of the policy loss begin with:
// (logp, old_logp, advantages, ref_logp, entropy, mask, cu_seqlens, reduction, clip_low,
//  clip_high, dual_clip, kl_coef, entropy_coef)
constexpr int kPolicyArgs = 13;
struct Policy {
  int dev;
  int64_t T, N;
  const float *logp, *old, *adv, *ref, *ent;
  const uint8_t *mask;
  const int32_t *cu;
  gdn_policy_shape_t shape;
};
Policy policy_of(PyObject *const *a) {
  Policy p;
  const at::Tensor &t = need(a[0], "logp", kF32, 1);
  p.dev = t.get_device();
  p.T = t.size(0);
  p.N = 1;
  auto values = [&](PyObject *o, const char *name) {
    return static_cast<const float *>(take_if(o, name, kF32, {p.T}, p.dev));
  };
  p.logp = static_cast<const float *>(t.data_ptr());
  p.old = static_cast<const float *>(take(a[1], "old_logp", kF32, {p.T}, p.dev));
  p.adv = static_cast<const float *>(take(a[2], "advantages", kF32, {p.T}, p.dev));
  p.ref = values(a[3], "ref_logp");
  p.ent = values(a[4], "entropy");
  p.mask = static_cast<const uint8_t *>(take_if(a[5], "mask", kFlags, {p.T}, p.dev));
  p.cu = nullptr;
  if (given(a[6])) {
    const at::Tensor &cu = need(a[6], "cu_seqlens", kI32, 1);
    p.N = cu.size(0) - 1;
    p.cu = static_cast<const int32_t *>(take(a[6], "cu_seqlens", kI32, {p.N + 1}, p.dev));
    if (p.N < 0) value_error("cu_seqlens must have at least one value");
  }
  p.shape = {p.T, p.N, (int32_t)number(a[7]), 0, number(a[8]), number(a[9]),
             given(a[10]) ? number(a[10]) : 0.0, given(a[3]) ? number(a[11]) : 0.0,
             given(a[4]) ? number(a[12]) : 0.0};
  return p;
}

// policy_fwd(..., stats, weight, workspace)
PyObject *policy_fwd(PyObject *const *a) {
  const Policy p = policy_of(a);
  void *const stream = stream_of(p.dev);
  a += kPolicyArgs;
  Out stats(a[0], "stats", at::kFloat, {5}, p.dev), weight(a[1], "weight", at::kFloat, {p.N}, p.dev);
  const Workspace ws = workspace(
      a[2], p.dev, [&](size_t *n) { return gdn_policy_loss_workspace(&p.shape, n); });
  check(gdn_policy_loss_fwd(&p.shape, p.logp, p.old, p.adv, p.ref, p.ent, p.mask, p.cu,
                            stats.get<float>(), weight.get<float>(), ws.ptr, ws.bytes,
                            stream));
  return tuple(stats, weight);
}

// policy_bwd(..., weight, d_loss, d_logp, d_entropy)
PyObject *policy_bwd(PyObject *const *a) {
  const Policy p = policy_of(a);
  const bool entropy = given(a[4]);
  void *const stream = stream_of(p.dev);
  a += kPolicyArgs;
  const float *w = static_cast<const float *>(take(a[0], "weight", kF32, {p.N}, p.dev));
  const double d_loss = number(a[1]);
  if (!entropy && given(a[3])) value_error("d_entropy is given without an entropy");
  Out none, dl(a[2], "d_logp", at::kFloat, {p.T}, p.dev);
  auto call = [&](Out &de) {
    check(gdn_policy_loss_bwd(&p.shape, p.logp, p.old, p.adv, p.ref, p.mask, p.cu, w, d_loss,
                              dl.get<float>(), de.get<float>(), stream));
    return tuple(dl, de);
  };
  if (!entropy) return call(none);
  Out de(a[3], "d_entropy", at::kFloat, {p.T}, p.dev);
  return call(de);
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

PyMethodDef g_methods[] = {
    {"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, nullptr},
    method<norm_fwd, 8>("norm_fwd"),
    method<norm_bwd, 11>("norm_bwd"),
    method<quantize_rows, 3>("quantize_rows"),
    method<linear_i8, 7>("linear_i8"),
    method<logprob_fwd, 7>("logprob_fwd"),
    method<logprob_bwd, 8>("logprob_bwd"),
    method<policy_fwd, kPolicyArgs + 3>("policy_fwd"),
    method<policy_bwd, kPolicyArgs + 4>("policy_bwd"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_policy_binding",
                        "The policy head's calls over torch tensors.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__policy_binding(void) { return PyModule_Create(&g_module); }
