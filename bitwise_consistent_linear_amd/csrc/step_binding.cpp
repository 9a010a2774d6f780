// Python binding of libgdn_step.so's calls (a CPython module over torch's tensors), for the
// reason that policy_binding.cpp gives: checks, allocations and lists of hundreds of tensors in
// Python would cost more than the launches.

#include "gdn_step.h"
#include "torch_binding.hpp"

#include <algorithm>
#include <vector>

namespace {

const char *last_error() { return gdn_step_last_error(); }

int64_t padded(int64_t c) { return (c + GDN_F8_BLOCK - 1) / GDN_F8_BLOCK * GDN_F8_BLOCK; }

// The shape of the scales of a matrix in 8 bits.
std::array<int64_t, 3> scale_shape(int64_t r, int64_t c) {
  return {(c + 4 * GDN_F8_BLOCK - 1) / (4 * GDN_F8_BLOCK), (r + 3) / 4 * 4, 4};
}

int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}

// quantize_f8(x, format, layout, q, scale, qt, scale_t); layout: 1 rows, 2 columns, 3 both
PyObject *quantize_f8(PyObject *const *a) {
  const Rows x = rows(a[0], "x", kFloat);
  const int64_t M = x.t.size(0), K = x.t.size(1), format = integer(a[1]), layout = integer(a[2]);
  const int dev = x.t.get_device();
  void *const stream = stream_of(dev);
  const at::ScalarType f8 = format == GDN_F8_E5M2 ? at::kFloat8_e5m2 : at::kFloat8_e4m3fn;
  auto call = [&](Out &q, Out &s, Out &qt, Out &st) {
    check(gdn_quantize_f8(x.t.data_ptr(), M, K, x.stride, code(x.t.scalar_type()),
                          (int32_t)format, q.get<uint8_t>(), s.get<uint8_t>(), qt.get<uint8_t>(),
                          st.get<uint8_t>(), stream));
  };
  Out none;
  if (layout == 1) {
    if (given(a[5]) || given(a[6])) value_error("layout 'rows' has no qt and scale_t");
    Out q(a[3], "q", f8, {M, padded(K)}, dev);
    Out s(a[4], "scale", at::kFloat8_e8m0fnu, scale_shape(M, K), dev);
    call(q, s, none, none);
    return tuple(q, s);
  }
  if (layout == 2 && (given(a[3]) || given(a[4])))
    value_error("layout 'columns' has no q and scale");
  Out qt(a[5], "qt", f8, {K, padded(M)}, dev);
  Out st(a[6], "scale_t", at::kFloat8_e8m0fnu, scale_shape(K, M), dev);
  if (layout == 2) {
    call(none, none, qt, st);
    return tuple(qt, st);
  }
  Out q(a[3], "q", f8, {M, padded(K)}, dev);
  Out s(a[4], "scale", at::kFloat8_e8m0fnu, scale_shape(M, K), dev);
  call(q, s, qt, st);
  return tuple(q, s, qt, st);
}

// linear_f8(xq, x_scale, wq, w_scale, bf16, y)
PyObject *linear_f8(PyObject *const *a) {
  const at::Tensor &xq = need(a[0], "xq", kF8, 2), &wq = need(a[2], "wq", kE4m3, 2);
  const int64_t M = xq.size(0), K = xq.size(1), N = wq.size(0);
  const int dev = xq.get_device();
  void *const stream = stream_of(dev);
  if (wq.size(1) != K)
    value_error("xq has rows of " + std::to_string(K) + " values but wq is " +
                std::to_string(N) + " x " + std::to_string(wq.size(1)));
  take(a[2], "wq", kE4m3, {N, K}, dev);
  const void *xs = take(a[1], "x_scale", kE8m0, scale_shape(M, K), dev);
  const void *ws = take(a[3], "w_scale", kE8m0, scale_shape(N, K), dev);
  const at::ScalarType yt = flag(a[4]) ? at::kBFloat16 : at::kFloat;
  Out y(a[5], "y", yt, {M, N}, dev);
  check(gdn_linear_f8_fwd(M, N, K, xq.scalar_type() == at::kFloat8_e5m2 ? GDN_F8_E5M2 : GDN_F8_E4M3,
                          static_cast<const uint8_t *>(xq.data_ptr()),
                          static_cast<const uint8_t *>(xs),
                          static_cast<const uint8_t *>(wq.data_ptr()),
                          static_cast<const uint8_t *>(ws), code(yt), y.get(), stream));
  return y.release();
}

// linear_f8_bwd(dy, wtq, wt_scale, xtq, xt_scale, format, dx_bf16, dw_bf16, dx, dw, workspace)
PyObject *linear_f8_bwd(PyObject *const *a) {
  const Rows dy = rows(a[0], "dy", kFloat);
  const int64_t M = dy.t.size(0), N = dy.t.size(1);
  const int dev = dy.t.get_device();
  void *const stream = stream_of(dev);
  const bool wants_dx = given(a[1]), wants_dw = given(a[3]);
  if (!wants_dx && !wants_dw) value_error("wtq or xtq is required");
  if ((!wants_dx && (given(a[2]) || given(a[8]))) || (!wants_dw && (given(a[4]) || given(a[9]))))
    value_error("a scale or a gradient is given without its 8-bit operand");
  const at::Tensor &one = need(a[wants_dx ? 1 : 3], wants_dx ? "wtq" : "xtq", kE4m3, 2);
  const int64_t K = one.size(0);
  const uint8_t *wtq = nullptr, *wts = nullptr, *xtq = nullptr, *xts = nullptr;
  auto bytes = [&](PyObject *o, const char *name, Types types, at::IntArrayRef shape) {
    return static_cast<const uint8_t *>(take(o, name, types, shape, dev));
  };
  if (wants_dx) {
    wtq = bytes(a[1], "wtq", kE4m3, {K, padded(N)});
    wts = bytes(a[2], "wt_scale", kE8m0, scale_shape(K, N));
  }
  if (wants_dw) {
    xtq = bytes(a[3], "xtq", kE4m3, {K, padded(M)});
    xts = bytes(a[4], "xt_scale", kE8m0, scale_shape(K, M));
  }
  const at::ScalarType xt = flag(a[6]) ? at::kBFloat16 : at::kFloat;
  const at::ScalarType wt = flag(a[7]) ? at::kBFloat16 : at::kFloat;
  const gdn_linear_f8_shape_t shape = {M, N, K, dy.stride, code(dy.t.scalar_type()),
                                       (int32_t)integer(a[5]), code(xt), code(wt)};
  auto call = [&](Out &dx, Out &dw) {
    const Workspace ws = workspace(
        a[10], dev, [&](size_t *n) { return gdn_linear_f8_bwd_workspace(&shape, n); });
    check(gdn_linear_f8_bwd(&shape, dy.t.data_ptr(), wtq, wts, xtq, xts, dx.get(), dw.get(),
                            ws.ptr, ws.bytes, stream));
    return tuple(dx, dw);
  };
  Out none;
  if (!wants_dw) {
    Out dx(a[8], "dx", xt, {M, K}, dev);
    return call(dx, none);
  }
  Out dw(a[9], "dw", wt, {N, K}, dev);
  if (!wants_dx) return call(none, dw);
  Out dx(a[8], "dx", xt, {M, K}, dev);
  return call(dx, dw);
}

// A parameter of the draw: a number for all rows, or a tensor with one for each.
struct Parameter {
  double all;
  const void *each;
};
Parameter parameter(PyObject *o, const char *name, Types types, int64_t M, int dev, double off) {
  if (THPVariable_Check(o)) return {off, take(o, name, types, {M}, dev)};
  return {number(o), nullptr};
}

// sample_tokens(logits, u, temperature, top_k, top_p, min_p, id64, ids, logp, workspace)
PyObject *sample_tokens(PyObject *const *a) {
  const Rows z = rows(a[0], "logits", kFloat);
  const int64_t M = z.t.size(0);
  const int dev = z.t.get_device();
  void *const stream = stream_of(dev);
  const void *u = take(a[1], "u", kReal, {M}, dev);
  const Parameter T = parameter(a[2], "temperature", kF32, M, dev, 1.0);
  const Parameter p = parameter(a[4], "top_p", kF32, M, dev, 1.0);
  const Parameter least = parameter(a[5], "min_p", kF32, M, dev, 0.0);
  const bool each_k = THPVariable_Check(a[3]);
  const void *ks = each_k ? take(a[3], "top_k", kI32, {M}, dev) : nullptr;
  const int64_t k = each_k ? 0 : integer(a[3]);
  if (k < 0) value_error("top_k must be >= 0, got " + std::to_string(k));
  const bool id64 = flag(a[6]);
  Out ids(a[7], "ids", id64 ? at::kLong : at::kInt, {M}, dev);
  Out logp(a[8], "logp", at::kFloat, {M}, dev);
  const gdn_sample_shape_t shape = {M, z.t.size(1), z.stride, code(z.t.scalar_type()),
                                    (int32_t)THPVariable_Unpack(a[1]).element_size(),
                                    id64 ? 8 : 4, (int32_t)std::min<int64_t>(k, INT32_MAX), T.all,
                                    p.all, least.all};
  const Workspace ws = workspace(
      a[9], dev, [&](size_t *n) { return gdn_sample_tokens_workspace(&shape, n); });
  check(gdn_sample_tokens(&shape, z.t.data_ptr(), u, static_cast<const float *>(T.each),
                          static_cast<const int32_t *>(ks), static_cast<const float *>(p.each),
                          static_cast<const float *>(least.each), ids.get(), logp.get<float>(),
                          ws.ptr, ws.bytes, stream));
  return tuple(ids, logp);
}

// A list or tuple of tensors.
class List {
 public:
  List(PyObject *o, const char *name) : name_(name) {
    if (!PyList_Check(o) && !PyTuple_Check(o)) {
      PyErr_Format(PyExc_TypeError, "%s must be a list or tuple of tensors", name);
      throw Refused{};
    }
    list_ = o;
    size_ = PySequence_Fast_GET_SIZE(o);
  }
  int64_t size() const { return size_; }
  // The i-th, a dense tensor on GPU `dev` (-1: any) of `numel` values (-1: any).
  const at::Tensor &at(int64_t i, Types types, int64_t numel, int dev) const {
    PyObject *o = PySequence_Fast_GET_ITEM(list_, i);
    if (THPVariable_Check(o)) {
      const at::Tensor &t = THPVariable_Unpack(o);
      if (t.is_cuda() && (dev < 0 || t.get_device() == dev) && admits(types, t.scalar_type()) &&
          t.is_contiguous() && (numel < 0 || t.numel() == numel))
        return t;
    }
    refuse_at(i, types, numel, dev);
  }

 private:
  [[noreturn]] void refuse_at(int64_t i, Types types, int64_t numel, int dev) const {
    PyObject *o = PySequence_Fast_GET_ITEM(list_, i);
    const std::string name = std::string(name_) + "[" + std::to_string(i) + "]";
    int dim = 1;
    if (THPVariable_Check(o)) {
      const at::Tensor &t = THPVariable_Unpack(o);
      dim = (int)t.dim();
      if (t.is_cuda() && dev >= 0 && t.get_device() != dev)
        value_error(name + " is on GPU " + std::to_string(t.get_device()) + ", expected GPU " +
                    std::to_string(dev));
      if (t.is_cuda() && admits(types, t.scalar_type()) && t.is_contiguous())
        value_error(name + " must have " + std::to_string(numel) + " values, got " +
                    std::to_string(t.numel()));
    }
    refuse(g_need, Py_BuildValue("(OsOi)", o, name.c_str(), g_dtypes[types], dim));
  }

  PyObject *list_;
  const char *name_;
  int64_t size_;
};

int current_device() {
  PyObject *r = PyObject_CallNoArgs(g_device);
  const long d = r ? PyLong_AsLong(r) : -1;
  Py_XDECREF(r);
  if (PyErr_Occurred()) throw Refused{};
  return (int)d;
}

// The values' type in a list whose tensors have one type.
Types one_type(const List &list, int64_t i, int dev) {
  return alone(list.at(i, kFloat, -1, dev).scalar_type());
}

// grad_norm(grads, max_norm, norm, factor, workspace)
PyObject *grad_norm(PyObject *const *a) {
  const List grads(a[0], "grads");
  const int64_t n = grads.size();
  const int dev = n ? (int)grads.at(0, kFloat, -1, -1).get_device() : current_device();
  void *const stream = stream_of(dev);
  const Types type = n ? one_type(grads, 0, dev) : kF32;
  std::vector<gdn_grad_tensor_t> list(n);
  for (int64_t i = 0; i < n; ++i) {
    const at::Tensor &g = grads.at(i, type, -1, dev);
    list[i] = {g.numel(), g.data_ptr()};
  }
  const double most = number(a[1]);
  Out norm(a[2], "norm", at::kFloat, {1}, dev), factor(a[3], "factor", at::kFloat, {1}, dev);
  const Workspace ws = workspace(
      a[4], dev, [&](size_t *b) { return gdn_grad_norm_workspace(list.data(), n, b); });
  check(gdn_grad_norm(list.data(), n, type == kBf16 ? GDN_DTYPE_BF16 : GDN_DTYPE_F32, most,
                      norm.get<float>(), factor.get<float>(), ws.ptr, ws.bytes, stream));
  return tuple(norm, factor);
}

// What autograd knows of a tensor that a kernel has written to.
void written(const at::Tensor &t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// adamw_step(params, grads, m, v, step, m_scale, v_scale, master, lr, beta1, beta2, eps,
//            weight_decay, grad_scale)
PyObject *adamw_step(PyObject *const *a) {
  const List params(a[0], "params"), grads(a[1], "grads"), ms(a[2], "m"), vs(a[3], "v");
  const int64_t n = params.size();
  if (grads.size() != n || ms.size() != n || vs.size() != n)
    value_error("params, grads, m and v must have as many tensors");
  if (n == 0) Py_RETURN_NONE;
  const int dev = (int)params.at(0, kFloat, -1, -1).get_device();
  void *const stream = stream_of(dev);
  const Types pt = one_type(params, 0, dev), gt = one_type(grads, 0, dev);
  const bool eight = given(a[5]);
  if (eight != given(a[6])) value_error("m_scale and v_scale are given together or not at all");
  std::vector<gdn_adamw_tensor_t> list(n);
  for (int64_t i = 0; i < n; ++i) {
    const at::Tensor &p = params.at(i, pt, -1, dev);
    const int64_t size = p.numel();
    list[i] = {size, p.data_ptr(), grads.at(i, gt, size, dev).data_ptr(),
               ms.at(i, eight ? kE4m3 : kF32, size, dev).data_ptr(),
               vs.at(i, eight ? kBytes : kF32, size, dev).data_ptr(), nullptr, nullptr, nullptr};
  }
  auto more = [&](PyObject *o, const char *name, float *gdn_adamw_tensor_t::*to, int64_t per) {
    const List values(o, name);
    if (values.size() != n) value_error(std::string(name) + " must have as many tensors as params");
    for (int64_t i = 0; i < n; ++i)
      list[i].*to = static_cast<float *>(
          values.at(i, kF32, (list[i].numel + per - 1) / per, dev).data_ptr());
  };
  if (eight) {
    more(a[5], "m_scale", &gdn_adamw_tensor_t::m_scale, GDN_ADAMW_BLOCK);
    more(a[6], "v_scale", &gdn_adamw_tensor_t::v_scale, GDN_ADAMW_BLOCK);
  }
  if (given(a[7])) {
    if (pt != kBf16) value_error("master needs bfloat16 params");
    more(a[7], "master", &gdn_adamw_tensor_t::master, 1);
  }
  // a tensor in the list twice would be updated by two workgroups at once
  std::vector<const void *> at;
  for (const gdn_adamw_tensor_t &t : list)
    if (t.numel > 0) at.push_back(t.param);
  std::sort(at.begin(), at.end());
  if (std::adjacent_find(at.begin(), at.end()) != at.end())
    value_error("params has a tensor twice");
  gdn_adamw_shape_t shape = {pt == kBf16 ? GDN_DTYPE_BF16 : GDN_DTYPE_F32,
                             gt == kBf16 ? GDN_DTYPE_BF16 : GDN_DTYPE_F32,
                             eight ? GDN_STATE_8BIT : GDN_STATE_F32, 0, 0.0, number(a[9]),
                             number(a[10]), number(a[11]), number(a[12]), 1};
  const int64_t *step_at = nullptr;
  const float *lr_at = nullptr;
  if (THPVariable_Check(a[4]))
    step_at = static_cast<const int64_t *>(take(a[4], "step", kI64, {1}, dev));
  else
    shape.step = integer(a[4]);
  if (THPVariable_Check(a[8]))
    lr_at = static_cast<const float *>(take(a[8], "lr", kF32, {1}, dev));
  else
    shape.lr = number(a[8]);
  const float *factor = static_cast<const float *>(take_if(a[13], "grad_scale", kF32, {1}, dev));
  check(gdn_adamw_step(&shape, list.data(), n, factor, step_at, lr_at, stream));
  auto wrote = [&](PyObject *o) {
    if (given(o))
      for (int64_t i = 0; i < n; ++i) written(THPVariable_Unpack(PySequence_Fast_GET_ITEM(o, i)));
  };
  for (int i : {0, 2, 3, 5, 6, 7}) wrote(a[i]);
  Py_RETURN_NONE;
}

// adamw_state_values(codes, scale, out)
PyObject *adamw_state_values(PyObject *const *a) {
  if (!THPVariable_Check(a[0])) refuse(g_need, Py_BuildValue("(OsOi)", a[0], "codes", g_dtypes[kE4m3], 1));
  const at::Tensor &any = THPVariable_Unpack(a[0]);
  const Types type = any.scalar_type() == at::kByte ? kBytes : kE4m3;
  const at::Tensor &codes = need(a[0], "codes", type, (int)any.dim());
  const int dev = codes.get_device();
  void *const stream = stream_of(dev);
  const int64_t n = codes.numel();
  const void *scale =
      take(a[1], "scale", kF32, {(n + GDN_ADAMW_BLOCK - 1) / GDN_ADAMW_BLOCK}, dev);
  Out out(a[2], "out", at::kFloat, codes.sizes(), dev);
  check(gdn_adamw_state_values(static_cast<const uint8_t *>(codes.data_ptr()),
                               static_cast<const float *>(scale), n,
                               type == kBytes ? GDN_MOMENT_V : GDN_MOMENT_M, out.get<float>(),
                               stream));
  return out.release();
}

PyMethodDef g_methods[] = {
    {"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, nullptr},
    method<quantize_f8, 7>("quantize_f8"),
    method<linear_f8, 6>("linear_f8"),
    method<linear_f8_bwd, 11>("linear_f8_bwd"),
    method<sample_tokens, 10>("sample_tokens"),
    method<grad_norm, 5>("grad_norm"),
    method<adamw_step, 14>("adamw_step"),
    method<adamw_state_values, 3>("adamw_state_values"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_step_binding",
                        "The calls of libgdn_step.so over torch tensors.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step_binding(void) { return PyModule_Create(&g_module); }
