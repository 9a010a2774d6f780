// Python binding of the policy head's calls (a CPython module over torch's tensors).
//
// The calls take a few microseconds on the GPU, and a training or decode step is a row of them:
// through ctypes, with every argument checked in Python, the layer norm of 256 rows cost 8.9 us
// of host time, of which its launch is 2.5 (its kernel runs 3.9); this way it costs 5.5. A call
// checks its tensors, allocates what it returns with torch (on the current stream) and enters the
// C ABI without a Python object in between. A check that fails hands the tensor to the Python
// function that names what is wrong; nothing has been launched by then.

#include "gdn_policy.h"
#include "torch_binding.hpp"

namespace {

const char *last_error() { return gdn_policy_last_error(); }

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
